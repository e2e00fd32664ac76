// fd_api.cu -- the extern "C" entry points declared in include/fd.h: host-side
// argument checks, the split planner and the dispatch to the kernels.  No
// entry point allocates memory or synchronises (except fd_device_status).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fd.h"
#include "fd_internal.h"

namespace {

using fd::kTile;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int current_sm_count() {
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return -1;
    if (dev >= 0 && dev < 64) cache[dev] = n;
    return n;
}

int check_shape(int B, int Hq, int Hkv, int L_max, int d) {
    if (B < 0 || Hq <= 0 || Hkv <= 0 || L_max < 0) return FD_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return FD_ERR_INVALID_ARG;
    if (B > 65535 || Hkv > 65535 || L_max > (1 << 30)) return FD_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FD_ERR_UNSUPPORTED;
    if (Hq / Hkv > 8) return FD_ERR_UNSUPPORTED;
    return FD_OK;
}

// Chunk plan shared by the planner queries, the workspace sizes and the
// launches.  `chunk_fixed` = 0 means per-sequence chunks of
// ceil(L_b / splits) rounded up to 64 tokens.
struct Plan {
    int splits;
    int chunk_fixed;
};

// The "Flash Decoding" tutorial (section 6, misconception 2) asks for a chunk
// count that keeps every compute unit busy, chunks of at least a few hundred
// tokens, and no more chunks than that: each costs merge work.  Here that is
// a cost model over whole 64-token tiles, in units of one tile's bytes at
// the GPU's full HBM bandwidth.  A wave of n CTAs with c tiles each takes
//   c * max(n, r),
// r being the number of CTAs whose copy pipelines together saturate HBM
// (a lone CTA streams at about 1/r of the GPU's bandwidth); CTAs beyond
// the resident slots form further waves; each chunk adds a small fixed cost
// and so does each wave (wave_tiles > 0: that many tiles of a CTA's time,
// for the passes whose CTAs are bound by their SM's issue, not by HBM).
// So: few, long chunks while HBM stays saturated, and no small trailing
// wave.  Ragged batches (lengths unknown on the host) take
// chunks such that sequences of length L_max span about four waves, so the
// hardware block scheduler can even out the load.
Plan plan_uncached(int B, int Hkv, int L_max, int requested, bool ragged, int ctas_per_sm, int sms, double r,
                   bool fill_slots, double wave_tiles);

// The cost model walks every chunk count (thousands for a 1M-token cache):
// its answers are remembered per thread for the last few argument sets.
Plan plan(int B, int Hkv, int L_max, int requested, bool ragged, int ctas_per_sm, int sms, double r,
          bool fill_slots = false, double wave_tiles = 0.0) {
    struct Entry {
        int B, Hkv, L_max, requested, ragged, ctas_per_sm, sms, fill_slots;
        double r, wave_tiles;
        Plan pl;
        bool used;
    };
    constexpr int kEntries = 8;
    thread_local Entry cache[kEntries] = {};
    thread_local int next = 0;
    for (const Entry& e : cache)
        if (e.used && e.B == B && e.Hkv == Hkv && e.L_max == L_max && e.requested == requested &&
            e.ragged == (int)ragged && e.ctas_per_sm == ctas_per_sm && e.sms == sms &&
            e.fill_slots == (int)fill_slots && e.r == r && e.wave_tiles == wave_tiles)
            return e.pl;
    const Plan pl = plan_uncached(B, Hkv, L_max, requested, ragged, ctas_per_sm, sms, r, fill_slots, wave_tiles);
    cache[next] = Entry{B, Hkv, L_max, requested, (int)ragged, ctas_per_sm, sms, (int)fill_slots, r, wave_tiles, pl,
                        true};
    next = (next + 1) % kEntries;
    return pl;
}

Plan plan_uncached(int B, int Hkv, int L_max, int requested, bool ragged, int ctas_per_sm, int sms, double r,
                   bool fill_slots, double wave_tiles) {
    Plan pl{1, 0};
    if (requested > 0) {
        pl.splits = requested;
        return pl;
    }
    const int tiles = (L_max + kTile - 1) / kTile;
    if (tiles <= 4 || sms <= 0) return pl;
    const long units = (long)B * Hkv;
    const long slots = (long)sms * (ctas_per_sm > 0 ? ctas_per_sm : 1);
    const int min_chunk_tiles = 4;  // 256 tokens
    int best_chunk = tiles;
    if (!ragged) {
        const double wave_cost = wave_tiles > 0.0 ? wave_tiles * (double)slots : 400.0, split_cost = 20.0;
        double best = 1e300;
        const int max_s = tiles / min_chunk_tiles;
        for (int S = 1; S <= max_s; ++S) {
            const int ct = (tiles + S - 1) / S;
            const int s_eff = (tiles + ct - 1) / ct;
            if (s_eff != S) continue;  // same chunk as a smaller S
            const long ctas = units * s_eff;
            const long full = ctas / slots, rest = ctas % slots;
            double cost = (double)full * ct * (slots > r ? (double)slots : r);
            if (rest) cost += (double)ct * (rest > r ? (double)rest : r);
            cost += wave_cost * (double)(full + (rest ? 1 : 0)) + split_cost * s_eff * units / (double)slots;
            if (cost < best - 1e-9) {
                best = cost;
                best_chunk = ct;
            }
        }
        // (bf16 pass) A single wave that leaves resident slots empty (some
        // SMs run two CTAs, others one) streams below the bandwidth the full
        // machine reaches; twice the chunks fill every slot once and most of
        // them a second time.  A context-length ladder (B = 1, 8, 32;
        // L = 4K..1M) measured this 5-6% faster at B = 32 and ~1% at B = 8,
        // and slower only where the halved chunks fall below 64 tiles, which
        // stay as they are.
        const int S1 = (tiles + best_chunk - 1) / best_chunk;
        const long n1 = units * S1;
        const int ct2 = (best_chunk + 1) / 2;
        const int S2 = (tiles + ct2 - 1) / ct2;
        const long n2 = units * S2;
        if (fill_slots && n1 >= sms && n1 < slots && ct2 >= 64 && n2 >= slots && n2 % slots >= slots / 2)
            best_chunk = ct2;
    } else {
        // aim at ~4 waves for sequences of length L_max, chunks of 8..256 tiles
        // (on a batch of lengths U[L_max/8, L_max] fewer, longer chunks win
        // until about four waves; shorter sequences then fill the gaps)
        long ct = (units * tiles + 4 * slots - 1) / (4 * slots);
        if (ct < 8) ct = 8;
        if (ct > 256) ct = 256;
        if (ct > tiles) ct = tiles;
        best_chunk = (int)ct;
    }
    pl.chunk_fixed = best_chunk * kTile;
    pl.splits = (L_max + pl.chunk_fixed - 1) / pl.chunk_fixed;
    if (pl.splits <= 1) pl = Plan{1, 0};
    return pl;
}

// CTAs that saturate HBM.  On GB300 a CTA of the d=128 pass (3 stages of
// 32 KiB in flight) streams ~64 GB/s alone, so ~110 would do in theory; one
// CTA per SM is the measured safe point (a chunk-count sweep of the 32K and
// 1M-token workloads has its optimum there).  The d=64 pass keeps 2/3 of the
// bytes in flight, so it needs 1.5x as many.
double saturating_ctas(int d, int sms) { return (d == 128 ? 1.0 : 1.5) * (sms > 0 ? sms : 1); }

Plan decode_plan(int B, int Hq, int Hkv, int L_max, int d, int requested, bool ragged) {
    const int sms = current_sm_count();
    const int occ = requested > 0 ? 1 : fd::decode_ctas_per_sm(d, Hq / Hkv, ragged);
    return plan(B, Hkv, L_max, requested, ragged, occ, sms, saturating_ctas(d, sms), true);
}

// The fp8 cache moves d + 4 bytes per row and operand where the bf16 cache
// moves 2d: a tile carries the bytes of a bf16 tile of half the head size.
Plan fp8_plan(int B, int Hq, int Hkv, int L_max, int d, int requested, bool ragged) {
    const int sms = current_sm_count();
    const int occ = requested > 0 ? 1 : fd::fp8_ctas_per_sm(d, ragged);
    return plan(B, Hkv, L_max, requested, ragged, occ, sms, saturating_ctas(d / 2, sms));
}

// The fp4 cache moves d/2 + d/32 bytes per row and operand, but its pass is
// bound by the widening of the codes on the CUDA cores, not by HBM: like the
// top-delta pass it needs every resident CTA slot busy.  (Counting only the
// CTAs that would saturate HBM left 48 of 304 slots empty on the 1M-token and
// FFD caches: 293 -> 250 us and 149 -> 130 us when the chunks fill them.)
// Each further wave costs about 4.5 tiles of a CTA's time (pipeline fill,
// the last tile, the combine): a chunk-count sweep at 3 CTAs/SM measured one
// full wave 7% faster than four on the FFD cache (124.3 vs 133.3 us) and 11%
// faster than two on MHA-32K (40.0 vs 45.0 us).
Plan fp4_plan(int B, int Hq, int Hkv, int L_max, int d, int requested, bool ragged) {
    const int sms = current_sm_count();
    const int occ = requested > 0 ? 1 : fd::fp4_ctas_per_sm(d, ragged);
    return plan(B, Hkv, L_max, requested, ragged, occ, sms, (double)occ * (sms > 0 ? sms : 1), false, 4.5);
}

Plan topdelta_plan(int B, int Hq, int Hkv, int L_max, int d, int requested) {
    const int sms = current_sm_count();
    const int occ = requested > 0 ? 1 : fd::topdelta_ctas_per_sm(d, Hq / Hkv);
    // the fused sparse pass is bound by its instruction issue, not by HBM: it
    // needs every resident CTA slot busy to reach full speed.  A further wave
    // costs it about 20 tiles of a CTA's time (the anchor pass, two pipelines
    // to fill, the last tiles): on the FFD cache one wave of 9 chunks ran
    // 272.7 us against 281.3 us for two waves of 19.
    return plan(B, Hkv, L_max, requested, false, occ, sms, (double)occ * (sms > 0 ? sms : 1), false, 20.0);
}

int to_status(cudaError_t e) { return e == cudaSuccess ? FD_OK : FD_ERR_CUDA; }

enum class Cache { BF16, FP8, FP4 };

Plan cache_plan(Cache cache, int B, int Hq, int Hkv, int L_max, int d, int requested, bool ragged) {
    switch (cache) {
        case Cache::FP8: return fp8_plan(B, Hq, Hkv, L_max, d, requested, ragged);
        case Cache::FP4: return fp4_plan(B, Hq, Hkv, L_max, d, requested, ragged);
        default: return decode_plan(B, Hq, Hkv, L_max, d, requested, ragged);
    }
}

// Chunks per sequence (negative status on bad arguments) and workspace bytes
// (0 on bad arguments) of a dense or paged call over the given cache.
int num_splits_for(Cache cache, int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    const int st = check_shape(B, Hq, Hkv, L_max, d);
    if (st != FD_OK) return -st;
    if (num_splits < 0) return -FD_ERR_INVALID_ARG;
    return cache_plan(cache, B, Hq, Hkv, L_max, d, num_splits, ragged != 0).splits;
}

size_t workspace_for(Cache cache, int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    if (check_shape(B, Hq, Hkv, L_max, d) != FD_OK || num_splits < 0) return 0;
    const Plan pl = cache_plan(cache, B, Hq, Hkv, L_max, d, num_splits, ragged != 0);
    return fd::decode_workspace_bytes(B, Hq, d, pl.splits);
}

// Validates the arguments every decode entry point shares, plans the chunks
// and enqueues the partial pass (+ merge) for the given cache.
int decode_common(fd::DecodeArgs& a, int num_splits, bool ragged, int out_dtype, void* workspace,
                  size_t workspace_bytes, void* stream, Cache cache) {
    const bool quantized = cache != Cache::BF16;  // scale arrays required
    if (out_dtype != FD_OUT_F32 && out_dtype != FD_OUT_BF16) return FD_ERR_INVALID_ARG;
    if (num_splits < 0 || !std::isfinite(a.scale)) return FD_ERR_INVALID_ARG;
    if (a.B > 0 && (!a.q || !a.k || !a.v || !a.out)) return FD_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.out)) return FD_ERR_INVALID_ARG;
    if (quantized && ((a.B > 0 && (!a.k_scales || !a.v_scales)) || !aligned16(a.k_scales) || !aligned16(a.v_scales)))
        return FD_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(a.lse) & 3u) || (reinterpret_cast<uintptr_t>(a.seq_lens) & 3u))
        return FD_ERR_INVALID_ARG;
    // tile copies address cache rows with 32-bit coordinates
    const long long cache_rows = a.page_table ? (long long)a.num_pages * a.Hkv * kTile
                                              : (long long)a.B * a.Hkv * a.L_max;
    if (cache_rows > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    const Plan pl = cache_plan(cache, a.B, a.Hq, a.Hkv, a.L_max, a.D, num_splits, ragged);
    const size_t need = fd::decode_workspace_bytes(a.B, a.Hq, a.D, pl.splits);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace)) return FD_ERR_INVALID_ARG;
    }
    a.splits = pl.splits;
    a.chunk_fixed = pl.chunk_fixed;
    a.out_bf16 = out_dtype == FD_OUT_BF16;
    float* ws = static_cast<float*>(workspace);
    a.part_o = ws;
    a.part_ml = ws ? ws + (size_t)a.B * a.Hq * pl.splits * a.D : nullptr;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return to_status(cache == Cache::FP8   ? fd::launch_decode_fp8(a, st)
                     : cache == Cache::FP4 ? fd::launch_decode_fp4(a, st)
                                           : fd::launch_decode(a, st));
}

// Contiguous cache [B, Hkv, L_max, ...]: K and V (codes for fp8/fp4) and, for
// the quantized caches, their scale arrays.
// The unified-max variant takes a finite fixed max value phi.
constexpr float kMaxAbsPhi = 1e30f;

int dense_entry(Cache cache, const void* q, const void* k, const void* v, const void* k_scales,
                const void* v_scales, const int32_t* seq_lens, int B, int Hq, int Hkv, int L_max, int d,
                float scale, int num_splits, void* out, int out_dtype, float* lse, void* workspace,
                size_t workspace_bytes, void* stream, bool unified = false, float phi = 0.f) {
    const int st = check_shape(B, Hq, Hkv, L_max, d);
    if (st != FD_OK) return st;
    if (unified && !(std::fabs(phi) <= kMaxAbsPhi)) return FD_ERR_INVALID_ARG;
    fd::DecodeArgs a = {};
    a.unified = unified ? 1 : 0;
    a.phi = phi;
    a.q = q;
    a.k = k;
    a.v = v;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.seq_lens = seq_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.L_max = L_max;
    a.D = d;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    return decode_common(a, num_splits, seq_lens != nullptr, out_dtype, workspace, workspace_bytes, stream, cache);
}

// Paged cache: pools [num_pages, Hkv, 64, ...] and a page table [B, max_pages].
int paged_entry(Cache cache, const void* q, const void* k_pages, const void* v_pages, const void* k_scales,
                const void* v_scales, const int32_t* page_table, int max_pages, int num_pages,
                const int32_t* seq_lens, int page_size, int B, int Hq, int Hkv, int d, float scale, int num_splits,
                void* out, int out_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream,
                bool unified = false, float phi = 0.f) {
    if (page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (unified && !(std::fabs(phi) <= kMaxAbsPhi)) return FD_ERR_INVALID_ARG;
    if (max_pages <= 0 || num_pages < 0 || max_pages > (1 << 24)) return FD_ERR_INVALID_ARG;
    const int L_max = max_pages * page_size;
    const int st = check_shape(B, Hq, Hkv, L_max, d);
    if (st != FD_OK) return st;
    if (B > 0 && (!page_table || !seq_lens)) return FD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(page_table) & 3u) return FD_ERR_INVALID_ARG;
    fd::DecodeArgs a = {};
    a.unified = unified ? 1 : 0;
    a.phi = phi;
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.L_max = L_max;
    a.D = d;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    return decode_common(a, num_splits, true, out_dtype, workspace, workspace_bytes, stream, cache);
}

// ---------------------------------------------------------------------------
// Attention of packed query rows (prompts, prompt tails) and the decode of a
// batch with a shared prefix.

// Chunks of the keys.
struct RowsPlan {
    int splits, chunk;
};

// `splits` chunks of max_k keys, whole 128-key blocks each.
RowsPlan rows_chunks(int max_k, long long splits, bool exact) {
    long long chunk = (max_k + splits - 1) / splits;
    chunk = (chunk + 127) / 128 * 128;
    if (chunk < 128) chunk = 128;
    RowsPlan pl;
    pl.chunk = (int)chunk;
    pl.splits = exact ? (int)splits : (int)((max_k + chunk - 1) / chunk);
    if (pl.splits < 1) pl.splits = 1;
    return pl;
}

// The shared part of a shared-prefix decode: `ctas` pieces of work per chunk,
// all alike, one per SM at a time; with `own` further pieces of about own_blocks
// blocks beside them.  A piece of c blocks takes about c + `piece` blocks of time
// (set-up, first copies, last output: 4 for a single tile, 14 for two tiles, whose
// records all SMs write at the same time; 128 sequences of 64 query heads behind 32K
// tokens: 146 us in 4 chunks, 154 us in 9; 64 behind 128K: 202 us in 9, 211 us in 19),
// every chunk costs merge work, so: the count with the least of that, the longest
// SM's share or the mean.  Own pieces are short, and with nothing but them running
// the copies do not fill HBM: where the SMs that the chunks leave free get through
// them in a chunk's time, that counts a tenth less (32 sequences behind 128K tokens:
// 13 chunks 107 us, 16 to 19 chunks 118 to 120 us).
RowsPlan shared_rows_plan(long long ctas, int max_k, int requested, double piece, long long own, double own_blocks) {
    if (requested > 0) return rows_chunks(max_k, requested, true);
    const int sms = current_sm_count(), blocks = (max_k + 127) / 128;
    long long best_s = 1;
    if (sms > 0 && ctas > 0) {
        double best = 1e300;
        for (long long S = 1; S <= blocks && (S == 1 || ctas * S <= 8LL * sms); ++S) {
            const long long c = (blocks + S - 1) / S;
            if ((blocks + c - 1) / c != S) continue;  // the chunks of a smaller count
            const double waves = (double)((ctas * S + sms - 1) / sms);
            const double shared = (double)c + piece, own_time = (double)own * (own_blocks + piece);
            const double mean = ((double)(ctas * S) * shared + own_time) / sms;
            const bool beside = own_time <= (double)(sms - ctas * S) * shared;
            const double busy = std::max(waves * shared, mean);
            const double cost = (own > 0 && !beside ? 1.1 * busy : busy) + (double)S / 8.0;
            if (cost < best) {
                best = cost;
                best_s = S;
            }
        }
    }
    return rows_chunks(max_k, best_s, false);
}

int check_rows(int B, int total_q, int Hq, int Hkv, int max_k, int d, int num_splits) {
    const int st = check_shape(B, Hq, Hkv, max_k, d);
    if (st != FD_OK) return st;
    if (total_q < 0 || total_q > (1 << 30) || num_splits < 0 || num_splits > 65535) return FD_ERR_INVALID_ARG;
    // grid x and the row indices of the tile copies are 32-bit
    const long long ctas = fd::rows_tiles(B, total_q, Hq / Hkv, -1, true) * Hkv;
    if (ctas * (num_splits > 0 ? num_splits : 1) > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    return FD_OK;
}

// Prompts: the kernel cuts what each tile attends into `splits` equal parts of at
// least `chunk` keys (the lengths are on the device).  One part while the tiles
// fill the SMs twice, else the count with the least of
//   E  every sequence max_k keys long: rounds of the SMs times a piece (c blocks
//      take about c + 6 blocks of time)
//   R  (more than one sequence) lengths from a quarter of max_k up: the work shared
//      out evenly and half of the longest piece behind it
// plus the records' way to memory and back and the merge.  max_k may be no more
// than the room of a table, so that 32K keys stand for all beyond.  With 32 query
// and 8 KV heads of 128: 2048 tokens alone 33 us in one part, 76 us in two; 512
// tokens behind 8192 cached ones 95 us in one, 64 us in two, 82 us in three; 2 x 64
// behind 32K 339 us in one, 65 us in nine, 78 us in sixteen; 16 x 8 behind 16K to 64K
// (64 query heads) 458 us in one, 344 us in three, 332 us in seven, 346 us in sixteen.
// per: query tokens of a piece of work.  maps: a differential call, whose records are twice as long and
// whose results leave the kernel without them otherwise (49K rows of short prompts 19 us in one part, 85 in
// two, 95 in three), so that a row costs something in itself; its pieces are single tiles, so that parts pay up
// to three rounds of the SMs: 40 x 8 tokens behind 1K to 32K 473 us in one part, 437 in four; 48 x 8 588 and 544
// (three); 40 x 16 behind 16K 487 and 462 (two); but 20 x 64 behind 1K to 16K 214 us in one, 246 in two.
RowsPlan pieces_plan(int B, int total_q, int Hq, int Hkv, int max_k, int num_splits, int per, bool maps) {
    RowsPlan pl;
    pl.splits = num_splits > 0 ? num_splits : 1;
    pl.chunk = num_splits > 0 ? 128 : 512;
    const int sms = num_splits > 0 ? 0 : current_sm_count();
    const long long mean = B > 0 ? (total_q + B - 1) / B : 0;  // tokens of a sequence
    const long long ctas = (long long)B * ((mean + per - 1) / per) * Hkv;
    if (sms <= 0 || ctas <= 0 || ctas >= (maps ? 3LL : 2LL) * sms) return pl;
    const double kPiece = 6.0, kMerge = 4.0;  // in blocks of time
    const double kRow = maps ? 7e-4 : 0.0, kRecords = maps ? 2.5e-4 : 1.6e-4;
    const double blocks = std::min(max_k, 1 << 15) / 128.0;
    const long long most = std::min((long long)max_k / pl.chunk, 8LL * sms / ctas + 1);
    double best = 1e300;
    for (long long S = 1; S == 1 || S <= most; ++S) {
        const double c = std::max(blocks / (double)S, 1.0), pieces = (double)(ctas * S);
        double cost = std::ceil(pieces / sms) * (c + kPiece);
        if (B > 1) {
            const double mean_piece = 0.625 * c + kPiece, longest = c + kPiece;
            cost = 0.5 * (cost + std::max(pieces * mean_piece / sms + 0.5 * longest, longest));
        }
        if (S > 1) cost += kMerge + (kRow + kRecords * (double)S) * (double)total_q * Hq;
        if (cost < best) {
            best = cost;
            pl.splits = (int)S;
        }
    }
    return pl;
}

RowsPlan prefill_plan(int B, int total_q, int Hq, int Hkv, int max_k, int num_splits) {
    return pieces_plan(B, total_q, Hq, Hkv, max_k, num_splits, fd::rows_tokens(B, total_q, Hq / Hkv, -1), false);
}

// The plan of a packed call, whose sequences share total_k: no more parts than a
// sequence of 1.6 times the mean fills (the longest one, if lengths run from a quarter of
// it up; 6 prompts of 256 tokens, 4 query heads: 9.4 us in the one part that this gives,
// 15.6 us in three).  The queries (fd_prefill_num_splits and the workspace size) are not
// told that a call is packed, so it never takes more parts than they say.
RowsPlan packed_plan(int B, int total_q, int Hq, int Hkv, int total_k, int num_splits) {
    RowsPlan pl = prefill_plan(B, total_q, Hq, Hkv, total_k, num_splits);
    if (pl.splits > 1 && num_splits == 0)
        pl.splits = std::min(pl.splits, std::max(1, (int)(1.6 * total_k / B) / pl.chunk));
    return pl;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A token stride covers the token's heads and keeps 16-byte rows.
bool stride_ok(long long s, int H, int d) { return s >= (long long)H * d && s % 8 == 0 && s <= (1LL << 32); }

// T rows of `bytes` bytes, `step` bytes apart.
struct Strided {
    const void* at;
    long long T, bytes, step;
};
bool overlap(const Strided& a, const Strided& b) {
    if (!a.at || !b.at || a.T <= 0 || b.T <= 0 || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    if (x >= y + (uintptr_t)((b.T - 1) * b.step + b.bytes) || y >= x + (uintptr_t)((a.T - 1) * a.step + a.bytes))
        return false;
    if (a.step != b.step) return true;
    // slices of the same rows (a fused projection): apart where their columns are
    const long long d = (long long)(y - x) % a.step, shift = d < 0 ? d + a.step : d;
    return !(a.bytes <= shift && shift + b.bytes <= a.step);
}

// The bytes [lo, hi) of a buffer.
struct Span {
    uintptr_t lo, hi;
};
Span span(const void* at, long long bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(at);
    return {x, at && bytes > 0 ? x + (uintptr_t)bytes : x};
}
bool meet(const Span& a, const Span& b) { return std::max(a.lo, b.lo) < std::min(a.hi, b.hi); }

// Whether a buffer that a call writes shares memory with another one, or with one that it reads.
template <size_t W, size_t R>
bool clash(const Span (&written)[W], const Span (&read)[R]) {
    bool any = false;
    for (size_t w = 0; w < W; ++w) {
        for (size_t o = w + 1; o < W; ++o) any |= meet(written[w], written[o]);
        for (size_t r = 0; r < R; ++r) any |= meet(written[w], read[r]);
    }
    return any;
}

int check_prefill(const fd::RowsArgs& a, int num_splits, int out_dtype) {
    const int st = check_rows(a.B, a.total_q, a.Hq, a.Hkv, a.max_k, a.D, num_splits);
    if (st != FD_OK) return st;
    if (out_dtype != FD_OUT_F32 && out_dtype != FD_OUT_BF16) return FD_ERR_INVALID_ARG;
    if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return FD_ERR_INVALID_ARG;
    if (!stride_ok(a.q_stride, a.Hq, a.D)) return FD_ERR_INVALID_ARG;
    const bool some = a.B > 0 && a.total_q > 0;
    if (some && (!a.q || !a.out || !a.cu_q)) return FD_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.out)) return FD_ERR_INVALID_ARG;
    if (!aligned4(a.lse) || !aligned4(a.cu_q) || !aligned4(a.cu_k) || !aligned4(a.seq_lens) ||
        !aligned4(a.page_table))
        return FD_ERR_INVALID_ARG;
    return FD_OK;
}

// A differential call: a piece of work has one tile, and either map its own records.
RowsPlan prefill_diff_plan(int B, int total_q, int Hq, int Hkv, int max_k, int num_splits, bool packed) {
    RowsPlan pl = pieces_plan(B, total_q, Hq, Hkv, max_k, num_splits, fd::rows_diff_tokens(Hq / Hkv), true);
    if (packed && pl.splits > 1 && num_splits == 0)  // (as packed_plan)
        pl.splits = std::min(pl.splits, std::max(1, (int)(1.6 * max_k / B) / pl.chunk));
    return pl;
}

int check_diff_rows(int B, int total_q, int Hq, int Hkv, int max_k, int d, int num_splits) {
    const int st = check_rows(B, total_q, Hq, Hkv, max_k, d, num_splits);
    if (st != FD_OK) return st;
    const long long ctas = fd::rows_diff_tiles(B, total_q, Hq / Hkv) * Hkv;
    return ctas * (num_splits > 0 ? num_splits : 1) > 0x7fffffffLL ? FD_ERR_UNSUPPORTED : FD_OK;
}

int check_mix(const fd::DiffMix& m, int Hq, bool some) {
    if (some && !m.lambda) return FD_ERR_INVALID_ARG;
    if (m.lambda_stride != 0 && (m.lambda_stride < Hq || m.lambda_stride > (1LL << 32))) return FD_ERR_INVALID_ARG;
    if (!aligned4(m.lambda) || !aligned16(m.weight)) return FD_ERR_INVALID_ARG;
    if (m.weight && !(m.eps > 0.f && std::isfinite(m.eps))) return FD_ERR_INVALID_ARG;
    return FD_OK;
}

long long lambda_bytes(const fd::DiffMix& m, int tokens, int Hq) {
    return 4 * ((tokens - 1) * m.lambda_stride + Hq);
}
// Bytes of a row of query heads in out_dtype.
long long out_row_bytes(int Hq, int D, int out_dtype) { return (long long)Hq * D * (out_dtype == FD_OUT_BF16 ? 2 : 4); }

bool diff_rows_clash(const fd::RowsArgs& a, const fd::DiffMix& m, int out_dtype, const void* workspace, size_t need) {
    const auto tokens = [&](const void* at, long long T, long long stride, int H) {
        return span(at, T > 0 ? 2 * ((T - 1) * stride + (long long)H * a.D) : 0);
    };
    const long long pool = (long long)a.num_pages * a.Hkv * kTile * a.D * 2;
    const bool paged = a.page_table != nullptr;
    const Span written[] = {span(a.out, a.total_q * out_row_bytes(a.Hq, a.D, out_dtype)), span(a.lse, 8LL * a.total_q * a.Hq),
                            span(workspace, (long long)need)};
    const Span read[] = {tokens(a.q, a.total_q, a.q_stride, a.Hq), paged ? span(a.k, pool) : tokens(a.k, a.total_k, a.k_stride, a.Hkv),
                  paged ? span(a.v, pool) : tokens(a.v, a.total_k, a.v_stride, a.Hkv), span(a.cu_q, 4LL * a.B + 4),
                  span(a.cu_k, 4LL * a.B + 4), span(a.seq_lens, 4LL * a.B),
                  span(a.page_table, 4LL * a.B * a.table_stride), span(m.lambda, lambda_bytes(m, a.total_q, a.Hq)),
                  span(m.weight, 4LL * a.D)};
    return clash(written, read);
}

// mix: the two maps of differential attention, or null.
int prefill_entry(fd::RowsArgs& a, const fd::DiffMix* mix, int num_splits, int out_dtype, void* workspace,
                  size_t workspace_bytes, void* stream) {
    int st = check_prefill(a, num_splits, out_dtype);
    if (st == FD_OK && mix) st = check_diff_rows(a.B, a.total_q, a.Hq, a.Hkv, a.max_k, a.D, num_splits);
    if (st == FD_OK && mix) st = check_mix(*mix, a.Hq, a.B > 0 && a.total_q > 0);
    if (st != FD_OK) return st;
    const RowsPlan pl = mix      ? prefill_diff_plan(a.B, a.total_q, a.Hq, a.Hkv, a.max_k, num_splits, a.cu_k != nullptr)
                        : a.cu_k ? packed_plan(a.B, a.total_q, a.Hq, a.Hkv, a.total_k, num_splits)
                                 : prefill_plan(a.B, a.total_q, a.Hq, a.Hkv, a.max_k, num_splits);
    const int rows = mix ? 2 * a.Hq : a.Hq;  // of records, a token
    const size_t need = fd::decode_workspace_bytes(a.total_q, rows, a.D, pl.splits);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace)) return FD_ERR_INVALID_ARG;
        if ((long long)a.total_q * a.Hq > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;  // the merge's grid
    }
    if (a.B == 0 || a.total_q == 0) return FD_OK;
    // (a piece of work whose scores rise far reads its queries again while its first results are written)
    if (mix && diff_rows_clash(a, *mix, out_dtype, workspace, need)) return FD_ERR_INVALID_ARG;
    a.splits = pl.splits;
    a.chunk = pl.chunk;
    a.out_bf16 = out_dtype == FD_OUT_BF16;
    a.direct = pl.splits == 1;
    a.fine = !a.out_bf16;
    a.rec0 = 0;
    a.rec_stride = pl.splits;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = need ? a.part_o + (size_t)a.total_q * rows * pl.splits * a.D : nullptr;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = mix ? fd::launch_rows_diff(a, *mix, s) : fd::launch_rows(a, s);
    if (e != cudaSuccess || a.direct) return to_status(e);
    if (mix)
        return to_status(fd::launch_merge_diff(a.part_o, a.part_ml, a.cu_q, a.B, a.total_q, a.Hq, a.D, pl.splits,
                                               nullptr, 0, 0, a.out, a.out_bf16, a.lse, *mix, s));
    return to_status(fd::launch_merge_list(a.part_o, a.part_ml, a.cu_q, a.B, a.total_q, a.Hq, a.D, pl.splits, a.out,
                                           a.out_bf16, a.lse, s));
}

// The two parts of a shared-prefix decode: chunks of the shared tokens, then
// chunks of every sequence's own tokens, in one list of partials.  While the
// batch's queries of a KV head fit one tile, both are work of one launch (when it
// was built, 8 sequences behind 8K tokens: 17.5 us, 20.4 us in two; 32 behind 128K:
// 105.8 and 112.9 us); beyond that the shared part is bound by the tensor cores, where a
// piece with a few own rows would waste a tile, and the split-KV pass takes the
// own tokens (128 behind 64K: 286 us together, 250 us apart).
struct SharedPlan {
    RowsPlan shared;
    bool together;
    RowsPlan own_rows;  // together
    Plan own;           // apart
    int list;           // records per (sequence, query head)
    int own_splits() const { return together ? own_rows.splits : own.splits; }
};

SharedPlan shared_plan_uncached(int B, int Hq, int Hkv, int prefix_len, int L_own, int d, int num_splits) {
    SharedPlan s;
    s.together = fd::rows_single(1, B, Hq / Hkv, -1);
    // Own tokens in pieces of up to 16 blocks, 16 pieces at most (32 sequences, 8 KV heads,
    // up to 4096 own tokens behind 32K: 82 us, 87 us with 8 blocks, 95 us with 32), and no
    // more than eight for every SM: the kernel cuts what a sequence really holds, and where a
    // table has room for much more each piece without tokens costs about a microsecond of an
    // SM (the same with room for 256K each: 78 us, 94 us with 16 pieces; 32 sequences that do
    // hold 50K on average behind 8K: 932 us, 922 us with 16).
    const int sms = current_sm_count();
    const long long units = (long long)B * Hkv;
    const int most = sms > 0 && units > 0 ? (int)std::min(16LL, std::max(2LL, (8LL * sms + units - 1) / units)) : 16;
    const auto own_pieces = [most](int L) {
        const int blocks = (L + 127) / 128;
        return rows_chunks(L, std::max(1, std::min((blocks + 15) / 16, most)), false);
    };
    s.own_rows = own_pieces(L_own);
    // one chunk each while the sequences fill the SMs and are short (128 sequences
    // of up to 1024 own tokens, 8 KV heads: 46.5 us, 60.5 us in the decode's
    // 14-tile chunks)
    const bool short_own = (long long)B * Hkv >= current_sm_count() && L_own <= 32 * kTile;
    s.own = decode_plan(B, Hq, Hkv, L_own, d, short_own ? 1 : 0, true);
    // L_own is the room of a table, which may be many times what the sequences hold: beyond
    // 4096 the prefix is cut as if they held 1024 tokens on average (32 sequences of up to 2048
    // behind 128K, in a table for 128K more each: 1013 us when its whole room counted, since
    // the prefix then stayed in one part; 112 us, 110 us in a tight table)
    const int likely = L_own <= 4096 ? L_own : 2048, pieces = own_pieces(likely).splits;
    s.shared = shared_rows_plan(fd::rows_tiles(1, B, Hq / Hkv, -1, false) * Hkv, prefix_len, num_splits,
                                s.together ? 4.0 : 14.0, s.together && L_own > 0 ? (long long)B * Hkv * pieces : 0,
                                0.5 * ((likely + 127) / 128) / pieces);
    s.list = s.shared.splits + (L_own > 0 ? s.own_splits() : 0);
    return s;
}

// Remembered per thread for the last few argument sets, like the decode's plans.
SharedPlan shared_plan(int B, int Hq, int Hkv, int prefix_len, int L_own, int d, int num_splits) {
    struct Entry {
        int key[8];
        SharedPlan pl;
    };
    constexpr int kEntries = 8;
    thread_local Entry cache[kEntries] = {};
    thread_local int next = 0;
    const int key[8] = {B, Hq, Hkv, prefix_len, L_own, d, num_splits, current_sm_count()};
    for (const Entry& e : cache)
        if (e.pl.list > 0 && std::memcmp(e.key, key, sizeof key) == 0) return e.pl;
    Entry& e = cache[next];
    next = (next + 1) % kEntries;
    std::memcpy(e.key, key, sizeof key);
    e.pl = shared_plan_uncached(B, Hq, Hkv, prefix_len, L_own, d, num_splits);
    return e.pl;
}

int check_shared(int B, int Hq, int Hkv, int prefix_len, int L_own, int d, int num_splits) {
    if (prefix_len < 0 || prefix_len > (1 << 30) || L_own < 0 || L_own > (1 << 30)) return FD_ERR_INVALID_ARG;
    const int st = check_shape(B, Hq, Hkv, L_own, d);
    return st != FD_OK ? st : check_rows(1, B, Hq, Hkv, prefix_len, d, num_splits);
}

// r: the shared part (keys, layout); o: the decode of every sequence's own tokens.
int shared_entry(fd::RowsArgs& r, fd::DecodeArgs& o, int prefix_len, int L_own, int num_splits, int out_dtype,
                 void* workspace, size_t workspace_bytes, void* stream) {
    if (out_dtype != FD_OUT_F32 && out_dtype != FD_OUT_BF16) return FD_ERR_INVALID_ARG;
    if (!(o.scale > 0.f) || !std::isfinite(o.scale)) return FD_ERR_INVALID_ARG;
    if (o.B > 0 && (!o.q || !o.out)) return FD_ERR_INVALID_ARG;
    if (o.B > 0 && prefix_len > 0 && (!r.k || !r.v)) return FD_ERR_INVALID_ARG;
    if (o.B > 0 && L_own > 0 && (!o.k || !o.v)) return FD_ERR_INVALID_ARG;
    if (!aligned16(o.q) || !aligned16(o.k) || !aligned16(o.v) || !aligned16(o.out) || !aligned16(r.k) ||
        !aligned16(r.v))
        return FD_ERR_INVALID_ARG;
    if (!aligned4(o.lse) || !aligned4(o.seq_lens) || !aligned4(o.page_table) || !aligned4(r.page_table))
        return FD_ERR_INVALID_ARG;
    // tile copies address cache rows with 32-bit coordinates
    const long long own_rows = o.page_table ? (long long)o.num_pages * o.Hkv * kTile : (long long)o.B * o.Hkv * L_own;
    if (own_rows > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    const SharedPlan pl = shared_plan(o.B, o.Hq, o.Hkv, prefix_len, L_own, o.D, num_splits);
    const size_t need = fd::decode_workspace_bytes(o.B, o.Hq, o.D, pl.list < 2 ? 2 : pl.list);
    if (!workspace || workspace_bytes < need) return FD_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return FD_ERR_INVALID_ARG;
    if (o.B == 0) return FD_OK;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* ws = static_cast<float*>(workspace);
    float* ml = ws + (size_t)o.B * o.Hq * pl.list * o.D;
    const int out_bf16 = out_dtype == FD_OUT_BF16;
    r.q = o.q;
    r.q_stride = (long long)o.Hq * o.D;
    r.B = 1;
    r.total_q = o.B;
    r.Hq = o.Hq;
    r.Hkv = o.Hkv;
    r.D = o.D;
    r.max_k = prefix_len;
    r.total_k = prefix_len;
    r.scale = o.scale;
    r.splits = pl.shared.splits;
    r.chunk = pl.shared.chunk;
    r.part_o = ws;
    r.part_ml = ml;
    r.rec0 = 0;
    r.rec_stride = pl.list;
    r.fine = !out_bf16;
    if (L_own > 0 && pl.together) {
        r.own_k = o.k;
        r.own_v = o.v;
        r.own_lens = o.seq_lens;
        r.own_table = o.page_table;
        r.own_table_stride = o.max_pages;
        r.own_max = L_own;
        r.own_skip = o.skip_tokens;
        r.own_splits = pl.own_rows.splits;
        r.own_chunk = std::min(pl.own_rows.chunk, 16 * 128);
        r.own_rec0 = pl.shared.splits;
    }
    cudaError_t e = fd::launch_rows(r, s);
    if (e != cudaSuccess) return to_status(e);
    if (L_own > 0 && !pl.together) {
        o.splits = pl.own.splits;
        o.chunk_fixed = pl.own.chunk_fixed;
        o.out_bf16 = out_bf16;
        o.part_o = ws;
        o.part_ml = ml;
        o.list_splits = pl.list;
        o.rec0 = pl.shared.splits;
        e = fd::launch_decode(o, s);
        if (e != cudaSuccess) return to_status(e);
    }
    // without own tokens nobody else looks at the lengths
    return to_status(fd::launch_merge_list(ws, ml, nullptr, 0, o.B, o.Hq, o.D, pl.list, o.out, out_bf16, o.lse, s,
                                           L_own == 0 ? o.seq_lens : nullptr, o.L_max));
}

int packed_entry(const fd::DiffMix* mix, const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                      long long v_stride, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B,
                      int total_q, int total_k, int Hq, int Hkv, int d, float scale, int causal, int num_splits,
                      void* out, int out_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (total_k < 0) return FD_ERR_INVALID_ARG;
    const int st = check_shape(B, Hq, Hkv, total_k, d);
    if (st != FD_OK) return st;
    if (!stride_ok(k_stride, Hkv, d) || !stride_ok(v_stride, Hkv, d)) return FD_ERR_INVALID_ARG;
    if (B > 0 && total_q > 0 && (!cu_seqlens_k || (total_k > 0 && (!k || !v)))) return FD_ERR_INVALID_ARG;
    fd::RowsArgs a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k_head_stride = a.v_head_stride = d;
    a.cu_q = cu_seqlens_q;
    a.cu_k = cu_seqlens_k;
    a.B = B;
    a.total_q = total_q;
    a.total_k = total_k;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = d;
    a.max_k = total_k;
    a.scale = scale;
    a.causal = causal != 0;
    a.out = out;
    a.lse = lse;
    return prefill_entry(a, mix, num_splits, out_dtype, workspace, workspace_bytes, stream);
}

int paged_rows_entry(const fd::DiffMix* mix, const void* q, const void* k_pages, const void* v_pages, long long q_stride,
                     const int32_t* page_table, int max_pages, int num_pages, const int32_t* cu_seqlens_q,
                     const int32_t* seq_lens, int page_size, int B, int total_q, int Hq, int Hkv, int d, float scale,
                     int causal, int num_splits, void* out, int out_dtype, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    if (page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (max_pages <= 0 || num_pages < 0 || max_pages > (1 << 24)) return FD_ERR_INVALID_ARG;
    const int st = check_shape(B, Hq, Hkv, max_pages * kTile, d);
    if (st != FD_OK) return st;
    if (B > 0 && total_q > 0 && (!page_table || !seq_lens || (num_pages > 0 && (!k_pages || !v_pages))))
        return FD_ERR_INVALID_ARG;
    if ((long long)num_pages * Hkv * kTile > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    fd::RowsArgs a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.k = k_pages;
    a.v = v_pages;
    a.cu_q = cu_seqlens_q;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.table_stride = max_pages;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.B = B;
    a.total_q = total_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = d;
    a.max_k = max_pages * kTile;
    a.scale = scale;
    a.causal = causal != 0;
    a.out = out;
    a.lse = lse;
    return prefill_entry(a, mix, num_splits, out_dtype, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" {

int fd_prefill_num_splits(int B, int total_q, int Hq, int Hkv, int max_k, int d, int num_splits) {
    const int st = check_rows(B, total_q, Hq, Hkv, max_k, d, num_splits);
    if (st != FD_OK) return -st;
    return prefill_plan(B, total_q, Hq, Hkv, max_k, num_splits).splits;
}

size_t fd_prefill_workspace_size(int B, int total_q, int Hq, int Hkv, int max_k, int d, int num_splits) {
    if (check_rows(B, total_q, Hq, Hkv, max_k, d, num_splits) != FD_OK) return 0;
    return fd::decode_workspace_bytes(total_q, Hq, d, prefill_plan(B, total_q, Hq, Hkv, max_k, num_splits).splits);
}

int fd_prefill_packed(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                      long long v_stride, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B,
                      int total_q, int total_k, int Hq, int Hkv, int d, float scale, int causal, int num_splits,
                      void* out, int out_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    return packed_entry(nullptr, q, k, v, q_stride, k_stride, v_stride, cu_seqlens_q, cu_seqlens_k, B, total_q, total_k,
                        Hq, Hkv, d, scale, causal, num_splits, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

int fd_prefill_paged(const void* q, const void* k_pages, const void* v_pages, long long q_stride,
                     const int32_t* page_table, int max_pages, int num_pages, const int32_t* cu_seqlens_q,
                     const int32_t* seq_lens, int page_size, int B, int total_q, int Hq, int Hkv, int d, float scale,
                     int causal, int num_splits, void* out, int out_dtype, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    return paged_rows_entry(nullptr, q, k_pages, v_pages, q_stride, page_table, max_pages, num_pages, cu_seqlens_q,
                            seq_lens, page_size, B, total_q, Hq, Hkv, d, scale, causal, num_splits, out, out_dtype, lse,
                            workspace, workspace_bytes, stream);
}

int fd_prefill_diff_num_splits(int B, int total_q, int Hq, int Hkv, int max_k, int d, int num_splits) {
    const int st = check_diff_rows(B, total_q, Hq, Hkv, max_k, d, num_splits);
    if (st != FD_OK) return -st;
    return prefill_diff_plan(B, total_q, Hq, Hkv, max_k, num_splits, false).splits;
}

size_t fd_prefill_diff_workspace_size(int B, int total_q, int Hq, int Hkv, int max_k, int d, int num_splits) {
    if (check_diff_rows(B, total_q, Hq, Hkv, max_k, d, num_splits) != FD_OK) return 0;
    return fd::decode_workspace_bytes(total_q, 2 * Hq, d,
                                      prefill_diff_plan(B, total_q, Hq, Hkv, max_k, num_splits, false).splits);
}

int fd_prefill_packed_diff(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                           long long v_stride, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B,
                           int total_q, int total_k, int Hq, int Hkv, int d, float scale, int causal,
                           const float* lambda, long long lambda_stride, const float* norm_weight, float norm_eps,
                           int num_splits, void* out, int out_dtype, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const fd::DiffMix mix = {lambda, lambda_stride, norm_weight, norm_eps};
    return packed_entry(&mix, q, k, v, q_stride, k_stride, v_stride, cu_seqlens_q, cu_seqlens_k, B, total_q, total_k, Hq,
                        Hkv, d, scale, causal, num_splits, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

int fd_prefill_paged_diff(const void* q, const void* k_pages, const void* v_pages, long long q_stride,
                          const int32_t* page_table, int max_pages, int num_pages, const int32_t* cu_seqlens_q,
                          const int32_t* seq_lens, int page_size, int B, int total_q, int Hq, int Hkv, int d,
                          float scale, int causal, const float* lambda, long long lambda_stride,
                          const float* norm_weight, float norm_eps, int num_splits, void* out, int out_dtype,
                          float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    const fd::DiffMix mix = {lambda, lambda_stride, norm_weight, norm_eps};
    return paged_rows_entry(&mix, q, k_pages, v_pages, q_stride, page_table, max_pages, num_pages, cu_seqlens_q, seq_lens,
                            page_size, B, total_q, Hq, Hkv, d, scale, causal, num_splits, out, out_dtype, lse,
                            workspace, workspace_bytes, stream);
}

size_t fd_shared_prefix_workspace_size(int B, int Hq, int Hkv, int prefix_len, int L_own, int d, int num_splits) {
    if (check_shared(B, Hq, Hkv, prefix_len, L_own, d, num_splits) != FD_OK) return 0;
    const int list = shared_plan(B, Hq, Hkv, prefix_len, L_own, d, num_splits).list;
    return fd::decode_workspace_bytes(B, Hq, d, list < 2 ? 2 : list);
}

int fd_decode_dense_shared_prefix(const void* q, const void* k_prefix, const void* v_prefix, int prefix_len,
                                  const void* k, const void* v, const int32_t* seq_lens, int B, int Hq, int Hkv,
                                  int L_max, int d, float scale, int num_splits, void* out, int out_dtype, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_shared(B, Hq, Hkv, prefix_len, L_max, d, num_splits);
    if (st != FD_OK) return st;
    fd::RowsArgs r = {};
    fd::DecodeArgs o = {};
    r.k = k_prefix;
    r.v = v_prefix;
    r.k_stride = r.v_stride = d;
    r.k_head_stride = r.v_head_stride = (long long)prefix_len * d;
    o.q = q;
    o.k = k;
    o.v = v;
    o.seq_lens = seq_lens;
    o.B = B;
    o.Hq = Hq;
    o.Hkv = Hkv;
    o.L_max = L_max;
    o.D = d;
    o.scale = scale;
    o.out = out;
    o.lse = lse;
    return shared_entry(r, o, prefix_len, L_max, num_splits, out_dtype, workspace, workspace_bytes, stream);
}

int fd_decode_paged_shared_prefix(const void* q, const void* k_pages, const void* v_pages,
                                  const int32_t* prefix_table, int prefix_pages, const int32_t* page_table,
                                  int max_pages, int num_pages, const int32_t* seq_lens, int page_size, int B, int Hq,
                                  int Hkv, int d, float scale, int num_splits, void* out, int out_dtype, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (max_pages <= 0 || num_pages < 0 || max_pages > (1 << 24)) return FD_ERR_INVALID_ARG;
    if (prefix_pages < 0 || prefix_pages > max_pages) return FD_ERR_INVALID_ARG;
    const int prefix_len = prefix_pages * kTile, L_own = (max_pages - prefix_pages) * kTile;
    const int st = check_shared(B, Hq, Hkv, prefix_len, L_own, d, num_splits);
    if (st != FD_OK) return st;
    if (B > 0 && (!page_table || !seq_lens || (prefix_pages > 0 && !prefix_table))) return FD_ERR_INVALID_ARG;
    if ((long long)num_pages * Hkv * kTile > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    fd::RowsArgs r = {};
    fd::DecodeArgs o = {};
    r.k = k_pages;
    r.v = v_pages;
    r.page_table = prefix_table ? prefix_table : page_table;  // no shared page: never read
    r.table_stride = prefix_pages;
    r.max_pages = prefix_pages;
    r.num_pages = num_pages;
    r.row_lens = seq_lens;
    o.q = q;
    o.k = k_pages;
    o.v = v_pages;
    o.seq_lens = seq_lens;
    o.page_table = page_table + prefix_pages;
    o.max_pages = max_pages;
    o.num_pages = num_pages;
    o.B = B;
    o.Hq = Hq;
    o.Hkv = Hkv;
    o.L_max = max_pages * kTile;
    o.D = d;
    o.scale = scale;
    o.skip_tokens = prefix_len;
    o.out = out;
    o.lse = lse;
    return shared_entry(r, o, prefix_len, L_own, num_splits, out_dtype, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------------------
// Differential attention of single tokens.

}  // extern "C"

namespace {

// The columns of both maps share a pass over the cache; its chunks are those of the plain decode, by
// the bytes.
Plan diff_plan(int B, int Hq, int Hkv, int L_max, int d, int requested, bool ragged) {
    const int sms = current_sm_count();
    const int occ = requested > 0 ? 1 : fd::diff_ctas_per_sm(d, Hq / Hkv, ragged);
    return plan(B, Hkv, L_max, requested, ragged, occ, sms, saturating_ctas(d, sms), true);
}

int diff_decode_entry(fd::DecodeArgs& a, const fd::DiffMix& mix, int num_splits, int out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const bool ragged = a.seq_lens != nullptr;
    if (out_dtype != FD_OUT_F32 && out_dtype != FD_OUT_BF16) return FD_ERR_INVALID_ARG;
    if (num_splits < 0 || !(a.scale > 0.f) || !std::isfinite(a.scale)) return FD_ERR_INVALID_ARG;
    if (a.B > 0 && (!a.q || !a.out)) return FD_ERR_INVALID_ARG;
    const long long cache_rows = a.page_table ? (long long)a.num_pages * a.Hkv * kTile
                                              : (long long)a.B * a.Hkv * a.L_max;
    if (cache_rows > 0 && (!a.k || !a.v)) return FD_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.out)) return FD_ERR_INVALID_ARG;
    if (!aligned4(a.lse) || !aligned4(a.seq_lens) || !aligned4(a.page_table)) return FD_ERR_INVALID_ARG;
    const int st = check_mix(mix, a.Hq, a.B > 0);
    if (st != FD_OK) return st;
    if (cache_rows > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;  // 32-bit row coordinates
    const Plan pl = diff_plan(a.B, a.Hq, a.Hkv, a.L_max, a.D, num_splits, ragged);
    const size_t need = fd::decode_workspace_bytes(a.B, 2 * a.Hq, a.D, pl.splits);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace)) return FD_ERR_INVALID_ARG;
        if ((long long)a.B * a.Hq > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;  // the merge's grid
    }
    // (in place over the queries is fine: a group's rows are read before they are written, by the same CTA or in
    // the merge)
    const bool in_place = a.out == a.q && out_dtype == FD_OUT_BF16;
    const Span written[] = {span(a.out, a.B * out_row_bytes(a.Hq, a.D, out_dtype)), span(a.lse, 8LL * a.B * a.Hq),
                            span(workspace, (long long)need)};
    const Span read[] = {span(in_place ? nullptr : a.q, 2LL * a.B * a.Hq * a.D), span(a.k, 2 * cache_rows * a.D),
                         span(a.v, 2 * cache_rows * a.D), span(a.seq_lens, 4LL * a.B),
                         span(a.page_table, 4LL * a.B * a.max_pages),
                         span(mix.lambda, a.B > 0 ? lambda_bytes(mix, a.B, a.Hq) : 0),
                         span(mix.weight, a.B > 0 ? 4LL * a.D : 0)};
    if (clash(written, read)) return FD_ERR_INVALID_ARG;
    a.splits = pl.splits;
    a.chunk_fixed = pl.chunk_fixed;
    a.out_bf16 = out_dtype == FD_OUT_BF16;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = need ? a.part_o + (size_t)a.B * 2 * a.Hq * pl.splits * a.D : nullptr;
    return to_status(fd::launch_decode_diff(a, mix, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fd_num_splits_diff(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    const int st = check_shape(B, Hq, Hkv, L_max, d);
    if (st != FD_OK) return -st;
    if (num_splits < 0) return -FD_ERR_INVALID_ARG;
    return diff_plan(B, Hq, Hkv, L_max, d, num_splits, ragged != 0).splits;
}

size_t fd_decode_diff_workspace_size(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    if (check_shape(B, Hq, Hkv, L_max, d) != FD_OK || num_splits < 0) return 0;
    return fd::decode_workspace_bytes(B, 2 * Hq, d, diff_plan(B, Hq, Hkv, L_max, d, num_splits, ragged != 0).splits);
}

int fd_decode_dense_diff(const void* q, const void* k, const void* v, const int32_t* seq_lens, int B, int Hq, int Hkv,
                         int L_max, int d, float scale, const float* lambda, long long lambda_stride,
                         const float* norm_weight, float norm_eps, int num_splits, void* out, int out_dtype, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_shape(B, Hq, Hkv, L_max, d);
    if (st != FD_OK) return st;
    fd::DecodeArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.seq_lens = seq_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.L_max = L_max;
    a.D = d;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    return diff_decode_entry(a, {lambda, lambda_stride, norm_weight, norm_eps}, num_splits, out_dtype, workspace,
                             workspace_bytes, stream);
}

int fd_decode_paged_diff(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                         int max_pages, int num_pages, const int32_t* seq_lens, int page_size, int B, int Hq, int Hkv,
                         int d, float scale, const float* lambda, long long lambda_stride, const float* norm_weight,
                         float norm_eps, int num_splits, void* out, int out_dtype, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (max_pages <= 0 || num_pages < 0 || max_pages > (1 << 24)) return FD_ERR_INVALID_ARG;
    const int st = check_shape(B, Hq, Hkv, max_pages * kTile, d);
    if (st != FD_OK) return st;
    if (B > 0 && (!page_table || !seq_lens)) return FD_ERR_INVALID_ARG;
    fd::DecodeArgs a = {};
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.L_max = max_pages * kTile;
    a.D = d;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    return diff_decode_entry(a, {lambda, lambda_stride, norm_weight, norm_eps}, num_splits, out_dtype, workspace,
                             workspace_bytes, stream);
}

// ---------------------------------------------------------------------------
// Page assignment and cache append.

int fd_assign_pages(const int32_t* cached_lens, const int32_t* new_lens, int B, int32_t* page_table, int max_pages,
                    int page_size, const int32_t* free_pages, int num_free, const int32_t* free_head, int total_new,
                    int32_t* seq_lens, int32_t* cu_seqlens, int64_t* slots, int32_t* free_head_out, void* stream) {
    if (page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (B < 0 || max_pages <= 0 || max_pages > (1 << 24) || num_free < 0 || total_new < 0) return FD_ERR_INVALID_ARG;
    if (B > 0 && (!cached_lens || !new_lens || !page_table || !seq_lens)) return FD_ERR_INVALID_ARG;
    if (!cu_seqlens || !free_head_out || (num_free > 0 && !free_pages) || (total_new > 0 && !slots))
        return FD_ERR_INVALID_ARG;
    if (!aligned4(cached_lens) || !aligned4(new_lens) || !aligned4(page_table) || !aligned4(free_pages) ||
        !aligned4(free_head) || !aligned4(seq_lens) || !aligned4(cu_seqlens) || !aligned16(slots) ||
        !aligned4(free_head_out))
        return FD_ERR_INVALID_ARG;
    // the CTAs read the inputs while others already write: an output may share memory with nothing else,
    // except the new lengths in place of the old ones and the head in place of the head
    const struct {
        const void* at;
        unsigned long long bytes;
    } buffers[] = {{page_table, 4ULL * B * max_pages}, {seq_lens, 4ULL * B}, {cu_seqlens, 4ULL * B + 4},
                   {slots, 8ULL * total_new}, {free_head_out, 4},  // the outputs, then the inputs
                   {cached_lens, 4ULL * B}, {new_lens, 4ULL * B}, {free_pages, 4ULL * num_free},
                   {free_head, free_head ? 4ULL : 0ULL}};
    for (int o = 0; o < 5; ++o) {
        for (int i = o + 1; i < 9; ++i) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(buffers[o].at), b = reinterpret_cast<uintptr_t>(buffers[i].at);
            const bool in_place = a == b && ((o == 1 && i == 5) || (o == 4 && i == 8));
            if (!in_place && a < b + buffers[i].bytes && b < a + buffers[o].bytes && buffers[i].bytes > 0 &&
                buffers[o].bytes > 0)
                return FD_ERR_INVALID_ARG;
        }
    }
    fd::AssignArgs a = {cached_lens, new_lens, B, page_table, max_pages, free_pages, num_free, free_head, total_new,
                        seq_lens, cu_seqlens, slots, free_head_out};
    return to_status(fd::launch_assign(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

int append_entry(fd::AppendArgs& a, int page_size, bool fp8, void* stream) {
    if (page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (a.T < 0 || a.num_pages < 0) return FD_ERR_INVALID_ARG;
    if (a.Hkv > 0 && (long long)a.T * a.Hkv > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    const int st = check_shape(0, a.Hkv, a.Hkv, 0, a.D);
    if (st != FD_OK) return st;
    if (!stride_ok(a.k_stride, a.Hkv, a.D) || !stride_ok(a.v_stride, a.Hkv, a.D)) return FD_ERR_INVALID_ARG;
    if (a.T > 0 && (!a.k || !a.v || !a.slots)) return FD_ERR_INVALID_ARG;
    if (a.T > 0 && a.num_pages > 0 && (!a.k_pages || !a.v_pages || (fp8 && (!a.k_scales || !a.v_scales))))
        return FD_ERR_INVALID_ARG;
    if (!aligned16(a.k) || !aligned16(a.v) || !aligned16(a.k_pages) || !aligned16(a.v_pages) ||
        !aligned4(a.k_scales) || !aligned4(a.v_scales) || (reinterpret_cast<uintptr_t>(a.slots) & 7u))
        return FD_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return to_status(fp8 ? fd::launch_append_fp8(a, s) : fd::launch_append(a, s));
}

}  // namespace

extern "C" {

int fd_append_kv_paged(const void* k, const void* v, long long k_stride, long long v_stride, const int64_t* slots,
                       int T, int Hkv, int d, void* k_pages, void* v_pages, int num_pages, int page_size,
                       void* stream) {
    fd::AppendArgs a = {k, v, k_stride, v_stride, slots, T, Hkv, d, num_pages, k_pages, v_pages, nullptr, nullptr};
    return append_entry(a, page_size, false, stream);
}

int fd_append_kv_paged_fp8(const void* k, const void* v, long long k_stride, long long v_stride,
                           const int64_t* slots, int T, int Hkv, int d, uint8_t* k_pages, float* k_page_scales,
                           uint8_t* v_pages, float* v_page_scales, int num_pages, int page_size, void* stream) {
    fd::AppendArgs a = {k, v, k_stride, v_stride, slots, T, Hkv, d, num_pages, k_pages, v_pages, k_page_scales,
                        v_page_scales};
    return append_entry(a, page_size, true, stream);
}

}  // extern "C"

namespace {

// The arguments that norms and rotation share.  a: the tensors; paged: keys and values go to the cache.
int rope_entry(fd::RopeArgs& a, const fd_rope* r, bool paged, bool fp8, int page_size, void* stream) {
    if (paged && page_size != kTile) return page_size > 0 ? FD_ERR_UNSUPPORTED : FD_ERR_INVALID_ARG;
    if (!r || a.T < 0 || a.Hq < 0 || a.Hkv < 0 || a.Hq > 65535 || a.Hkv > 65535 || a.num_pages < 0)
        return FD_ERR_INVALID_ARG;
    if (a.Hq + a.Hkv == 0 || (paged && a.Hkv == 0)) return FD_ERR_INVALID_ARG;
    if (a.D != 64 && a.D != 128) return FD_ERR_UNSUPPORTED;
    const int dh = r->halves ? a.D / 2 : a.D;
    if (r->rot <= 0 || r->rot > dh || r->max_pos <= 0 || r->B < 0) return FD_ERR_INVALID_ARG;
    if (r->rot % 16 != 0) return FD_ERR_UNSUPPORTED;
    if ((long long)a.T * std::max(a.Hq, a.Hkv) > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;
    const bool q = a.Hq > 0, k = a.Hkv > 0, some = a.T > 0;
    if ((q && (!stride_ok(a.q_stride, a.Hq, a.D) || !stride_ok(a.q_out_stride, a.Hq, a.D))) ||
        (k && !stride_ok(a.k_stride, a.Hkv, a.D)) || (k && paged && !stride_ok(a.v_stride, a.Hkv, a.D)) ||
        (k && !paged && !stride_ok(a.k_out_stride, a.Hkv, a.D)))
        return FD_ERR_INVALID_ARG;
    if (some && ((q && (!a.q || !a.q_out)) || (k && !a.k) || (k && !paged && !a.k_out) || (paged && (!a.v || !a.slots))))
        return FD_ERR_INVALID_ARG;
    if (some && paged && a.num_pages > 0 && (!a.k_pages || !a.v_pages || (fp8 && (!a.k_scales || !a.v_scales))))
        return FD_ERR_INVALID_ARG;
    if (some && (!r->cos_sin || (!r->positions && (!r->cu_seqlens || (r->B > 0 && !r->seq_lens)))))
        return FD_ERR_INVALID_ARG;
    if ((r->q_weight || r->k_weight) && !(r->norm_eps > 0.f && std::isfinite(r->norm_eps))) return FD_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.q_out) || !aligned16(a.k_out) ||
        !aligned16(a.k_pages) || !aligned16(a.v_pages) || !aligned16(r->cos_sin) || !aligned16(r->q_weight) ||
        !aligned16(r->k_weight) || !aligned4(r->positions) || !aligned4(r->cu_seqlens) || !aligned4(r->seq_lens) ||
        !aligned4(a.k_scales) || !aligned4(a.v_scales) || (reinterpret_cast<uintptr_t>(a.slots) & 7u))
        return FD_ERR_INVALID_ARG;
    // rows, pools and scales that are written share no memory with anything but, in place, the very rows that they
    // replace
    const auto rows = [&](const void* at, int H, long long stride) {
        return Strided{at, a.T, 2LL * H * a.D, 2 * stride};
    };
    const Strided qo = rows(a.q_out, a.Hq, a.q_out_stride), ko = rows(a.k_out, a.Hkv, a.k_out_stride);
    const Strided qi = rows(a.q, a.Hq, a.q_stride), ki = rows(a.k, a.Hkv, a.k_stride), vi = rows(a.v, a.Hkv, a.v_stride);
    const auto same = [](const Strided& x, const Strided& y) {
        return x.at == y.at && (x.step == y.step || x.T == 1) && x.bytes == y.bytes;
    };
    if (q && ((overlap(qo, qi) && !same(qo, qi)) || overlap(qo, ki) || overlap(qo, vi) || overlap(qo, ko)))
        return FD_ERR_INVALID_ARG;
    if (k && !paged && ((overlap(ko, ki) && !same(ko, ki)) || overlap(ko, qi))) return FD_ERR_INVALID_ARG;
    const auto extent = [](const Strided& x) { return span(x.at, x.T > 0 && x.bytes > 0 ? (x.T - 1) * x.step + x.bytes : 0); };
    const long long slot_rows = some ? (long long)a.num_pages * a.Hkv * kTile : 0, pool = slot_rows * a.D * (fp8 ? 1 : 2);
    const Span written[] = {span(a.k_pages, pool), span(a.v_pages, pool), span(a.k_scales, 4 * slot_rows),
                            span(a.v_scales, 4 * slot_rows), extent(qo)};
    const Span read[] = {span(r->cos_sin, 4LL * r->max_pos * r->rot), span(r->q_weight, 4LL * dh),
                         span(r->k_weight, 4LL * dh), span(r->positions, 4LL * a.T), span(r->cu_seqlens, 4LL * r->B + 4),
                         span(r->seq_lens, 4LL * r->B), span(a.slots, 8LL * a.T)};
    const Span keys_out[] = {extent(ko)}, rows_in[] = {extent(qi), extent(ki), extent(vi)};
    if (clash(written, read) || clash(keys_out, read)) return FD_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
        for (const Span& in : rows_in)
            if (meet(written[i], in)) return FD_ERR_INVALID_ARG;
    a.cos_sin = r->cos_sin;
    a.max_pos = r->max_pos;
    a.rot = r->rot;
    a.interleaved = r->interleaved != 0;
    a.halves = r->halves != 0;
    a.positions = r->positions;
    a.cu = r->cu_seqlens;
    a.lens = r->seq_lens;
    a.B = r->B;
    a.q_weight = r->q_weight;
    a.k_weight = r->k_weight;
    a.eps = r->norm_eps;
    return to_status(fd::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

const uint16_t* bits16(const void* p) { return static_cast<const uint16_t*>(p); }

int append_rope(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                long long v_stride, const int64_t* slots, int T, int Hq, int Hkv, int d, const fd_rope* rope,
                void* q_out, long long q_out_stride, void* k_pages, float* k_scales, void* v_pages, float* v_scales,
                int num_pages, int page_size, bool fp8, void* stream) {
    fd::RopeArgs a = {};
    a.q = bits16(q);
    a.k = bits16(k);
    a.v = bits16(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slots;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = d;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q_out_stride = q_out_stride;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.num_pages = num_pages;
    return rope_entry(a, rope, true, fp8, page_size, stream);
}

}  // namespace

extern "C" {

int fd_norm_rope(const void* q, const void* k, long long q_stride, long long k_stride, int T, int Hq, int Hkv, int d,
                 const fd_rope* rope, void* q_out, void* k_out, long long q_out_stride, long long k_out_stride,
                 void* stream) {
    fd::RopeArgs a = {};
    a.q = bits16(q);
    a.k = bits16(k);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = d;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.k_out = static_cast<uint16_t*>(k_out);
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    return rope_entry(a, rope, false, false, kTile, stream);
}

int fd_append_kv_paged_rope(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                            long long v_stride, const int64_t* slots, int T, int Hq, int Hkv, int d,
                            const fd_rope* rope, void* q_out, long long q_out_stride, void* k_pages, void* v_pages,
                            int num_pages, int page_size, void* stream) {
    return append_rope(q, k, v, q_stride, k_stride, v_stride, slots, T, Hq, Hkv, d, rope, q_out, q_out_stride,
                           k_pages, nullptr, v_pages, nullptr, num_pages, page_size, false, stream);
}

int fd_append_kv_paged_rope_fp8(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                                long long v_stride, const int64_t* slots, int T, int Hq, int Hkv, int d,
                                const fd_rope* rope, void* q_out, long long q_out_stride, uint8_t* k_pages,
                                float* k_page_scales, uint8_t* v_pages, float* v_page_scales, int num_pages,
                                int page_size, void* stream) {
    return append_rope(q, k, v, q_stride, k_stride, v_stride, slots, T, Hq, Hkv, d, rope, q_out, q_out_stride,
                           k_pages, k_page_scales, v_pages, v_page_scales, num_pages, page_size, true, stream);
}

int fd_abi_version(void) { return FD_ABI_VERSION; }

const char* fd_status_string(int status) {
    switch (status) {
        case FD_OK: return "FD_OK";
        case FD_ERR_INVALID_ARG: return "FD_ERR_INVALID_ARG: invalid argument";
        case FD_ERR_UNSUPPORTED: return "FD_ERR_UNSUPPORTED: shape not supported (d, group size or page size)";
        case FD_ERR_WORKSPACE_TOO_SMALL: return "FD_ERR_WORKSPACE_TOO_SMALL: workspace smaller than required";
        case FD_ERR_BAD_PAGE_TABLE: return "FD_ERR_BAD_PAGE_TABLE: a page id was outside the page pool";
        case FD_ERR_CUDA: return "FD_ERR_CUDA: a CUDA call failed";
        case FD_ERR_DEVICE_TIMEOUT: return "FD_ERR_DEVICE_TIMEOUT: a kernel pipeline wait hit its time limit";
        case FD_ERR_OUT_OF_PAGES: return "FD_ERR_OUT_OF_PAGES: the list of free pages was used up";
        default: return "unknown fd_status";
    }
}

int fd_num_splits(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    return num_splits_for(Cache::BF16, B, Hq, Hkv, L_max, d, num_splits, ragged);
}

size_t fd_decode_workspace_size(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    return workspace_for(Cache::BF16, B, Hq, Hkv, L_max, d, num_splits, ragged);
}

int fd_decode_dense(const void* q, const void* k, const void* v, const int32_t* seq_lens,
                    int B, int Hq, int Hkv, int L_max, int d, float scale, int num_splits,
                    void* out, int out_dtype, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return dense_entry(Cache::BF16, q, k, v, nullptr, nullptr, seq_lens, B, Hq, Hkv, L_max, d, scale, num_splits,
                       out, out_dtype, lse, workspace, workspace_bytes, stream);
}

int fd_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                    const int32_t* page_table, int max_pages, int num_pages,
                    const int32_t* seq_lens, int page_size,
                    int B, int Hq, int Hkv, int d, float scale, int num_splits,
                    void* out, int out_dtype, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return paged_entry(Cache::BF16, q, k_pages, v_pages, nullptr, nullptr, page_table, max_pages, num_pages,
                       seq_lens, page_size, B, Hq, Hkv, d, scale, num_splits, out, out_dtype, lse, workspace,
                       workspace_bytes, stream);
}

int fd_decode_dense_unified(const void* q, const void* k, const void* v, const int32_t* seq_lens,
                            int B, int Hq, int Hkv, int L_max, int d, float scale, float phi, int num_splits,
                            void* out, int out_dtype, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
    return dense_entry(Cache::BF16, q, k, v, nullptr, nullptr, seq_lens, B, Hq, Hkv, L_max, d, scale, num_splits,
                       out, out_dtype, lse, workspace, workspace_bytes, stream, true, phi);
}

int fd_decode_paged_unified(const void* q, const void* k_pages, const void* v_pages,
                            const int32_t* page_table, int max_pages, int num_pages,
                            const int32_t* seq_lens, int page_size,
                            int B, int Hq, int Hkv, int d, float scale, float phi, int num_splits,
                            void* out, int out_dtype, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
    return paged_entry(Cache::BF16, q, k_pages, v_pages, nullptr, nullptr, page_table, max_pages, num_pages,
                       seq_lens, page_size, B, Hq, Hkv, d, scale, num_splits, out, out_dtype, lse, workspace,
                       workspace_bytes, stream, true, phi);
}

int fd_quantize_kv_fp8(const void* x, const int32_t* seq_lens, int B, int H, int L_max, int d,
                       uint8_t* codes, float* scales, void* stream) {
    const int st = check_shape(B, H, H, L_max, d);
    if (st != FD_OK) return st;
    if (B > 0 && L_max > 0 && (!x || !codes || !scales)) return FD_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return FD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(seq_lens) & 3u) return FD_ERR_INVALID_ARG;
    fd::Fp8QuantArgs a = {x, seq_lens, B, H, L_max, d, codes, scales};
    return to_status(fd::launch_quantize_fp8(a, static_cast<cudaStream_t>(stream)));
}

int fd_num_splits_fp8(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    return num_splits_for(Cache::FP8, B, Hq, Hkv, L_max, d, num_splits, ragged);
}

size_t fd_decode_fp8_workspace_size(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    return workspace_for(Cache::FP8, B, Hq, Hkv, L_max, d, num_splits, ragged);
}

int fd_decode_dense_fp8(const void* q, const uint8_t* k_codes, const float* k_scales, const uint8_t* v_codes,
                        const float* v_scales, const int32_t* seq_lens, int B, int Hq, int Hkv, int L_max, int d,
                        float scale, int num_splits, void* out, int out_dtype, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
    return dense_entry(Cache::FP8, q, k_codes, v_codes, k_scales, v_scales, seq_lens, B, Hq, Hkv, L_max, d, scale,
                       num_splits, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

int fd_decode_paged_fp8(const void* q, const uint8_t* k_pages, const float* k_page_scales, const uint8_t* v_pages,
                        const float* v_page_scales, const int32_t* page_table, int max_pages, int num_pages,
                        const int32_t* seq_lens, int page_size, int B, int Hq, int Hkv, int d, float scale,
                        int num_splits, void* out, int out_dtype, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
    return paged_entry(Cache::FP8, q, k_pages, v_pages, k_page_scales, v_page_scales, page_table, max_pages,
                       num_pages, seq_lens, page_size, B, Hq, Hkv, d, scale, num_splits, out, out_dtype, lse,
                       workspace, workspace_bytes, stream);
}

int fd_quantize_kv_fp4(const void* x, const int32_t* seq_lens, int B, int H, int L_max, int d,
                       uint8_t* codes, uint8_t* scales, void* stream) {
    const int st = check_shape(B, H, H, L_max, d);
    if (st != FD_OK) return st;
    if (B > 0 && L_max > 0 && (!x || !codes || !scales)) return FD_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return FD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(seq_lens) & 3u) return FD_ERR_INVALID_ARG;
    fd::Fp4QuantArgs a = {x, seq_lens, B, H, L_max, d, codes, scales, 0};
    return to_status(fd::launch_quantize_fp4(a, static_cast<cudaStream_t>(stream)));
}

int fd_quantize_v_fp4(const void* x, const int32_t* seq_lens, int B, int H, int L_max, int d,
                      uint8_t* codes, uint8_t* scales, void* stream) {
    const int st = check_shape(B, H, H, L_max, d);
    if (st != FD_OK) return st;
    if (B > 0 && L_max > 0 && (!x || !codes || !scales)) return FD_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return FD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(seq_lens) & 3u) return FD_ERR_INVALID_ARG;
    fd::Fp4QuantArgs a = {x, seq_lens, B, H, L_max, d, codes, scales, 1};
    return to_status(fd::launch_quantize_fp4(a, static_cast<cudaStream_t>(stream)));
}

int fd_num_splits_fp4(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    return num_splits_for(Cache::FP4, B, Hq, Hkv, L_max, d, num_splits, ragged);
}

size_t fd_decode_fp4_workspace_size(int B, int Hq, int Hkv, int L_max, int d, int num_splits, int ragged) {
    return workspace_for(Cache::FP4, B, Hq, Hkv, L_max, d, num_splits, ragged);
}

int fd_decode_dense_fp4(const void* q, const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                        const uint8_t* v_scales, const int32_t* seq_lens, int B, int Hq, int Hkv, int L_max, int d,
                        float scale, int num_splits, void* out, int out_dtype, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
    return dense_entry(Cache::FP4, q, k_codes, v_codes, k_scales, v_scales, seq_lens, B, Hq, Hkv, L_max, d, scale,
                       num_splits, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

int fd_decode_paged_fp4(const void* q, const uint8_t* k_pages, const uint8_t* k_page_scales, const uint8_t* v_pages,
                        const uint8_t* v_page_scales, const int32_t* page_table, int max_pages, int num_pages,
                        const int32_t* seq_lens, int page_size, int B, int Hq, int Hkv, int d, float scale,
                        int num_splits, void* out, int out_dtype, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
    return paged_entry(Cache::FP4, q, k_pages, v_pages, k_page_scales, v_page_scales, page_table, max_pages,
                       num_pages, seq_lens, page_size, B, Hq, Hkv, d, scale, num_splits, out, out_dtype, lse,
                       workspace, workspace_bytes, stream);
}

int fd_quantize_keys(const void* k, const int32_t* seq_lens, int B, int Hkv, int L_max, int d,
                     uint8_t* codes, void* mn_scale, int8_t* res, void* res_scale, void* stream) {
    const int st = check_shape(B, Hkv, Hkv, L_max, d);
    if (st != FD_OK) return st;
    if (B > 0 && L_max > 0 && (!k || !codes || !mn_scale || !res || !res_scale)) return FD_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(codes) || !aligned16(mn_scale) || !aligned16(res) || !aligned16(res_scale))
        return FD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(seq_lens) & 3u) return FD_ERR_INVALID_ARG;
    fd::QuantArgs a = {k, seq_lens, B, Hkv, L_max, d, codes, mn_scale, res, res_scale};
    return to_status(fd::launch_quantize(a, static_cast<cudaStream_t>(stream)));
}

size_t fd_topdelta_workspace_size(int B, int Hq, int Hkv, int L_max, int d, int num_splits) {
    if (check_shape(B, Hq, Hkv, L_max, d) != FD_OK || num_splits < 0) return 0;
    const Plan pl = topdelta_plan(B, Hq, Hkv, L_max, d, num_splits);
    return fd::decode_workspace_bytes(B, Hq, d, pl.splits);
}

}  // extern "C"

namespace {

int topdelta_entry(const void* q, const uint8_t* codes, const void* mn_scale, const int8_t* res,
                   const void* res_scale, const void* v, const int32_t* seq_lens,
                   int B, int Hq, int Hkv, int L_max, int d, float scale, float delta,
                   int n_sink, int window, int num_splits,
                   void* out, int out_dtype, float* lse, uint32_t* sel_mask, int32_t* sel_count,
                   void* workspace, size_t workspace_bytes, void* stream, bool group_union) {
    const int st = check_shape(B, Hq, Hkv, L_max, d);
    if (st != FD_OK) return st;
    if (out_dtype != FD_OUT_F32 && out_dtype != FD_OUT_BF16) return FD_ERR_INVALID_ARG;
    if (num_splits < 0 || !std::isfinite(scale) || std::isnan(delta) || delta < 0.f) return FD_ERR_INVALID_ARG;
    if (n_sink < 0 || window < 0) return FD_ERR_INVALID_ARG;
    if (L_max % 4 != 0) return FD_ERR_UNSUPPORTED;  // keeps every tile copy 16-byte aligned
    if ((long long)B * Hkv * L_max > 0x7fffffffLL) return FD_ERR_UNSUPPORTED;  // 32-bit row coordinates
    if (B > 0 && (!q || !codes || !mn_scale || !res || !res_scale || !v || !out)) return FD_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(codes) || !aligned16(mn_scale) || !aligned16(res) || !aligned16(res_scale) ||
        !aligned16(v) || !aligned16(out))
        return FD_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(sel_mask) & 3u) || (reinterpret_cast<uintptr_t>(sel_count) & 3u))
        return FD_ERR_INVALID_ARG;
    const Plan pl = topdelta_plan(B, Hq, Hkv, L_max, d, num_splits);
    const size_t need = fd::decode_workspace_bytes(B, Hq, d, pl.splits);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace)) return FD_ERR_INVALID_ARG;
    }
    fd::TopDeltaArgs a = {};
    a.q = q;
    a.codes = codes;
    a.mn_scale = mn_scale;
    a.res = res;
    a.res_scale = res_scale;
    a.v = v;
    a.seq_lens = seq_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.L_max = L_max;
    a.D = d;
    a.scale = scale;
    a.delta = delta;
    a.n_sink = n_sink;
    a.window = window;
    a.splits = pl.splits;
    a.chunk_fixed = pl.chunk_fixed;
    a.group_union = group_union ? 1 : 0;
    a.out = out;
    a.out_bf16 = out_dtype == FD_OUT_BF16;
    a.lse = lse;
    a.sel_mask = sel_mask;
    a.sel_count = sel_count;
    float* ws = static_cast<float*>(workspace);
    a.part_o = ws;
    a.part_ml = ws ? ws + (size_t)B * Hq * pl.splits * d : nullptr;
    return to_status(fd::launch_topdelta(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fd_decode_topdelta(const void* q, const uint8_t* codes, const void* mn_scale, const int8_t* res,
                       const void* res_scale, const void* v, const int32_t* seq_lens,
                       int B, int Hq, int Hkv, int L_max, int d, float scale, float delta,
                       int n_sink, int window, int num_splits,
                       void* out, int out_dtype, float* lse, uint32_t* sel_mask, int32_t* sel_count,
                       void* workspace, size_t workspace_bytes, void* stream) {
    return topdelta_entry(q, codes, mn_scale, res, res_scale, v, seq_lens, B, Hq, Hkv, L_max, d, scale, delta,
                          n_sink, window, num_splits, out, out_dtype, lse, sel_mask, sel_count, workspace,
                          workspace_bytes, stream, false);
}

int fd_decode_topdelta_group_union(const void* q, const uint8_t* codes, const void* mn_scale, const int8_t* res,
                                   const void* res_scale, const void* v, const int32_t* seq_lens,
                                   int B, int Hq, int Hkv, int L_max, int d, float scale, float delta,
                                   int n_sink, int window, int num_splits,
                                   void* out, int out_dtype, float* lse, uint32_t* sel_mask, int32_t* sel_count,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    return topdelta_entry(q, codes, mn_scale, res, res_scale, v, seq_lens, B, Hq, Hkv, L_max, d, scale, delta,
                          n_sink, window, num_splits, out, out_dtype, lse, sel_mask, sel_count, workspace,
                          workspace_bytes, stream, true);
}

int fd_debug_inject_wait_timeout(unsigned long long wait_limit_ns, int withhold_tile) {
    fd::inject_wait_timeout(wait_limit_ns, withhold_tile);
    return FD_OK;
}

int fd_device_status(int clear, void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FD_ERR_CUDA;
    unsigned a = 0, b = 0, c = 0, e = 0, r = 0, m = 0, g = 0, x = 0, y = 0, z = 0;
    if (fd::decode_status_read(&a, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::topdelta_status_read(&b, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::fp8_status_read(&c, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::fp4_status_read(&e, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::rows_status_read(&r, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::merge_status_read(&m, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::pages_status_read(&g, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::diff_status_read(&x, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::rows_diff_status_read(&y, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    if (fd::rope_status_read(&z, clear != 0) != cudaSuccess) return FD_ERR_CUDA;
    const unsigned bits = a | b | c | e | r | m | g | x | y | z;
    if (bits & 2u) return FD_ERR_DEVICE_TIMEOUT;
    if (bits & 1u) return FD_ERR_BAD_PAGE_TABLE;
    if (bits & 8u) return FD_ERR_OUT_OF_PAGES;
    if (bits & 4u) return FD_ERR_INVALID_ARG;
    return FD_OK;
}

}  // extern "C"
