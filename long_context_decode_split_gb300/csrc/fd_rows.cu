// fd_rows.cu -- attention of packed query rows for sm_103a: whole prompts,
// prompt tails over a paged cache, and the decode of a batch with a shared
// prefix.  A tile holds consecutive query tokens of one sequence times the G
// query heads of one KV head (row = token * G + head, 128 / G tokens), so every
// key and value read serves the whole group.
//
// For a row with the visible keys [0, n):
//   s_j = scale <q, k_j>,  out = sum_j e^(s_j) v_j / sum_j e^(s_j),
//   lse = ln sum_j e^(s_j)
// (no visible key, or none of weight: out = 0, lse = -inf) in one pass over the
// keys: m is the running maximum, l the running sum of 2^(s_j log2e - m), and O is
// rescaled when m moves.  Scores, m, l and O are binary32, and l takes the weights
// unrounded.  The product with V wants both operands of one type, so the weights
// enter it as bf16: as one term for bf16 results (2^-8 relative at most), as
// hi + lo for float32 results (2^-16).
#include <cmath>
#include <type_traits>

#include "fd_device.cuh"
#include "fd_internal.h"
#include "fd_tma.h"

namespace fd {

__device__ unsigned int g_status_rows;

namespace {

struct RowsParams {
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* seq_lens;
    const int32_t* row_lens;
    const int32_t* page_table;
    int max_pages, num_pages;
    long long table_stride;
    int B, total_q, total_k, Hq, Hkv, G, tok;
    int max_k;
    float scale_log2;
    int causal;
    int splits, chunk;
    int tiles;  // slots of every (head, chunk)
    int side_by_side;  // the tiles of a chunk follow each other, else the chunks of a tile
    unsigned long long wait_limit_ns;  // time limit of every pipeline wait
    int withhold_tile;                 // >= 0: fault injection, that block's keys of each chunk are never copied
    void* out;
    int out_bf16;
    float* lse;
    float* part_o;
    float* part_ml;
    int rec0, rec_stride, direct;
    int wide;      // results (or records) are 32-byte aligned
    int zero_row;  // a row past the page pool: a tile copied from there is zeros
    // every query token's own keys (a shared-prefix decode of a single tile)
    int shared_work;  // pieces of work before those
    const int32_t* own_lens;
    const int32_t* own_table;
    long long own_table_stride;
    int own_max, own_skip, own_splits, own_chunk, own_rec0;
};

// The tensor maps of a launch: queries, keys, values; then the same of the own keys.
struct RowsMaps {
    CUtensorMap q, k, v, own_q, own_k, own_v;
};

// One tile's place: the sequence, its query tokens and its keys.
struct RowsItem {
    int own;  // a query token with its own keys
    int seq;
    int q0, Lq;  // first query token of the sequence in the packed array, and their number
    int k0, Lk;  // the same of its keys (k0 = 0 when paged)
    int t0;      // first token of the tile within the sequence
};

__device__ __forceinline__ int checked(int c, int lo, int hi) {
    if (c < lo || c > hi) {
        if ((threadIdx.x & 31) == 0) atomicOr(&g_status_rows, kStatusBadSeqLen);
        return c < lo ? lo : hi;
    }
    return c;
}

// All lanes of a warp together.  Tile slots: sequence s owns the slots from
// floor(cu_q[s] / per) + s up to those of s + 1, at least as many as the tiles it
// has (`per` tokens each), so a slot's sequence is found by a search of cu_q
// alone.
__device__ __forceinline__ RowsItem find_item(const RowsParams& p, int slot, int per) {
    int lo = 0;
    if (p.cu_q) {
        // the last s with first_slot(s) <= slot; each round every lane probes one of 32 places
        const int lane = threadIdx.x & 31;
        int n = p.B;  // the answer is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int s = lo + lane * step;
            const bool below = lane * step < n && min(max(p.cu_q[s], 0), p.total_q) / per + s <= slot;
            const unsigned votes = __ballot_sync(0xffffffffu, below);
            const int hit = votes ? 31 - __clz(votes) : 0;
            lo += hit * step;
            n = min(step, n - hit * step);
        }
    }
    // every load first (one memory latency), then the checks
    int q0 = 0, q1 = p.total_q, k0 = 0, k1 = p.page_table ? p.max_k : p.total_k;
    if (p.cu_q) {
        q0 = p.cu_q[lo];
        q1 = p.cu_q[lo + 1];
    }
    if (p.page_table) {
        if (p.seq_lens) k1 = p.seq_lens[lo];
    } else if (p.cu_k) {
        k0 = p.cu_k[lo];
        k1 = p.cu_k[lo + 1];
    }
    RowsItem it;
    it.own = 0;
    it.seq = lo;
    it.q0 = checked(q0, 0, p.total_q);
    it.Lq = checked(q1, it.q0, p.total_q) - it.q0;
    const int most = p.page_table ? p.max_k : p.total_k;
    it.k0 = checked(k0, 0, most);
    it.Lk = checked(k1, it.k0, most) - it.k0;
    it.t0 = (slot - (it.q0 / per + it.seq)) * per;
    return it;
}

// Query token b with its own keys.
__device__ __forceinline__ RowsItem own_item(const RowsParams& p, int b) {
    RowsItem it;
    it.own = 1;
    it.seq = it.q0 = b;
    it.Lq = 1;
    it.k0 = it.t0 = 0;
    it.Lk = p.own_lens ? max(checked(p.own_lens[b], 0, p.own_skip + p.own_max) - p.own_skip, 0) : p.own_max;
    return it;
}

// Keys that query token t of the item's sequence sees.
__device__ __forceinline__ int visible_keys(const RowsParams& p, const RowsItem& it, int t) {
    int n = it.Lk;
    if (it.own) return n;
    if (p.causal) n = min(n, it.Lk - it.Lq + t + 1);
    if (p.row_lens) n = min(n, p.row_lens[it.q0 + t]);
    return max(n, 0);
}

constexpr int kRows = 128;    // rows of a tile: the lanes of an accumulator in tensor memory
constexpr int kBlock = 128;   // keys per step
constexpr int kThreads = 384; // two softmax warpgroups, then the copy warp, two MMA warps and an idle one
constexpr int kCopyWarp = 8, kMmaWarp = 9;  // (kMmaWarp + i issues pipeline i's products)
// Registers per thread after the split: 168 x 384 at launch = 216 x 256 + 72 x 128.
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;

// A running maximum is replaced only when a row exceeds it by more than this
// (log2 units): the weights then stay below 2^8, far inside binary32 and bf16
// range, and O is rescaled a few times per sequence instead of at every block.
constexpr float kRescaleAt = 8.f;

template <int D, bool DUAL>
struct RowsGeo {
    static constexpr int BOX = 128 * 128;           // 128 rows x 64 bf16 channels
    static constexpr int BOXES = D / 64;
    static constexpr int TILE = BOXES * BOX;        // 128 rows of D channels
    static constexpr int TILES = DUAL ? 2 : 1;      // of query rows
    static constexpr int STAGES = D == 128 ? (DUAL ? 5 : 6) : 8;
    // Two tiles share one ring; the pipelines of a single tile have one each.
    // (Every consumer of a ring waits for every tile of it: a barrier's parity
    // tells only two phases apart.)
    static constexpr int RING = DUAL ? STAGES : STAGES / 2;
    static constexpr int SMEM = 1024 + (TILES + STAGES) * TILE + (2 * STAGES + 18) * 8 + 16 + 2 * 64 + 16 + 2 * 128 * 4;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// ---- tensor memory and tcgen05 ------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 lanes (one row per thread); tmem_wait_ld ties the
// registers to the wait, so nothing reads them before it.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptors, 128-byte swizzle: the lower word holds the
// address and the leading byte offset in units of 16 bytes, the upper one the
// stride byte offset (1024: groups of 8 rows or tokens), version 1, layout 2.
constexpr uint32_t kDescHi = 1024u >> 4 | 1u << 14 | 2u << 29;
// Channels contiguous (Q and K): the leading offset is not used.
__device__ __forceinline__ uint32_t desc_rows(uint32_t addr) { return (addr & 0x3ffffu) >> 4 | 1u << 16; }
// Tokens as the contraction, channels contiguous (V): 64-channel boxes 128 * 128 bytes apart.
__device__ __forceinline__ uint32_t desc_cols(uint32_t addr) { return (addr & 0x3ffffu) >> 4 | (128u * 128u >> 4) << 16; }

// Instruction descriptor: bf16 x bf16 -> fp32, M = 128, N columns; bit 16: B
// with its N index contiguous.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_cols) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_cols ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | 8u << 24;
}
// One thread of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// A value that all lanes hold, in a form that the compiler knows to be uniform
// (tcgen05 operands live in uniform registers).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

// D[tmem] (+)= A[smem] B[smem]^T, 16 deep; a and b are lower descriptor words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
// The same with A in tensor memory (bf16 pairs, one 32-bit column per pair).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
// `bar` gets one arrival when every MMA this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const void* tmap, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// ---- work distribution ------------------------------------------------------------

// The next CTA of the grid that has not started yet is cancelled and its index
// written to `answer` (16 bytes, counted on `bar`): a running CTA takes its
// work over, without a counter in memory.
__device__ __forceinline__ void next_cta_request(void* answer, uint64_t* bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}
// Index of the cancelled CTA, or -1: none is left (then no further request).
__device__ __forceinline__ int next_cta(const void* answer) {
    uint32_t x, ok;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %1, 1, 0, p;\n\t"
        "mov.b32 %0, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, _}, r;\n\t}"
        : "=r"(x), "=r"(ok)
        : "r"(smem_u32(answer))
        : "memory");
    // order the read before the next answer's write
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return ok ? (int)x : -1;
}

// Named barrier whose threads all learn whether any of them passed `x`.
__device__ __forceinline__ bool named_barrier_or(int id, int nthreads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
        "bar.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(nthreads), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// A paged item's row of the page table, and how many entries of it hold its keys.
__device__ __forceinline__ const int32_t* table_of(const RowsParams& p, const RowsItem& it) {
    return it.own ? p.own_table + (size_t)it.seq * p.own_table_stride : p.page_table + (size_t)it.seq * p.table_stride;
}
__device__ __forceinline__ int pages_of(const RowsParams& p, const RowsItem& it) {
    const int n = (it.Lk + kTile - 1) / kTile;
    return it.own ? n : min(n, p.max_pages);
}

// A piece of work as the copy warp hands it to the others.
struct Work {
    int valid;  // 0: there is no more
    RowsItem it;
    int h;
    int c0, c1;  // its keys [c0, c1)
    int rec;     // its record
    int nb[2];   // blocks of keys of each pipeline
};

// 32 bytes to global memory: whole sectors from one thread.  `wide`: the
// address is 32-byte aligned (16 otherwise).
__device__ __forceinline__ void store32(void* at, const uint32_t* x, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                     "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(at)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4*>(at)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// A warp writes l = 0 to record `rec` of `tokens` query tokens times a group's
// heads.  (Unrolled, the loop's code cost long pieces 2%.)
__device__ __forceinline__ void mark_empty(float* part_ml, int token, int tokens, int G, int h, int Hq, int rec_stride,
                                        int rec) {
#pragma unroll 1
    for (int x = threadIdx.x & 31; x < tokens * G; x += 32) {
        const size_t row = (size_t)(token + x / G) * Hq + h * G + x % G;
        reinterpret_cast<float2*>(part_ml)[row * rec_stride + rec] = make_float2(-INFINITY, 0.f);
    }
}

// ---- the pass -------------------------------------------------------------------
//
// S = Q K^T and O += P V run on tcgen05 with S, P and O in tensor memory.  Two
// pipelines (i = 0, 1) alternate on the tensor cores: while the softmax
// warpgroup of one turns its S into P, the other's products run.
//   DUAL    the two pipelines hold two tiles of query rows and share every
//           block of keys and values
//   single  both hold the same tile and take the even and the odd blocks; their
//           (m, l, O) are joined at the end
// A thread of a softmax warpgroup owns one row: 128 scores in registers, no
// shuffles.  P (bf16) overwrites the first half of S; the products of a
// pipeline run in the order they are issued, so S of block j + 1 is computed
// after P of block j was read.  Tensor memory columns: S0 S1 | O0 O1.
// Keys and values pass through rings of 128-row tiles (K V K V ..).
//
// A CTA goes from one piece of work to the next without a stop: the copy warp
// is ahead with the next queries and keys, and the next piece's first products
// run while the softmax warpgroups write the last one's results.  Pieces come in
// the order of (tile, KV head): the SMs that run at the same time then read the
// same keys of a sequence from L2 (longest tiles first, across sequences: ragged
// prompts 6% slower; one head after the other: prompt tails 19% slower).
//
// What bounds it, and what each choice brought (32 query heads, 8 KV heads,
// d = 128):
//   * long prompts: the tensor cores at the power limit.  32K tokens take
//     5.2-5.3 ms in a loop (1.66-1.69 PFLOP/s of the causal products; a bf16
//     matrix product in a loop reaches 1.72) and 4.7 ms in a short run (1.88;
//     1.97).  64 cycles an MMA of the 128 x 128 x 16 shape.
//   * an MMA is taken about when it starts to run, so whatever the issuing warp
//     does in between leaves the tensor cores idle: operands that the compiler
//     knows to be uniform, 1463 -> 1651 TFLOP/s; a warp per pipeline, whose waits
//     and commits run beside the other's products, 1679 -> 1780.
//   * a block's softmax is about 1100 cycles (60 to read S, 280 maximum, 690
//     weights, 40 to store P) beside 2 x 1024 of products.  Handing P over in
//     halves, three-operand maxima, a last block cut to its keys and a warpgroup
//     of its own for the output all measured slower or the same.
//   * short prompts pay about 3 us a piece of work between its last product and the
//     next one's first: the output (1.3 us), the next work and its scores, their
//     softmax with both warpgroups at once (8 prompts of 257 to 6143 tokens, 64 query
//     heads: 0.96 ms in a short run, 1.02 ms in a loop, 1.5-1.6 PFLOP/s).  It is not the
//     copies: the next queries in L2 ahead of time, or its first keys before its
//     queries, changed nothing; nor the stores: whole lines traded between lanes took
//     longer.
//   * few query rows (drafts, a shared prefix): HBM.  16 x 8 drafted tokens of 64
//     query heads on 16K-64K cached ones 332 us, 6.4 TB/s.
//
// FINE (float32 results): weights as hi + lo, both in tensor memory over their S, and a
// second pass of the same V for lo.  8000 tokens, 32 and 8 heads: 423 us, 318 us with one
// term; 16 tokens on 16000 keys 133 and 101 us.  bf16 results take one term, whose error is
// like that of their own rounding; as hi + lo their single tiles would take 372 us
// instead of 337 (16 x 8 drafted tokens on 16K-64K) and 118 instead of 108 (shared 128K x 32).
template <int D, bool PAGED, bool DUAL, bool FINE>
__global__ void __launch_bounds__(kThreads, 1)
rows_kernel(const __grid_constant__ RowsMaps maps, const RowsParams p) {
    using Geo = RowsGeo<D, DUAL>;
    constexpr int TILES = Geo::TILES, STAGES = Geo::STAGES, RING = Geo::RING;
    constexpr int BOXES = Geo::BOXES, BOX = Geo::BOX, TILE = Geo::TILE;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sq = smem;
    unsigned char* ring = smem + TILES * TILE;
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + STAGES * TILE);
    uint64_t* empty = full + STAGES;
    uint64_t* q_full = empty + STAGES;
    uint64_t* q_empty = q_full + 2;     // [2] each, a tile (the second one DUAL only)
    uint64_t* s_full = q_empty + 2;     // [2] S of the next block is complete
    uint64_t* p_full = s_full + 2;      // [2] P is in place, and O is rescaled
    uint64_t* o_full = p_full + 2;      // [2] O is complete
    uint64_t* work_full = o_full + 2;   // [2]
    uint64_t* work_empty = work_full + 2;
    uint64_t* next_full = work_empty + 2;
    uint64_t* drained = next_full + 1;
    unsigned char* answer = reinterpret_cast<unsigned char*>(drained + 3);  // 16 bytes
    Work* work = reinterpret_cast<Work*>(answer + 16);                      // [2]
    static_assert(sizeof(Work) <= 64, "room for two pieces of work");
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(work + 2);
    float* join = reinterpret_cast<float*>(tmem_at + 4);  // [2][128] what the pipelines tell each other (single)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], DUAL ? 2 : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], DUAL ? 1 : 2);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&work_full[i], 1);
            mbar_init(&work_empty[i], 10);
            mbar_init(&drained[i], 1);
        }
        mbar_init(next_full, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_at, 512);
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    pdl_wait_primary();  // the previous kernel in the stream may still be running
    pdl_launch_dependents();

    if (warp >= kCopyWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kCopyWarp) {
            // ---------------- work and copies ----------------
            bool ok = true;
            int n0 = 0, n1 = 0;   // tiles through the ring of pipeline 0 (or both) and 1
            int qn[2] = {0, 0};   // loads of either query tile
            int wn = 0;           // pieces of work
            int id = blockIdx.x;
            for (int asked = 0; ok; ++asked) {
                Work w;
                w.valid = id >= 0;
                bool some = !w.valid;
                if (w.valid) {
                    const bool own = !DUAL && id >= p.shared_work;
                    const int at = own ? id - p.shared_work : id;
                    const int splits = own ? p.own_splits : p.splits;
                    int split, place;  // place: the tile, or the query token with own keys
                    if (!own && p.side_by_side) {
                        place = at % p.tiles;
                        w.h = at / p.tiles % p.Hkv;
                        split = at / p.tiles / p.Hkv;
                    } else {
                        w.h = at % p.Hkv;
                        split = at / p.Hkv % splits;
                        place = at / p.Hkv / splits;
                    }
                    w.it = own ? own_item(p, place) : find_item(p, p.tiles - 1 - place, TILES * p.tok);
                    some = w.it.t0 >= 0 && w.it.t0 < w.it.Lq;
                    // equal parts of what the tiles (or the query token) see
                    int seen = w.it.Lk;
                    if (!own && p.causal) seen -= w.it.Lq - min(w.it.Lq, w.it.t0 + TILES * p.tok);
                    const int blocks = (max(seen, 0) + kBlock - 1) / kBlock;
                    const int chunk = max(own ? p.own_chunk : p.chunk, (blocks + splits - 1) / splits * kBlock);
                    w.c0 = split * chunk;
                    w.c1 = min(w.it.Lk, w.c0 + chunk);
                    w.rec = (own ? p.own_rec0 : p.rec0) + split;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int first = w.it.t0 + (DUAL ? i : 0) * p.tok;
                        const int ntok = min(p.tok, w.it.Lq - first);
                        int most = w.c1;
                        if (p.causal) most = min(most, w.it.Lk - w.it.Lq + first + ntok);
                        most -= w.c0;
                        w.nb[i] = ntok > 0 && most > 0 ? (most + kBlock - 1) / kBlock : 0;
                    }
                    // A part behind the end of the keys (a short context in a wide table has many) gets
                    // l = 0 in its records here; the merge then skips their O.  (Every 256th is handed on:
                    // the other warps wait for work with a time limit.  So are those of two tiles, whose
                    // contexts have fewer parts: the code alone cost 512 tokens 0.3 of 11.8 us.)
                    if (!DUAL && some && (own || split > 0) && w.nb[0] == 0 && w.nb[1] == 0 && (asked & 255) != 255) {
                        mark_empty(p.part_ml, w.it.q0 + w.it.t0, own ? 1 : min(TILES * p.tok, w.it.Lq - w.it.t0), p.G,
                                   w.h, p.Hq, p.rec_stride, w.rec);
                        some = false;
                    }
                }
                if (some) {
                    // hand it on (or the end)
                    const int slot = wn & 1;
                    ok = warp_wait(&work_empty[slot], ((uint32_t)(wn >> 1) & 1u) ^ 1u, p.wait_limit_ns);
                    if (!ok) break;
                    if (lane == 0) {
                        work[slot] = w;
                        mbar_arrive(&work_full[slot]);
                    }
                    ++wn;
                    if (!w.valid) break;
                    const int blocks = max(w.nb[0], w.nb[1]);
                    if (blocks > 0) {
                        auto query = [&](int i) {  // tile i of the queries
                            if (DUAL && w.nb[i] == 0) return;
                            ok = ok && warp_wait(&q_empty[i], ((uint32_t)qn[i] & 1u) ^ 1u, p.wait_limit_ns);
                            if (!ok) return;
                            ++qn[i];
                            if (lane == 0) {
                                const uint32_t qbytes = (uint32_t)((w.it.own ? 1 : p.tok) * p.G * D * 2);
                                const void* map = w.it.own ? static_cast<const void*>(&maps.own_q) : &maps.q;
                                mbar_arrive_expect_tx(&q_full[i], qbytes);
                                for (int bx = 0; bx < BOXES; ++bx)
                                    tma_load_3d(sq + i * TILE + bx * BOX, map, 64 * bx, w.h * p.G,
                                                w.it.q0 + w.it.t0 + i * p.tok, &q_full[i]);
                            }
                        };
                        query(0);
                        if (!ok) break;
                        // Page ids by the warp, 32 pages a register: the windows of 16 blocks alternate
                        // between two of them, the next one fetched when the keys are 4 blocks into the
                        // current one (the values are at most 2 blocks behind).
                        int window[2] = {-1, -1};
                        const int pages = PAGED ? pages_of(p, w.it) : 0;
                        auto fetch = [&](int win) {
                            const int pi = w.c0 / kTile + 32 * win + lane;
                            return pi < pages ? table_of(p, w.it)[pi] : -1;
                        };
                        auto page = [&](int rel) {  // of page `rel` of the chunk
                            return __shfl_sync(0xffffffffu, rel & 32 ? window[1] : window[0], rel & 31);
                        };
                        // block j of the keys (which = 0) or values (1) into the next stage
                        auto load = [&](int j, int which) {
                            int page0 = 0, page1 = 0;
                            if (PAGED) {
                                if (which == 0 && j == 0) window[0] = fetch(0);
                                if (which == 0 && (j & 15) == 4) {
                                    const int next = fetch((j >> 4) + 1);
                                    if (j & 16) window[0] = next;
                                    else window[1] = next;
                                }
                                page0 = page(2 * j);
                                page1 = page(2 * j + 1);
                            }
                            int& n = !DUAL && (j & 1) ? n1 : n0;
                            const int s = (!DUAL && (j & 1) ? RING : 0) + n % RING;
                            ok = ok && warp_wait(&empty[s], ((uint32_t)(n / RING) & 1u) ^ 1u, p.wait_limit_ns);
                            if (!ok) return;
                            // (fault injection: that key tile gets no copy and no arrival)
                            if (lane == 0 && (which || j != p.withhold_tile)) {
                                const void* map = which ? static_cast<const void*>(&maps.v) : &maps.k;
                                unsigned char* dst = ring + s * TILE;
                                const int at = w.c0 + j * kBlock;
                                mbar_arrive_expect_tx(&full[s], TILE);
                                if (PAGED) {
#pragma unroll
                                    for (int half = 0; half < 2; ++half) {
                                        const int pg = half ? page1 : page0;
                                        int y = p.zero_row;  // past the pool: zeros
                                        if (pg >= 0 && pg < p.num_pages) y = (pg * p.Hkv + w.h) * kTile;
                                        else if (at + half * kTile < w.it.Lk) atomicOr(&g_status_rows, kStatusBadPage);
#pragma unroll
                                        for (int bx = 0; bx < BOXES; ++bx)
                                            tma_load_2d(dst + bx * BOX + half * (BOX / 2), map, 64 * bx, y, &full[s]);
                                    }
                                } else {
                                    int y = w.h;
                                    if (w.it.own) {
                                        map = which ? &maps.own_v : &maps.own_k;
                                        y += w.it.seq * p.Hkv;
                                    }
#pragma unroll
                                    for (int bx = 0; bx < BOXES; ++bx)
                                        tma_load_3d(dst + bx * BOX, map, 64 * bx, y, w.it.k0 + at, &full[s]);
                                }
                            }
                            ++n;
                        };
                        constexpr int AHEAD = DUAL ? 1 : 2;  // blocks by which the keys run ahead of the values
                        for (int j = 0; j < AHEAD && j < blocks; ++j) load(j, 0);
                        // The second tile's queries before the first values when paged, behind them when
                        // not (the other way round each 1% slower).
                        if (DUAL && PAGED) query(1);
                        for (int j = 0; ok && j < blocks; ++j) {
                            load(j, 1);
                            if (DUAL && !PAGED && j == 0) query(1);
                            if (j + AHEAD < blocks) load(j + AHEAD, 0);
                        }
                        if (!ok) break;
                    }
                }
                // all copies of this piece are under way: ask for the next one
                if (lane == 0) {
                    mbar_arrive_expect_tx(next_full, 16);
                    next_cta_request(answer, next_full);
                }
                ok = warp_wait(next_full, (uint32_t)asked & 1u, p.wait_limit_ns);
                if (ok) id = next_cta(answer);
                __syncwarp();
            }
            if (!ok) {
                // the others stopped early: let the copies in flight land before the CTA ends
                if (lane == 0) atomicOr(&g_status_rows, kStatusTimeout);
                for (int i = 0; i < 2; ++i)
                    if (qn[i] > 0) mbar_wait(&q_full[i], (uint32_t)(qn[i] - 1) & 1u, p.wait_limit_ns);
                for (int u = max(0, n0 - RING); u < n0; ++u)
                    mbar_wait(&full[u % RING], (uint32_t)(u / RING) & 1u, p.wait_limit_ns);
                for (int u = max(0, n1 - RING); u < n1; ++u)
                    mbar_wait(&full[RING + u % RING], (uint32_t)(u / RING) & 1u, p.wait_limit_ns);
                mbar_wait(next_full, 0, p.wait_limit_ns);
                mbar_wait(next_full, 1, p.wait_limit_ns);
            }
        } else if (warp < kMmaWarp + 2) {
            // ---------------- products ----------------
            // One warp per pipeline: an MMA is taken about when it starts to run, so what a warp does
            // between its products (waits, commits) leaves the tensor cores to the other one.
            constexpr uint32_t IQK = mma_desc(kBlock, false), IPV = mma_desc(D, true);
            const uint32_t ring_at = smem_u32(ring), tm = uniform(tmem);
            const uint32_t i = uniform(warp - kMmaWarp);
            const uint32_t q_desc = desc_rows(smem_u32(sq) + (DUAL ? i : 0) * TILE);
            const uint32_t s_tm = tm + i * 128, o_tm = tm + 256 + i * D;
            bool ok = true;
            uint32_t n0 = 0, qn = 0, rounds = 0;  // ring position, pieces of work with keys, blocks so far
            auto arrive = [&](uint32_t n) {  // tile n of the pipeline's ring is there: its stage
                const uint32_t s = (DUAL ? 0 : i * RING) + n % RING;
                ok = ok && warp_wait(&full[s], (n / RING) & 1u, p.wait_limit_ns);
                return s;
            };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) mma_commit(bar);
            };
            auto qk = [&](uint32_t stage) {  // S = Q K^T
                const uint32_t ka = desc_rows(ring_at + stage * TILE);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk / 4) * BOX + (kk % 4) * 32) >> 4;
                        mma_ss(s_tm, q_desc + off, ka + off, IQK, kk > 0);
                    }
                    mma_commit(&s_full[i]);
                    mma_commit(&empty[stage]);
                }
            };
            auto pv = [&](uint32_t stage, bool first) {  // O += P V
                const uint32_t va = desc_cols(ring_at + stage * TILE);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < (FINE ? 2 : 1) * kBlock / 16; ++kk)  // (lo lies behind hi)
                        mma_ts(o_tm, s_tm + kk * 8, va + (kk % (kBlock / 16) * 16 * 128 >> 4), IPV, !first || kk > 0);
                    mma_commit(&empty[stage]);
                }
            };
            for (int wn = 0; ok; ++wn) {
                const int slot = wn & 1;
                ok = warp_wait(&work_full[slot], (uint32_t)(wn >> 1) & 1u, p.wait_limit_ns);
                if (!ok) break;
                const Work& w = work[slot];
                const bool valid = uniform(w.valid) != 0;
                const int nb0 = (int)uniform(w.nb[0]), nb1 = (int)uniform(w.nb[1]);
                const int left0 = w.it.Lk - w.c0;  // keys of the sequence from the chunk on
                __syncwarp();
                if (lane == 0) mbar_arrive(&work_empty[slot]);
                if (!valid) break;
                const int blocks = max(nb0, nb1);
                if (blocks == 0) continue;
                // the pipeline's rounds: blocks 0, 1, .. or every second one from i on
                const int nb = DUAL ? (i ? nb1 : nb0) : (blocks + 1 - (int)i) / 2;
                const int in_ring = DUAL ? blocks : nb;
                // Value rows past the sequence may hold anything; their weight is 0, but 0 * NaN is NaN.
                // (Both warps of a shared tile clear them, each before its own products: the second
                // stores zeros over zeros, before the tile is released.)
                auto clear_tail = [&](int j, uint32_t stage) {
                    const int rows = left0 - j * kBlock;
                    if (rows >= kBlock) return;
                    unsigned char* v = ring + stage * TILE;
                    for (int x = lane; x < (kBlock - rows) * 8; x += 32)
#pragma unroll
                        for (int bx = 0; bx < BOXES; ++bx)
                            *reinterpret_cast<uint4*>(v + bx * BOX + rows * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                };
                const uint32_t qt = DUAL ? i : 0;
                if (!DUAL || nb > 0) {
                    ok = warp_wait(&q_full[qt], qn & 1u, p.wait_limit_ns);
                    ++qn;
                }
                if (ok && nb > 0) {
                    const uint32_t s0 = arrive(n0);
                    if (!ok) break;
                    qk(s0);
                    if (nb == 1) commit(&q_empty[qt]);
                    for (int r = 0; r < nb; ++r) {
                        const bool more = r + 1 < nb;
                        const uint32_t sv = arrive(n0 + 2 * r + 1);
                        if (!ok) break;
                        clear_tail(DUAL ? r : 2 * r + (int)i, sv);
                        const uint32_t sk = more ? arrive(n0 + 2 * r + 2) : 0;
                        ok = ok && warp_wait(&p_full[i], rounds & 1u, p.wait_limit_ns);
                        if (!ok) break;
                        ++rounds;
                        tc_fence_after();
                        pv(sv, r == 0);
                        if (more) qk(sk);
                        else commit(&o_full[i]);
                        if (r + 2 == nb) commit(&q_empty[qt]);
                    }
                } else if (!DUAL && ok && lane == 0) {
                    mbar_arrive(q_empty);
                }
                // tiles that only the other pipeline needs
                for (int x = 2 * nb; ok && x < 2 * in_ring; ++x) {
                    const uint32_t s = arrive(n0 + x);
                    if (ok && lane == 0) mbar_arrive(&empty[s]);
                }
                n0 += 2 * in_ring;
            }
            if (!ok) {
                if (lane == 0) atomicOr(&g_status_rows, kStatusTimeout);
                commit(&drained[i]);
                warp_wait(&drained[i], 0, p.wait_limit_ns);
            }
        }
    } else {
        // ---------------- softmax, one row per thread ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int i = warp >> 2;  // pipeline
        const int r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes per warp, lane in the upper half
        const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + 256;
        const int tk = r / p.G;
        bool ok = true;
        uint32_t s_round = 0, o_round = 0;
        for (int wn = 0; DUAL ? ok : true; ++wn) {
            const int slot = wn & 1;
            ok = ok && warp_wait(&work_full[slot], (uint32_t)(wn >> 1) & 1u, p.wait_limit_ns);
            // the warpgroups of a single tile meet at barriers: all of them stop, or none
            if (DUAL ? !ok : named_barrier_or(2, 256, !ok)) break;
            const Work& wk = work[slot];
            const bool valid = wk.valid != 0;
            RowsItem it = wk.it;
            if (DUAL) it.own = 0;  // known to be
            const int h = wk.h, c0 = wk.c0, c1 = wk.c1, rec_at = wk.rec;
            const int nb = i ? wk.nb[1] : wk.nb[0];
            const int all = wk.nb[0];
            __syncwarp();
            if (lane == 0) mbar_arrive(&work_empty[slot]);
            if (!valid) break;
            const int first = it.t0 + (DUAL ? i : 0) * p.tok;
            const bool live = tk < p.tok && first + tk < it.Lq;
            const int lim = live ? min(visible_keys(p, it, first + tk), c1) - c0 : 0;
            const int rounds = DUAL ? nb : (nb + 1 - i) / 2;
            const int32_t* table = PAGED ? table_of(p, it) : nullptr;
            const int pages = PAGED ? pages_of(p, it) : 0;
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            for (int round = 0; round < rounds; ++round) {
                const int j = DUAL ? round : 2 * round + i;
                const int left = lim - j * kBlock;  // visible keys from this block on
                bool bad[2] = {false, false};
                if (PAGED) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int pi = (c0 + j * kBlock) / kTile + half;
                        if (pi < pages) {
                            const int pg = table[pi];
                            bad[half] = pg < 0 || pg >= p.num_pages;
                        }
                    }
                }
                ok = warp_wait(&s_full[i], s_round & 1u, p.wait_limit_ns);
                if (!ok) break;
                ++s_round;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s[c], s_at + 32 * c);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) tie32(s[c]);
                if (__any_sync(0xffffffffu, left < kBlock || bad[0] || bad[1])) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int n = bad[c >> 1] ? 0 : min(max(left - 32 * c, 0), 32);
                        const uint32_t seen = n < 32 ? (1u << n) - 1u : 0xffffffffu;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen & 1u << e)) s[c][e] = 0xff800000u;  // -inf
                    }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) mx[c] = fmaxf(mx[c], __uint_as_float(s[c][e]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                if (__any_sync(0xffffffffu, top > m + kRescaleAt)) {
                    const float mn = fmaxf(m, top);
                    const float a = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
                    m = mn;
                    l2 = f2mul(l2, make_float2(a, a));
                    if (round > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(o, o_at + i * D + 32 * c);
                            tmem_wait_ld();
                            tie32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                            tmem_st32(o_at + i * D + 32 * c, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nb2 = make_float2(-base, -base);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w[32], lo[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = 2 * half + e / 16, x = 2 * (e % 16);
                        float2 f = f2fma(make_float2(__uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1])), sc2, nb2);
                        f = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                        l2 = __fadd2_rn(l2, f);
                        if (FINE) split_bf16(f.x, f.y, w[e], lo[e]);
                        else w[e] = pack_bf16(f.x, f.y);
                    }
                    tmem_st32(s_at + 32 * half, w);
                    if (FINE) tmem_st32(s_at + 64 + 32 * half, lo);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
            }
            const int head = h * p.G + r - tk * p.G;
            const size_t row = (size_t)(it.q0 + first + tk) * p.Hq + head;
            const size_t rec = row * p.rec_stride + rec_at;
            // l is 0 only where nothing of weight was seen.  A NaN or +inf score makes it NaN (m skips NaN
            // and may still be -inf), and that has to pass on to the result: hence no test l > 0.
            float l = ok ? l2.x + l2.y : 0.f;
            auto statistics = [&] {
                if (!p.direct) {
                    p.part_ml[2 * rec] = m;
                    p.part_ml[2 * rec + 1] = l;
                } else if (p.lse) {
                    p.lse[row] = l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
                }
            };
            // what does not need O goes before the wait for it
            const float inv_own = l != 0.f ? 1.f / l : 0.f;
            if (DUAL && live) statistics();
            if (ok && rounds > 0) {
                ok = warp_wait(&o_full[i], o_round & 1u, p.wait_limit_ns);
                ++o_round;
            }
            tc_fence_after();
            if (!ok) {
                l = 0.f;
                m = -INFINITY;
            }
            // factors of the O of pipeline 0 and 1
            float f0 = i ? 0.f : 1.f, f1 = i ? 1.f : 0.f;
            if (!DUAL) {
                // pipeline 0 learns m and l of pipeline 1 and tells the factors; each
                // warpgroup then writes half of the channels of the joined result
                if (i == 1) {
                    join[r] = m;
                    join[128 + r] = l;
                }
                tc_fence_before();
                named_barrier(1, 256);  // (both O are complete: each warpgroup has waited for its own)
                if (i == 0) {
                    const float m1 = join[r], l1 = join[128 + r], m0 = m;
                    m = fmaxf(m0, m1);
                    f0 = m0 == -INFINITY ? 0.f : exp2_approx(m0 - m);
                    f1 = m1 == -INFINITY ? 0.f : exp2_approx(m1 - m);
                    l = f0 * l + f1 * l1;
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    join[r] = f0 *= inv;
                    join[128 + r] = f1 *= inv;
                }
                named_barrier(1, 256);
                tc_fence_after();
                if (i == 1) {
                    f0 = join[r];
                    f1 = join[128 + r];
                }
            }
            auto channels = [&](int c, float (&f)[32]) {  // 32 of the result's
                uint32_t o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] = 0.f;
                if (DUAL ? rounds > 0 : all > 0) {
                    const float by = DUAL ? inv_own : f0;
                    tmem_ld32(o, o_at + (DUAL ? i * D : 0) + c);
                    tmem_wait_ld();
                    tie32(o);
                    if (by != 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * by;
                    }
                }
                if (!DUAL && all > 1) {
                    tmem_ld32(o, o_at + D + c);
                    tmem_wait_ld();
                    tie32(o);
                    if (f1 != 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] += __uint_as_float(o[e]) * f1;
                    }
                }
            };
            // This code runs once a piece: fetching it takes longer than running it, so its loops are
            // rolled up (32 prompts of 512: 116 us unrolled, 100 us).
            constexpr int MINE = DUAL ? D : D / 2;  // channels that this warpgroup writes
            const int c_mine = DUAL ? 0 : i * MINE;
            if (p.direct && p.out_bf16) {
                uint16_t* dst = static_cast<uint16_t*>(p.out) + row * D;
#pragma unroll 1
                for (int c = c_mine; c < c_mine + MINE; c += 32) {
                    float f[32];
                    channels(c, f);
                    if (!live) continue;
                    uint32_t x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
                    store32(dst + c, x, p.wide);
                    store32(dst + c + 16, x + 8, p.wide);
                }
            } else {
                float* dst = p.direct ? static_cast<float*>(p.out) + row * D : p.part_o + rec * D;
                // the merge skips records with l = 0 (of a single tile, only pipeline 0 knows the joined l)
                const bool wanted = live && (p.direct || (DUAL ? l != 0.f : f0 != 0.f || f1 != 0.f));
#pragma unroll 1
                for (int c = c_mine; c < c_mine + MINE; c += 32) {
                    float f[32];
                    channels(c, f);
                    if (!wanted) continue;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        store32(dst + c + 8 * e, reinterpret_cast<uint32_t*>(f) + 8 * e, p.wide);
                }
            }
            if (!DUAL && live && i == 0) statistics();
            tc_fence_before();
            if (!DUAL) named_barrier(1, 256);  // both O and the factors are read
        }
        if (!ok && lane == 0) atomicOr(&g_status_rows, kStatusTimeout);
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

int rows_tok(int G) { return kRows / G; }

// Two tiles per CTA when the sequences fill more than one on average (64 x 128 tokens
// behind 2048: 207 us in two, 287 us in one; 64 x 24: 113 and 100 us; between one tile
// and two within 12% of each other), or when packed sequences have a block of keys on
// average, which a single tile would leave to one of its pipelines (64 x 24 tokens
// alone: 17.8 us in two, 21.9 us in one; 256 x 16 on 100 keys 51 and 60 us).  packed_k:
// the keys of a packed call, -1 else.
bool rows_dual(int B, int total_q, int G, long long packed_k) {
    if (B <= 0) return false;
    return total_q / B > rows_tok(G) || (packed_k >= 0 && packed_k <= (long long)kBlock * B);
}

template <int D, bool PAGED, bool DUAL, bool FINE>
cudaError_t launch_kernel(const RowsMaps& maps, const RowsParams& p, dim3 grid, cudaStream_t stream) {
    constexpr auto kernel = rows_kernel<D, PAGED, DUAL, FINE>;
    constexpr int SMEM = RowsGeo<D, DUAL>::SMEM;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        // the warpgroups' register shares are cut from what the block is launched with
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kernel);
        if (e != cudaSuccess) return e;
        if (attr.numRegs * kThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
        if (dev < 64) done[dev] = true;
    }
    return launch_pdl(kernel, grid, dim3(kThreads), SMEM, stream, maps, p);
}

}  // namespace

bool rows_single(int B, int total_q, int G, int packed_k) { return !rows_dual(B, total_q, G, packed_k); }

int rows_tokens(int B, int total_q, int G, int packed_k) {
    return rows_tok(G) * (rows_dual(B, total_q, G, packed_k) ? 2 : 1);
}

long long rows_tiles(int B, int total_q, int G, int packed_k, bool offsets) {
    const int per = rows_tokens(B, total_q, G, packed_k);
    return offsets ? (long long)total_q / per + B : ((long long)total_q + per - 1) / per;
}

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t stream) {
    if (a.total_q == 0 || a.B == 0) return cudaSuccess;
    RowsParams p;
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.seq_lens = a.seq_lens;
    p.row_lens = a.row_lens;
    p.page_table = a.page_table;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.table_stride = a.table_stride;
    p.B = a.B;
    p.total_q = a.total_q;
    p.total_k = a.total_k;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.tok = rows_tok(p.G);
    p.max_k = a.max_k;
    p.scale_log2 = a.scale * kLog2e;
    p.causal = a.causal;
    p.splits = a.splits;
    p.chunk = a.chunk;
    p.out = a.out;
    p.out_bf16 = a.out_bf16;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_ml = a.part_ml;
    p.rec0 = a.rec0;
    p.rec_stride = a.rec_stride;
    p.direct = a.direct;
    p.wide = (reinterpret_cast<uintptr_t>(a.direct ? a.out : static_cast<void*>(a.part_o)) & 31u) == 0;
    const bool paged = a.page_table != nullptr;
    const uint64_t pool_rows = paged ? (uint64_t)a.num_pages * a.Hkv * kTile : 0;
    p.zero_row = (int)(pool_rows > 0 ? pool_rows : 1);
    RowsMaps m;
    if (!make_token_map(&m.q, a.q, a.D, a.Hq, a.total_q, a.D, a.q_stride, p.G, p.tok)) return cudaErrorInvalidValue;
    bool ok = true;
    if (paged && pool_rows > 0) {
        ok = make_row_map(&m.k, a.k, pool_rows, (uint32_t)a.D * 2) &&
             make_row_map(&m.v, a.v, pool_rows, (uint32_t)a.D * 2);
    } else if (paged) {  // an empty pool: nothing is read, any well-formed map will do
        ok = make_row_map(&m.k, a.q, 1, (uint32_t)a.D * 2);
        m.v = m.k;
    } else if (a.total_k > 0) {
        ok = make_token_map(&m.k, a.k, a.D, a.Hkv, a.total_k, a.k_head_stride, a.k_stride, 1, kBlock) &&
             make_token_map(&m.v, a.v, a.D, a.Hkv, a.total_k, a.v_head_stride, a.v_stride, 1, kBlock);
    } else {
        m.k = m.v = m.q;
    }
    m.own_q = m.own_k = m.own_v = m.q;
    const int packed_k = a.cu_k ? a.total_k : -1;
    const bool dual = rows_dual(a.B, a.total_q, p.G, packed_k);
    const long long own_work = a.own_max > 0 ? (long long)a.total_q * a.Hkv * a.own_splits : 0;
    if (own_work > 0) {
        if (dual) return cudaErrorInvalidValue;
        ok = ok && make_token_map(&m.own_q, a.q, a.D, a.Hq, a.total_q, a.D, a.q_stride, p.G, 1);
        if (!paged) {
            const long long head = (long long)a.own_max * a.D;
            ok = ok && make_token_map(&m.own_k, a.own_k, a.D, a.total_q * a.Hkv, a.own_max, head, a.D, 1, kBlock) &&
                 make_token_map(&m.own_v, a.own_v, a.D, a.total_q * a.Hkv, a.own_max, head, a.D, 1, kBlock);
        }
    }
    if (!ok) return cudaErrorInvalidValue;
    p.own_lens = a.own_lens;
    p.own_table = a.own_table;
    p.own_table_stride = a.own_table_stride;
    p.own_max = a.own_max;
    p.own_skip = a.own_skip;
    p.own_splits = a.own_splits;
    p.own_chunk = a.own_chunk;
    p.own_rec0 = a.own_rec0;
    const long long tiles = rows_tiles(a.B, a.total_q, p.G, packed_k, a.cu_q != nullptr);
    p.tiles = (int)tiles;
    // one sequence of keys for all tiles: those of a chunk read it from L2 together
    p.side_by_side = a.cu_q == nullptr;
    injected_timeout(&p.wait_limit_ns, &p.withhold_tile);
    p.shared_work = (int)(tiles * a.Hkv * a.splits);
    const dim3 grid((unsigned)(p.shared_work + own_work));
    const auto launch = [&](auto d, auto pages) {
        constexpr int D = decltype(d)::value;
        constexpr bool P = decltype(pages)::value;
        if (dual) return a.fine ? launch_kernel<D, P, true, true>(m, p, grid, stream)
                                : launch_kernel<D, P, true, false>(m, p, grid, stream);
        return a.fine ? launch_kernel<D, P, false, true>(m, p, grid, stream)
                      : launch_kernel<D, P, false, false>(m, p, grid, stream);
    };
    using std::integral_constant;
    if (a.D == 128) return paged ? launch(integral_constant<int, 128>(), std::true_type())
                                 : launch(integral_constant<int, 128>(), std::false_type());
    return paged ? launch(integral_constant<int, 64>(), std::true_type())
                 : launch(integral_constant<int, 64>(), std::false_type());
}

cudaError_t rows_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_rows, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_rows, &zero, sizeof(unsigned));
}

}  // namespace fd
