// fd_rows.cu -- attention of packed query rows for sm_103a: whole prompts,
// prompt tails over a paged cache, and the shared part of a shared-prefix
// decode.  A tile holds TOK consecutive query tokens of one sequence times the
// G query heads of one KV head (row = token * G + head), so every key and
// value read serves the whole group.
//
// For a row with the visible keys [0, n):
//   s_j = scale <q, k_j>,  out = sum_j e^(s_j) v_j / sum_j e^(s_j),
//   lse = ln sum_j e^(s_j)
// in one pass over the keys: m is the running maximum, l the running sum of
// 2^(s_j log2e - m), and O is rescaled when m moves.
#include <cmath>

#include "fd_device.cuh"
#include "fd_internal.h"

namespace fd {

__device__ unsigned int g_status_rows;

namespace {

struct RowsParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride, k_head_stride, v_head_stride;
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
    int chunk;
    void* out;
    int out_bf16;
    float* lse;
    float* part_o;
    float* part_ml;
    int rec0, rec_stride, direct;
};

// One tile's place: the sequence, its query tokens and its keys.
struct RowsItem {
    int seq;
    int q0, Lq;  // first query token of the sequence in the packed array, and their number
    int k0, Lk;  // the same of its keys (k0 = 0 when paged)
    int t0;      // first token of the tile within the sequence
};

__device__ __forceinline__ int checked_offset(const int32_t* cu, int i, int lo, int hi) {
    const int c = cu[i];
    if (c < lo || c > hi) {
        if (threadIdx.x == 0) atomicOr(&g_status_rows, kStatusBadSeqLen);
        return c < lo ? lo : hi;
    }
    return c;
}

// Tile slots: sequence s owns the slots floor(cu_q[s] / per) + s up to those of
// s + 1, at least as many as the tiles it has (`per` tokens each), so a slot's
// sequence is found by a search of cu_q alone.
__device__ __forceinline__ RowsItem find_item(const RowsParams& p, int slot, int per) {
    RowsItem it;
    it.seq = 0;
    it.q0 = 0;
    it.Lq = p.total_q;
    it.k0 = 0;
    if (p.cu_q) {
        // the last s with first_slot(s) <= slot; each round every lane probes one of 32 places
        const int lane = threadIdx.x & 31;
        int lo = 0, n = p.B;  // the answer is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int s = lo + lane * step;
            const bool below = lane * step < n && min(max(p.cu_q[s], 0), p.total_q) / per + s <= slot;
            const unsigned votes = __ballot_sync(0xffffffffu, below);
            const int hit = votes ? 31 - __clz(votes) : 0;
            lo += hit * step;
            n = min(step, n - hit * step);
        }
        it.seq = lo;
        it.q0 = checked_offset(p.cu_q, lo, 0, p.total_q);
        it.Lq = checked_offset(p.cu_q, lo + 1, it.q0, p.total_q) - it.q0;
    }
    it.t0 = (slot - (it.q0 / per + it.seq)) * per;
    if (p.page_table) {
        it.Lk = clamped_len(p.seq_lens, it.seq, p.max_k, &g_status_rows);
    } else if (p.cu_k) {
        it.k0 = checked_offset(p.cu_k, it.seq, 0, p.total_k);
        it.Lk = checked_offset(p.cu_k, it.seq + 1, it.k0, p.total_k) - it.k0;
    } else {
        it.Lk = p.total_k;
    }
    return it;
}

// Keys that query token t of the item's sequence sees.
__device__ __forceinline__ int visible_keys(const RowsParams& p, const RowsItem& it, int t) {
    int n = it.Lk;
    if (p.causal) n = min(n, it.Lk - it.Lq + t + 1);
    if (p.row_lens) n = min(n, p.row_lens[it.q0 + t]);
    return max(n, 0);
}

// Four warps, 16 rows each; keys in tiles of 64.
template <int D, bool PAGED>
__global__ void __launch_bounds__(128) rows_kernel(const RowsParams p) {
    constexpr int C = D / 8;  // 16-byte chunks of a row
    __shared__ __align__(1024) unsigned char smem[2 * 64 * D * 2];
    unsigned char* sk = smem;
    unsigned char* sv = smem + 64 * D * 2;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3, mi = lane >> 3;
    const int h = blockIdx.x % p.Hkv, split = blockIdx.y;
    const RowsItem it = find_item(p, (int)(gridDim.x / p.Hkv - 1 - blockIdx.x / p.Hkv), p.tok);
    if (it.t0 < 0 || it.t0 >= it.Lq) return;
    const int ntok = min(p.tok, it.Lq - it.t0);

    int lim[2], token[2], head[2];
    bool live[2];
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = warp * 16 + gid + 8 * i;
        token[i] = r / p.G;
        head[i] = h * p.G + r % p.G;
        live[i] = r < p.tok * p.G && token[i] < ntok;
        lim[i] = live[i] ? visible_keys(p, it, it.t0 + token[i]) : 0;
        token[i] += it.q0 + it.t0;
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(p.q + (size_t)token[i] * p.q_stride + (size_t)head[i] * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qa[kk][i] = live[i] ? qr[8 * kk + tig] : 0u;
            qa[kk][2 + i] = live[i] ? qr[8 * kk + 4 + tig] : 0u;
        }
    }
    const int c0 = split * p.chunk;
    int most = it.Lk;
    if (p.causal) most = min(most, it.Lk - it.Lq + it.t0 + ntok);
    const int c1 = min(most, c0 + p.chunk);

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int t = c0; t < c1; t += 64) {
        const int rows = min(64, c1 - t);
        bool ok = true;
        size_t krow = 0, vrow = 0;
        long long ks = p.k_stride, vs = p.v_stride;
        if (PAGED) {
            const int pg = p.page_table[(size_t)it.seq * p.table_stride + t / kTile];
            ok = pg >= 0 && pg < p.num_pages;
            if (!ok && threadIdx.x == 0) atomicOr(&g_status_rows, kStatusBadPage);
            krow = vrow = ((size_t)pg * p.Hkv + h) * kTile * D;
            ks = vs = D;
        } else {
            krow = (size_t)(it.k0 + t) * p.k_stride + (size_t)h * p.k_head_stride;
            vrow = (size_t)(it.k0 + t) * p.v_stride + (size_t)h * p.v_head_stride;
        }
        if (!ok) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * C; i += 128) {
            const int r = i / C, c = i % C;
            uint4 kk = make_uint4(0u, 0u, 0u, 0u), vv = kk;
            if (r < rows) {
                kk = *reinterpret_cast<const uint4*>(p.k + krow + (size_t)r * ks + c * 8);
                vv = *reinterpret_cast<const uint4*>(p.v + vrow + (size_t)r * vs + c * 8);
            }
            *reinterpret_cast<uint4*>(sk + swz(r, c)) = kk;
            *reinterpret_cast<uint4*>(sv + swz(r, c)) = vv;
        }
        __syncthreads();
        float s[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(smem_u32(sk) + swz(8 * n + 8 * (mi >> 1) + (lane & 7), 2 * kk + (mi & 1)), b0, b1, b2, b3);
                mma_bf16(s[n], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
                mma_bf16(s[n + 1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b2, b3);
            }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = t + 8 * n + 2 * tig + (e & 1);
                s[n][e] = col < min(lim[e >> 1], c1) ? s[n][e] * p.scale_log2 : -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
            }
        float a[2], base[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            const float mn = fmaxf(m[i], mx[i]);
            base[i] = mn == -INFINITY ? 0.f : mn;
            a[i] = exp2_approx(m[i] - base[i]);
            m[i] = mn;
            l[i] *= a[i];
        }
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[n][e] = exp2_approx(s[n][e] - base[e >> 1]);
                l[e >> 1] += s[n][e];
            }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= a[e >> 1];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const uint32_t a0 = pack_bf16(s[2 * kk][0], s[2 * kk][1]), a1 = pack_bf16(s[2 * kk][2], s[2 * kk][3]);
            const uint32_t a2 = pack_bf16(s[2 * kk + 1][0], s[2 * kk + 1][1]);
            const uint32_t a3 = pack_bf16(s[2 * kk + 1][2], s[2 * kk + 1][3]);
#pragma unroll
            for (int n = 0; n < D / 8; n += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(smem_u32(sv) + swz(16 * kk + 8 * (mi & 1) + (lane & 7), n + (mi >> 1)), b0, b1, b2, b3);
                mma_bf16(o[n], a0, a1, a2, a3, b0, b1);
                mma_bf16(o[n + 1], a0, a1, a2, a3, b2, b3);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (!live[i]) continue;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        const size_t row = (size_t)token[i] * p.Hq + head[i];
        const size_t rec = row * p.rec_stride + p.rec0 + split;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            const float x = o[n][2 * i] * inv, y = o[n][2 * i + 1] * inv;
            const int dim = 8 * n + 2 * tig;
            if (!p.direct) *reinterpret_cast<float2*>(p.part_o + rec * D + dim) = make_float2(x, y);
            else if (p.out_bf16)
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + dim) = pack_bf16(x, y);
            else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * D + dim) = make_float2(x, y);
        }
        if (tig == 0) {
            if (!p.direct) {
                p.part_ml[2 * rec] = l[i] > 0.f ? m[i] : -INFINITY;
                p.part_ml[2 * rec + 1] = l[i];
            } else if (p.lse) {
                p.lse[row] = l[i] > 0.f ? (m[i] + __log2f(l[i])) * kLn2 : -INFINITY;
            }
        }
    }
}

int rows_tok(int G) { return 64 / G; }

}  // namespace

long long rows_tiles(int B, int total_q, int G) { return (long long)total_q / rows_tok(G) + B; }

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t stream) {
    if (a.total_q == 0 || a.B == 0) return cudaSuccess;
    RowsParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint16_t*>(a.k);
    p.v = static_cast<const uint16_t*>(a.v);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.k_head_stride = a.k_head_stride;
    p.v_head_stride = a.v_head_stride;
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
    p.chunk = a.chunk;
    p.out = a.out;
    p.out_bf16 = a.out_bf16;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_ml = a.part_ml;
    p.rec0 = a.rec0;
    p.rec_stride = a.rec_stride;
    p.direct = a.direct;
    const long long tiles = rows_tiles(a.B, a.total_q, p.G);
    const dim3 grid((unsigned)(tiles * a.Hkv), (unsigned)a.splits);
    const bool paged = a.page_table != nullptr;
    if (a.D == 128)
        return paged ? launch_pdl(rows_kernel<128, true>, grid, dim3(128), 0, stream, p)
                     : launch_pdl(rows_kernel<128, false>, grid, dim3(128), 0, stream, p);
    return paged ? launch_pdl(rows_kernel<64, true>, grid, dim3(128), 0, stream, p)
                 : launch_pdl(rows_kernel<64, false>, grid, dim3(128), 0, stream, p);
}

cudaError_t rows_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_rows, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_rows, &zero, sizeof(unsigned));
}

}  // namespace fd
