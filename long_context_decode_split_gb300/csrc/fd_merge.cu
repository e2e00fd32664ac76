// fd_merge.cu -- merge of lists of partial results for sm_103a: the parts of a
// prompt tile's keys, and the chunks of a shared-prefix decode.  (In a file of its
// own: beside the rows kernel, whatever changed this code moved that one's in
// memory, and 8000 tokens of one KV head took 87 to 94 us.)
#include "fd_device.cuh"
#include "fd_internal.h"

namespace fd {

__device__ unsigned int g_status_merge;

namespace {

// Merge of a list of n partials per row (every (m, l) written; l = 0 where
// nothing was attended, and O then need not be): out = sum_i w_i O_i / sum_i w_i,
// w_i = 2^(m_i - M) l_i.
// A NaN l (a NaN score, m = -inf where it saw no other) makes the row NaN.
// W warps per row (1: eight rows per CTA; 8: one row, the warps taking every
// eighth record and joining through shared memory), eight records in flight.
// The records come from L2, and the length of the list bounds it: 10 us of a
// shared prefix of 128 sequences.
template <int D, int W>
__global__ void __launch_bounds__(256)
merge_list_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml, const int32_t* __restrict__ cu,
                  int B, long long rows, int Hq, int n, void* __restrict__ out, int out_bf16, float* __restrict__ lse,
                  const int32_t* __restrict__ lens, int len_most) {
    constexpr int E = D / 32;  // channels per lane
    constexpr int AHEAD = 8;
    __shared__ float part[W > 1 ? W : 1][D + 1];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int w0 = W > 1 ? warp : 0;
    const long long row = (long long)blockIdx.x * (8 / W) + warp / W;
    if (row >= rows) return;
    if (cu) {
        const int token = (int)(row / Hq);
        if (token < cu[0] || token >= cu[B]) return;
    }
    if (lens && lane == 0) {  // lengths that no other part of the call looks at
        const int len = lens[row / Hq];
        if (len < 0 || len > len_most) atomicOr(&g_status_merge, kStatusBadSeqLen);
    }
    const float2* ml = reinterpret_cast<const float2*>(part_ml) + row * n;
    const float* po = part_o + row * n * D + lane * E;
    auto load = [&](int i, float (&v)[E]) {
        if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4*>(po + (size_t)i * D);
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(po + (size_t)i * D);
            v[0] = x.x; v[1] = x.y;
        }
    };
    float v[AHEAD][E];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        if (w0 + u * W < n) load(w0 + u * W, v[u]);
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float top = M == -INFINITY ? 0.f : M;
    float sum = 0.f, acc[E] = {};
    // this warp's records i = w0 + W j, 32 at a time
    const int mine = (n - w0 + W - 1) / W;
    for (int base = 0; base < mine; base += 32) {
        float w = 0.f;
        if (base + lane < mine) {
            const float2 x = ml[w0 + W * (base + lane)];
            if (x.y != 0.f) w = exp2_approx(x.x - top) * x.y;
        }
        const int cnt = 32 - __clz(__ballot_sync(0xffffffffu, w != 0.f));  // up to the last one that counts
        for (int j = 0; j < cnt; j += AHEAD) {
            if (base + j > 0) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u)
                    if (j + u < cnt) load(w0 + W * (base + j + u), v[u]);
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const float wu = __shfl_sync(0xffffffffu, w, (j + u) & 31);
                if (j + u < cnt && wu != 0.f) {
                    sum += wu;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += wu * v[u][e];
                }
            }
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
        if (lane == 0) part[warp][D] = sum;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int u = 1; u < W; ++u) {
            sum += part[u][D];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += part[u][lane * E + e];
        }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
    if (out_bf16) {
        uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + row * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) o[e / 2] = pack_bf16(acc[e], acc[e + 1]);
    } else {
        float* o = static_cast<float*>(out) + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = acc[e];
    }
    if (lane == 0 && lse) lse[row] = sum != 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_merge_list(const float* part_o, const float* part_ml, const int32_t* cu, int B, int tokens, int Hq,
                              int D, int n, void* out, int out_bf16, float* lse, cudaStream_t stream,
                              const int32_t* lens, int len_most) {
    const long long rows = (long long)tokens * Hq;
    // few rows with long lists leave most of the GPU idle with a warp each (the whole
    // call, 256 rows: 14 records 17.0 us with a warp each, 15.1 us with eight, 9 records 16.9
    // and 17.2 us; 512 rows: 12 records 20.3 and 20.7 us, 20 records 20.6 and 17.0 us;
    // 8192 rows of 20 records 220 and 233 us)
    const bool wide = n > (rows <= 256 ? 8 : 16) && rows < 4096;
    const dim3 grid((unsigned)(wide ? rows : (rows + 7) / 8));
    const auto kernel = D == 128 ? (wide ? merge_list_kernel<128, 8> : merge_list_kernel<128, 1>)
                                 : (wide ? merge_list_kernel<64, 8> : merge_list_kernel<64, 1>);
    return launch_pdl(kernel, grid, dim3(256), 0, stream, part_o, part_ml, cu, B, rows, Hq, n, out, out_bf16, lse,
                      lens, len_most);
}

cudaError_t merge_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_merge, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_merge, &zero, sizeof(unsigned));
}

}  // namespace fd
