// fd_pages.cu -- the paged cache's bookkeeping and writes for sm_103a: pages
// and slots for the new tokens of a batch, and the new key and value rows
// stored at those slots (bf16, or e4m3 codes with a scale per row).
#include <cstdint>

#include "fd_device.cuh"
#include "fd_internal.h"

namespace fd {

__device__ unsigned int g_status_pages;

namespace {

constexpr int kAssignThreads = 1024;

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kTile - 1) / kTile; }

// Exclusive sums over the block of two values per thread (and their totals).
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb,
                                            long long* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        red[warp] = a;
        red[32 + warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
        long long x = red[lane], y = red[32 + lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        red[lane] = x;
        red[32 + lane] = y;
    }
    __syncthreads();
    ta = red[31];
    tb = red[63];
    a += (warp ? red[warp - 1] : 0) - a0;
    b += (warp ? red[32 + warp - 1] : 0) - b0;
    __syncthreads();  // red may be used again
}

struct AssignParams {
    const int32_t* cached_lens;
    const int32_t* new_lens;
    int B;
    int32_t* page_table;
    int max_pages;
    const int32_t* free_pages;
    int num_free;
    const int32_t* free_head;
    int total_new;
    int32_t* seq_lens;
    int32_t* cu_new;
    int64_t* slots;
    int32_t* free_head_out;
};

// One block: sequences in groups of 1024, one per thread, with running sums of
// their new tokens and pages.  Inputs of a group are in registers before its
// outputs are written, so outputs may be the inputs' own buffers.
__global__ void __launch_bounds__(kAssignThreads) assign_kernel(const AssignParams p) {
    __shared__ long long red[64];
    __shared__ int cu_s[kAssignThreads + 1];
    __shared__ int cached_s[kAssignThreads];
    __shared__ int end_s[kAssignThreads];
    __shared__ long long base_s[kAssignThreads];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    long long head = p.free_head ? p.free_head[0] : 0;
    bool bad = false, out_of_pages = false;
    if (head < 0) {
        head = 0;
        bad = true;
    }
    const long long cap = (long long)p.max_pages * kTile;
    long long tokens = 0, pages = 0;  // before this group
    for (int b0 = 0; b0 < p.B; b0 += kAssignThreads) {
        const int b = b0 + tid;
        int cached = 0, fresh = 0, end = 0;
        if (b < p.B) {
            cached = p.cached_lens[b];
            fresh = p.new_lens[b];
            // a length that the table cannot hold is cut, and reported; the
            // tokens cut off keep their place among the slots
            if (cached < 0 || cached > cap || fresh < 0 || fresh > cap - cached) bad = true;
            cached = (int)min(max((long long)cached, 0LL), cap);
            fresh = max(fresh, 0);
            end = cached + (int)min((long long)fresh, cap - cached);
        }
        const int before = pages_of(cached), need = pages_of(end) - before;
        long long tok = fresh, pg = need, ttok, tpg;
        block_scan2(tok, pg, ttok, tpg, red);
        tok += tokens;
        pg += pages;
        cu_s[tid] = (int)min(tok, (long long)p.total_new);
        cached_s[tid] = cached;
        end_s[tid] = end;
        base_s[tid] = pg;
        if (tid == 0) cu_s[min(p.B - b0, kAssignThreads)] = (int)min(tokens + ttok, (long long)p.total_new);
        if (b < p.B) {
            p.cu_new[b] = cu_s[tid];
            p.seq_lens[b] = end;
            for (int i = 0; i < need; ++i) {
                const long long at = head + pg + i;
                if (at >= p.num_free) out_of_pages = true;
                p.page_table[(size_t)b * p.max_pages + before + i] = at < p.num_free ? p.free_pages[at] : -1;
            }
        }
        __syncthreads();
        const int n = min(p.B - b0, kAssignThreads);
        const int t0 = cu_s[0], t1 = cu_s[n];
        for (int t = t0 + tid; t < t1; t += kAssignThreads) {
            int lo = 0, hi = n;  // the last sequence with cu <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (cu_s[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int c = cached_s[lo];
            const long long pos = (long long)c + t - cu_s[lo];
            const int j = (int)(pos / kTile), first = pages_of(c);
            int page;
            if (pos >= end_s[lo]) {
                page = -1;
            } else if (j < first) {
                page = p.page_table[(size_t)(b0 + lo) * p.max_pages + j];
            } else {
                const long long at = head + base_s[lo] + j - first;
                page = at < p.num_free ? p.free_pages[at] : -1;
            }
            p.slots[t] = page < 0 ? -1 : (int64_t)page * kTile + (int)(pos % kTile);
        }
        tokens += ttok;
        pages += tpg;
        __syncthreads();
    }
    if (tokens > p.total_new) bad = true;
    for (long long t = tokens + tid; t < p.total_new; t += kAssignThreads) p.slots[t] = -1;
    __syncthreads();  // free_head is read (B = 0 passes no barrier above)
    if (tid == 0) {
        p.cu_new[p.B] = (int)min(tokens, (long long)p.total_new);
        p.free_head_out[0] = (int)min(head + pages, (long long)p.num_free);
    }
    if (bad) atomicOr(&g_status_pages, kStatusBadSeqLen);
    if (out_of_pages) atomicOr(&g_status_pages, kStatusOutOfPages);
}

struct AppendParams {
    const uint16_t* k;
    const uint16_t* v;
    long long k_stride, v_stride;
    const int64_t* slots;
    int T, Hkv, num_pages;
    void* k_pages;
    void* v_pages;
    float* k_scales;
    float* v_scales;
};

// Row of (slot, head) in the pools, or -1 for a slot that is not written.
__device__ __forceinline__ long long pool_row(const AppendParams& p, int t, int h) {
    const long long s = p.slots[t];
    if (s < 0) return -1;
    if (s >= (long long)p.num_pages * kTile) {
        atomicOr(&g_status_pages, kStatusBadPage);
        return -1;
    }
    return (s / kTile * p.Hkv + h) * kTile + s % kTile;
}

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    constexpr int C = D / 8;  // 16-byte chunks of a row
    pdl_wait_primary();
    pdl_launch_dependents();
    const long long n = (long long)p.T * p.Hkv * C;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const int c = (int)(i % C);
        const int h = (int)(i / C % p.Hkv), t = (int)(i / C / p.Hkv);
        const long long row = pool_row(p, t, h);
        if (row < 0) continue;
        const uint4 kk = *reinterpret_cast<const uint4*>(p.k + (size_t)t * p.k_stride + (size_t)h * D + c * 8);
        const uint4 vv = *reinterpret_cast<const uint4*>(p.v + (size_t)t * p.v_stride + (size_t)h * D + c * 8);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k_pages) + row * D + c * 8) = kk;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_pages) + row * D + c * 8) = vv;
    }
}

// Two fp32 -> two e4m3 codes (round to nearest even, saturating), `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u16 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// The row as fd_quantize_kv_fp8 encodes it: s = max |x| / 448, codes e4m3(x / s)
// (binary32 divisions, so that both write the same bytes).  The row's D / 8
// lanes hold 8 channels each.
template <int D>
__device__ __forceinline__ void encode_row(const uint16_t* x, uint8_t* codes, float* scale, bool live, int c) {
    constexpr int C = D / 8;
    const uint4 w = live ? *reinterpret_cast<const uint4*>(x + c * 8) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    float2 f[4];
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[e] = bf16x2_to_float2(ws[e]);
        amax = fmaxf(amax, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
    }
#pragma unroll
    for (int o = C / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax / 448.0f;
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t pair = s != 0.f ? e4m3_pair(f[e].x / s, f[e].y / s) : 0u;
        out[e >> 1] |= pair << (16 * (e & 1));
    }
    if (!live) return;
    *reinterpret_cast<uint2*>(codes + c * 8) = make_uint2(out[0], out[1]);
    if (c == 0) *scale = s;
}

template <int D>
__global__ void __launch_bounds__(256) append_fp8_kernel(const AppendParams p) {
    constexpr int C = D / 8;
    pdl_wait_primary();
    pdl_launch_dependents();
    const long long n = (long long)p.T * p.Hkv * C;
    const long long step = (long long)gridDim.x * 256;
    // every lane of a warp runs the same rounds: the shuffles need them all
    for (long long i0 = (long long)blockIdx.x * 256 + (threadIdx.x & ~31); i0 < n; i0 += step) {
        const long long i = i0 + (threadIdx.x & 31);
        const int c = (int)(i % C);
        const int h = (int)(i / C % p.Hkv), t = (int)(i / C / p.Hkv);
        const long long row = i < n ? pool_row(p, t, h) : -1;
        encode_row<D>(p.k + (size_t)t * p.k_stride + (size_t)h * D, static_cast<uint8_t*>(p.k_pages) + row * D,
                      p.k_scales + row, row >= 0, c);
        encode_row<D>(p.v + (size_t)t * p.v_stride + (size_t)h * D, static_cast<uint8_t*>(p.v_pages) + row * D,
                      p.v_scales + row, row >= 0, c);
    }
}

AppendParams append_params(const AppendArgs& a) {
    return AppendParams{static_cast<const uint16_t*>(a.k), static_cast<const uint16_t*>(a.v), a.k_stride, a.v_stride,
                        a.slots, a.T, a.Hkv, a.num_pages, a.k_pages, a.v_pages, a.k_scales, a.v_scales};
}

// Blocks of 256 threads for n pieces of work: all of them while they are few,
// else eight per SM in turn.
cudaError_t append_grid(long long n, unsigned* grid) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long want = (n + 255) / 256, most = (long long)sms * 8;
    *grid = (unsigned)(want < most ? want : most);
    return e;
}

}  // namespace

cudaError_t launch_assign(const AssignArgs& a, cudaStream_t stream) {
    AssignParams p{a.cached_lens, a.new_lens, a.B, a.page_table, a.max_pages, a.free_pages, a.num_free, a.free_head,
                   a.total_new, a.seq_lens, a.cu_new, a.slots, a.free_head_out};
    return launch_pdl(assign_kernel, dim3(1), dim3(kAssignThreads), 0, stream, p);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    unsigned grid = 0;
    const cudaError_t e = append_grid((long long)a.T * a.Hkv * (a.D / 8), &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(a.D == 128 ? append_kernel<128> : append_kernel<64>, dim3(grid), dim3(256), 0, stream,
                      append_params(a));
}

cudaError_t launch_append_fp8(const AppendArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    unsigned grid = 0;
    const cudaError_t e = append_grid((long long)a.T * a.Hkv * (a.D / 8), &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(a.D == 128 ? append_fp8_kernel<128> : append_fp8_kernel<64>, dim3(grid), dim3(256), 0, stream,
                      append_params(a));
}

cudaError_t pages_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_pages, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_pages, &zero, sizeof(unsigned));
}

}  // namespace fd
