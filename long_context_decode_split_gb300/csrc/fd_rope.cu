// fd_rope.cu -- norms and rotation of query and key heads by position for
// sm_103a, and the same on the way into the paged cache (bf16, or e4m3 codes with
// a scale per row), the values beside them.
//
// For a head x of n channels at position t:
//   y = x / sqrt(mean(x^2) + eps) * w               (with a weight; else y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the pairs (a, b) of the
//   first `rot` channels, cos and sin from row t of a table
// in binary32, rounded once: to bf16, or to the e4m3 codes.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "fd_device.cuh"
#include "fd_encode.cuh"
#include "fd_internal.h"

namespace fd {

__device__ unsigned int g_status_rope;

namespace {

// HBM bounds the large calls: 20.5K tokens of 32 + 8 heads of 128 with norms in 67-70 us (6.0-6.3 TB/s, rows read
// and written), 31K tokens of them into the e4m3 cache in 116-119 us (6.0-6.1 TB/s).  What counts is the bytes that
// an SM has on their way: the chain behind a row (position, its angles) takes longer than the row itself.
// Four rows a thread and six blocks of 128 threads an SM (80 registers, of which these forms spill 40 to 76 bytes)
// measured best, where the kept one took 66.5 and 116: two rows 68.5 and 122 us, four in three blocks of 256 69.6
// and 127 us, one in four of 256 91 and 168 us.
constexpr int kThreads = 128, kBlocksPerSM = 6;

// The token's sequence: the last s with cu[s] <= t.  All lanes together; each round every lane
// probes one of 32 places.
__device__ __forceinline__ int sequence_of(const RopeArgs& p, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool below = lane * step < n && p.cu[lo + lane * step] <= t;
        const unsigned votes = __ballot_sync(0xffffffffu, below);
        const int hit = votes ? 31 - __clz(votes) : 0;
        lo += hit * step;
        n = min(step, n - hit * step);
    }
    return lo;
}

// Row of the table for token t, -1 for a token that is left out.  All lanes together; the
// tokens of a warp ascend.
__device__ __forceinline__ int row_of(const RopeArgs& p, int t) {
    long long pos;
    if (p.positions) {
        pos = p.positions[t];
        if (pos < 0) return -1;
    } else {
        if (p.B == 0) return -1;
        const int t0 = __shfl_sync(0xffffffffu, t, 0), t1 = __shfl_sync(0xffffffffu, t, 31);
        int s = 0;
        for (int x = t0; x <= t1; ++x) {
            const int found = sequence_of(p, x);
            if (x == t) s = found;
        }
        const int a = p.cu[s], b = p.cu[s + 1];
        if (t < a || t >= b) return -1;
        pos = (long long)p.lens[s] - b + t;
    }
    if (pos < 0 || pos >= p.max_pos) {
        atomicOr(&g_status_rope, kStatusBadSeqLen);
        pos = pos < 0 ? 0 : p.max_pos - 1;
    }
    return (int)pos;
}

// Reports offsets that run backwards or out of [0, T], those between which no token lies too.  Blocks of their own: within
// the others the test cost the e4m3 append registers (118 -> 123 us).
__device__ __forceinline__ void check_offsets(const RopeArgs& p, unsigned block, unsigned blocks) {
    for (long long s = (long long)block * kThreads + threadIdx.x; s < p.B; s += (long long)blocks * kThreads) {
        const int a = p.cu[s], b = p.cu[s + 1];
        if (a < 0 || a > b || b > p.T) atomicOr(&g_status_rope, kStatusBadSeqLen);
    }
}

// The 16 channels of a row that a lane holds: two runs of 8, which pair with each other (halves of
// the rotated part), or the pairs within them (neighbours).  Lane j of the DH / 16 of a head.
struct Lane {
    int at0, at1;  // channels within the head
    bool turns;    // they are rotated, by the angles 8j .. 8j + 7
    int j;
};
template <int DH>
__device__ __forceinline__ Lane lane_of(const RopeArgs& p, int j) {
    Lane l;
    const int np = p.rot / 16;
    l.j = j;
    l.turns = j < np;
    const bool apart = l.turns && !p.interleaved;
    l.at0 = apart ? 8 * j : 16 * j;
    l.at1 = apart ? p.rot / 2 + 8 * j : 16 * j + 8;
    return l;
}

struct Angles {
    float2 c[4], s[4];
};
__device__ __forceinline__ void load8(float2* f, const float* at) {
    const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void load_angles(Angles& a, const RopeArgs& p, const Lane& l, int row) {
    if (!l.turns || row < 0) return;  // not used
    const float* at = p.cos_sin + (size_t)row * p.rot + 8 * l.j;
    load8(a.c, at);
    load8(a.s, at + p.rot / 2);
}

// The lane's weights of the norm.
struct Weights {
    float2 w[8];
};
__device__ __forceinline__ void load_weights(Weights& w, const float* from, const Lane& l) {
    load8(w.w, from + l.at0);
    load8(w.w + 4, from + l.at1);
}

// Norm (NORM) and rotation of the head whose channels the DH / 16 lanes hold as bf16 (all lanes together).  Whether
// the head's squares leave binary32, as they do from 2^60 on: x is then worthless.  LARGE: such a head, and sqrt(eps) with
// it, by 2^-96 before its norm, in range whatever it is.
template <int DH, bool NORM, bool LARGE>
__device__ __forceinline__ bool turn(float (&x)[16], const uint4& a, const uint4& b, const RopeArgs& p, const Lane& l,
                                     const Angles& g, const Weights& w) {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float2 y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = bf16x2_to_float2(u[e]);
    bool large = false;
    if (NORM) {
        const auto squares = [&] {
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = f2fma(y[e], y[e], sum);
            float all = sum.x + sum.y;
#pragma unroll
            for (int o = DH / 32; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            return all;
        };
        float all = squares(), eps = p.eps;
        large = all == INFINITY;
        if (LARGE) {
            const float by = large ? 0x1p-96f : 1.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = f2mul(y[e], make_float2(by, by));
            eps = eps * by * by;
            all = squares();
        }
        const float r = rsqrtf(all * (1.f / DH) + eps);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = f2mul(f2mul(y[e], r2), w.w[e]);
    }
    if (l.turns && p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = e & 1 ? g.c[e / 2].y : g.c[e / 2].x, s = e & 1 ? g.s[e / 2].y : g.s[e / 2].x;
            y[e] = make_float2(y[e].x * c - y[e].y * s, y[e].y * c + y[e].x * s);
        }
    } else if (l.turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y0 = y[e], y1 = y[4 + e], minus = make_float2(-y1.x, -y1.y);
            y[e] = f2fma(minus, g.s[e], f2mul(y0, g.c[e]));
            y[4 + e] = f2fma(y0, g.s[e], f2mul(y1, g.c[e]));
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[2 * e] = y[e].x;
        x[2 * e + 1] = y[e].y;
    }
    return large;
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Rows of one operand to rows: heads hg, hg + groups, .. of token t (all lanes together).  Returns which of the lane's
// RPT rows are left, not yet written, for the LARGE form: one row, the one `from` heads on, where `wanted`.  (A branch to
// it within the rows made the call 5% slower.)
template <int D, int DH, int RPT, bool NORM, bool LARGE = false>
__device__ __forceinline__ unsigned rows_to_rows(const RopeArgs& p, const uint16_t* in, long long stride, uint16_t* out,
                                                 long long out_stride, const float* weight, int H, int groups,
                                                 unsigned block, int from = 0, bool wanted = true) {
    constexpr int C = D / 16;  // lanes of a row
    const int c = threadIdx.x % C;
    const unsigned item = block * (kThreads / C) + threadIdx.x / C;
    const unsigned at_t = item / (unsigned)groups;
    const bool in_range = at_t < (unsigned)p.T;
    const int t = in_range ? (int)at_t : p.T - 1;
    const int hg = from + (int)(item - at_t * groups);
    const Lane l = lane_of<DH>(p, c % (DH / 16));
    const int part = c / (DH / 16) * DH;
    const uint16_t* row = in + (size_t)t * stride + hg * D + part;
    uint4 a[RPT], b[RPT];
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int h = u * groups;
        if (in_range && hg + h < H) {
            a[u] = *reinterpret_cast<const uint4*>(row + h * D + l.at0);
            b[u] = *reinterpret_cast<const uint4*>(row + h * D + l.at1);
        } else {
            a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    Weights w;
    if (NORM) load_weights(w, weight, l);
    const int at = row_of(p, t);
    Angles g = {};
    load_angles(g, p, l, at);
    unsigned left = 0;
    uint16_t* to = out + (size_t)t * out_stride + hg * D + part;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int h = u * groups;
        float x[16];
        const bool large = turn<DH, NORM, LARGE>(x, a[u], b[u], p, l, g, w);
        if (!wanted || !in_range || at < 0 || hg + h >= H) continue;
        if (!LARGE && large) {
            left |= 1u << u;
            continue;
        }
        *reinterpret_cast<uint4*>(to + h * D + l.at0) = pack8(x);
        *reinterpret_cast<uint4*>(to + h * D + l.at1) = pack8(x + 8);
    }
    return left;
}

// Key rows of a token, turned, and its value rows to their slot of the pools: heads hg, hg + groups,
// .. (all lanes together).  Returns which of the lane's key rows are left for the LARGE form: heads as above, e4m3
// rows that have to be divided too.  That form writes no values.  (Its code in a branch within the rows cost nothing in
// a loop and 3% beside cold caches: 31K tokens 153.5 us instead of 149.)
template <int D, int DH, int RPT, bool FP8, bool NORM, bool LARGE = false>
__device__ __forceinline__ unsigned rows_to_pages(const RopeArgs& p, int groups, unsigned block, int from = 0,
                                                  bool mine = true) {
    constexpr int C = D / 16;
    const int c = threadIdx.x % C;
    const unsigned item = block * (kThreads / C) + threadIdx.x / C;
    const unsigned at_t = item / (unsigned)groups;
    const bool in_range = at_t < (unsigned)p.T;
    const int t = in_range ? (int)at_t : p.T - 1;
    const int hg = from + (int)(item - at_t * groups);
    const Lane l = lane_of<DH>(p, c % (DH / 16));
    const int part = c / (DH / 16) * DH;
    const long long slot = p.slots[t];
    const uint16_t* kr = p.k + (size_t)t * p.k_stride + hg * D + part;
    const uint16_t* vr = p.v + (size_t)t * p.v_stride + hg * D + c * 16;
    uint4 a[RPT], b[RPT], v0[RPT], v1[RPT];
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int h = u * groups;
        if (in_range && hg + h < p.Hkv) {
            a[u] = *reinterpret_cast<const uint4*>(kr + h * D + l.at0);
            b[u] = *reinterpret_cast<const uint4*>(kr + h * D + l.at1);
            if (!LARGE) {
                v0[u] = reinterpret_cast<const uint4*>(vr + h * D)[0];
                v1[u] = reinterpret_cast<const uint4*>(vr + h * D)[1];
            }
        } else {
            a[u] = b[u] = v0[u] = v1[u] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const int at = row_of(p, t);
    bool live = in_range && at >= 0 && slot >= 0;
    if (live && slot >= (long long)p.num_pages * kTile) {
        atomicOr(&g_status_rope, kStatusBadPage);
        live = false;
    }
    Weights w;
    if (NORM) load_weights(w, p.k_weight, l);
    Angles g = {};
    load_angles(g, p, l, at);
    const size_t row0 = live ? (size_t)((slot / kTile * p.Hkv + hg) * kTile + slot % kTile) : 0;
    // the values first: they wait for no angles
#pragma unroll
    for (int u = 0; u < (LARGE ? 0 : RPT); ++u) {
        const bool wanted = live && hg + u * groups < p.Hkv;
        const size_t row = row0 + (size_t)u * groups * kTile;
        if constexpr (FP8) {
            const uint32_t v[8] = {v0[u].x, v0[u].y, v0[u].z, v0[u].w, v1[u].x, v1[u].y, v1[u].z, v1[u].w};
            encode_row<C>(v, static_cast<uint8_t*>(p.v_pages) + row * D, p.v_scales + row, wanted, c);
        } else if (wanted) {
            uint4* vp = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_pages) + row * D + c * 16);
            vp[0] = v0[u];
            vp[1] = v1[u];
        }
    }
    unsigned left = 0;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const bool wanted = mine && live && hg + u * groups < p.Hkv;
        const size_t row = row0 + (size_t)u * groups * kTile;
        float x[16];
        bool later = turn<DH, NORM, LARGE>(x, a[u], b[u], p, l, g, w);
        if constexpr (FP8) {
            later = encode_floats<C, LARGE>(x, later, static_cast<uint8_t*>(p.k_pages) + row * D, p.k_scales + row,
                                            wanted, c, part + l.at0, part + l.at1);
        } else if (wanted) {  // (what a large head leaves there is written over)
            uint16_t* kp = static_cast<uint16_t*>(p.k_pages) + row * D + part;
            *reinterpret_cast<uint4*>(kp + l.at0) = pack8(x);
            *reinterpret_cast<uint4*>(kp + l.at1) = pack8(x + 8);
        }
        if (!LARGE && later) left |= 1u << u;
    }
    return left;
}

enum { kToRows, kToPages, kToPagesFp8 };

// The first q_blocks blocks take the queries, the others of work_blocks the keys (and values), any behind them the
// offsets; RPT rows a thread, on the way to pages RPP keys and their values.
template <int D, int DH, int TO, int RPT, int RPP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM)
rope_kernel(const RopeArgs p, unsigned q_blocks, int q_groups, int k_groups, unsigned work_blocks) {
    pdl_wait_primary();
    pdl_launch_dependents();
    if (blockIdx.x >= work_blocks) {
        check_offsets(p, blockIdx.x - work_blocks, gridDim.x - work_blocks);
        return;
    }
    // the rows of an operand, then those with squares that left binary32
    const auto to_rows = [&](auto norm, const uint16_t* in, long long stride, uint16_t* out, long long out_stride,
                             const float* weight, int H, int groups, unsigned block) {
        constexpr bool NORM = decltype(norm)::value;
        unsigned left = rows_to_rows<D, DH, RPT, NORM>(p, in, stride, out, out_stride, weight, H, groups, block);
        if constexpr (NORM) {
            if (__any_sync(0xffffffffu, left != 0u)) {
#pragma unroll 1
                for (int u = 0; u < RPT; ++u, left >>= 1)
                    rows_to_rows<D, DH, 1, true, true>(p, in, stride, out, out_stride, weight, H, groups, block, u * groups,
                                                       left & 1u);
            }
        }
    };
    const std::true_type with_norm;
    const std::false_type without;
    if (blockIdx.x < q_blocks) {
        if (p.q_weight) to_rows(with_norm, p.q, p.q_stride, p.q_out, p.q_out_stride, p.q_weight, p.Hq, q_groups, blockIdx.x);
        else to_rows(without, p.q, p.q_stride, p.q_out, p.q_out_stride, nullptr, p.Hq, q_groups, blockIdx.x);
        return;
    }
    const unsigned block = blockIdx.x - q_blocks;
    if constexpr (TO == kToRows) {
        if (p.k_weight) to_rows(with_norm, p.k, p.k_stride, p.k_out, p.k_out_stride, p.k_weight, p.Hkv, k_groups, block);
        else to_rows(without, p.k, p.k_stride, p.k_out, p.k_out_stride, nullptr, p.Hkv, k_groups, block);
    } else {
        constexpr bool FP8 = TO == kToPagesFp8;
        const auto to_pages = [&](auto norm) {
            constexpr bool NORM = decltype(norm)::value;
            unsigned left = rows_to_pages<D, DH, RPP, FP8, NORM>(p, k_groups, block);
            if ((FP8 || NORM) && __any_sync(0xffffffffu, left != 0u)) {
#pragma unroll 1
                for (int u = 0; u < RPP; ++u, left >>= 1)
                    rows_to_pages<D, DH, 1, FP8, NORM, true>(p, k_groups, block, u * k_groups, left & 1u);
            }
        };
        if (p.k_weight) to_pages(with_norm);
        else to_pages(without);
    }
}

template <int D, int DH, int RPT, int RPP>
cudaError_t launch(const RopeArgs& p, cudaStream_t stream) {
    const int qg = (p.Hq + RPT - 1) / RPT, kr = p.slots ? RPP : RPT, kg = (p.Hkv + kr - 1) / kr;
    const auto blocks = [&](int groups) { return ((long long)p.T * groups * (D / 16) + kThreads - 1) / kThreads; };
    const unsigned qb = (unsigned)blocks(qg);
    const unsigned work = (unsigned)(qb + blocks(kg));
    const dim3 grid(work + (p.positions ? 0u : (unsigned)std::min(((long long)p.B + kThreads - 1) / kThreads, 32LL)));
    const auto kernel = !p.slots      ? rope_kernel<D, DH, kToRows, RPT, RPP>
                        : p.k_scales ? rope_kernel<D, DH, kToPagesFp8, RPT, RPP>
                                     : rope_kernel<D, DH, kToPages, RPT, RPP>;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, p, qb, qg, kg, work);
}

// One row a thread while all of them are on the GPU at once: more rows then only make each thread's chain
// longer (30 rows of three tokens 1.5-1.65 us, 2.07 us with four a thread).
template <int D, int DH>
cudaError_t launch_for(const RopeArgs& p, cudaStream_t stream) {
    int sms = 0, dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long threads = (long long)p.T * (p.Hq + p.Hkv) * (D / 16);
    return threads <= (long long)sms * kBlocksPerSM * kThreads ? launch<D, DH, 1, 1>(p, stream)
                                                               : launch<D, DH, 4, 2>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& p, cudaStream_t stream) {
    if (p.T == 0 || p.Hq + p.Hkv == 0) return cudaSuccess;
    if (p.D == 128) return p.halves ? launch_for<128, 64>(p, stream) : launch_for<128, 128>(p, stream);
    return p.halves ? launch_for<64, 32>(p, stream) : launch_for<64, 64>(p, stream);
}

cudaError_t rope_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_rope, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_rope, &zero, sizeof(unsigned));
}

}  // namespace fd
