// fd_rope.cu -- norms and rotation of query and key heads by position for
// sm_103a, and the same on the way into the paged cache (bf16, or e4m3 codes with
// a scale per row), the values beside them.
//
// For a head x of n channels at position t:
//   y = x / sqrt(mean(x^2) + eps) * w               (with a weight; else y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the pairs (a, b) of the
//   first `rot` channels, cos and sin from row t of a table
// in binary32, rounded once: to bf16, or to the e4m3 codes.
#include <cstdint>

#include "fd_device.cuh"
#include "fd_encode.cuh"
#include "fd_internal.h"

namespace fd {

__device__ unsigned int g_status_rope;

namespace {

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
        if (a < 0 || a > b || b > p.T) atomicOr(&g_status_rope, kStatusBadSeqLen);
        if (t < a || t >= b) return -1;
        pos = (long long)p.lens[s] - b + t;
    }
    if (pos < 0 || pos >= p.max_pos) {
        atomicOr(&g_status_rope, kStatusBadSeqLen);
        pos = pos < 0 ? 0 : p.max_pos - 1;
    }
    return (int)pos;
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
    float c[8], s[8];
};
__device__ __forceinline__ void load8(float (&f)[8], const float* at) {
    const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load_angles(Angles& a, const RopeArgs& p, const Lane& l, int row) {
    if (l.turns && row >= 0) {
        const float* at = p.cos_sin + (size_t)row * p.rot + 8 * l.j;
        load8(a.c, at);
        load8(a.s, at + p.rot / 2);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a.c[e] = 1.f, a.s[e] = 0.f;
    }
}

// Norm and rotation of the head whose channels the DH / 16 lanes hold as bf16.
template <int DH>
__device__ __forceinline__ void turn(float (&x)[16], const uint4& a, const uint4& b, const RopeArgs& p, const Lane& l,
                                     const Angles& g, const float* w) {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 f = bf16x2_to_float2(u[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
    if (w) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int o = DH / 32; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum * (1.f / DH) + p.eps);
        float w0[8], w1[8];
        load8(w0, w + l.at0);
        load8(w1, w + l.at1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] *= r * w0[e];
            x[8 + e] *= r * w1[e];
        }
    }
    if (!l.turns) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (p.interleaved) {
            const float y0 = x[2 * e], y1 = x[2 * e + 1];
            x[2 * e] = y0 * g.c[e] - y1 * g.s[e];
            x[2 * e + 1] = y1 * g.c[e] + y0 * g.s[e];
        } else {
            const float y0 = x[e], y1 = x[8 + e];
            x[e] = y0 * g.c[e] - y1 * g.s[e];
            x[8 + e] = y1 * g.c[e] + y0 * g.s[e];
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Rows of one operand to rows: heads hg, hg + groups, .. of token t (all lanes together).
template <int D, int DH, int RPT>
__device__ __forceinline__ void rows_to_rows(const RopeArgs& p, const uint16_t* in, long long stride, uint16_t* out,
                                             long long out_stride, const float* w, int H, int groups, long long i) {
    constexpr int C = D / 16;  // lanes of a row
    const int c = (int)(i % C);
    const long long item = i / C;
    const bool in_range = item < (long long)p.T * groups;
    const int t = in_range ? (int)(item / groups) : p.T - 1;
    const int hg = in_range ? (int)(item - (long long)t * groups) : 0;
    const Lane l = lane_of<DH>(p, c % (DH / 16));
    const int part = c / (DH / 16) * DH;
    const uint16_t* row = in + (size_t)t * stride + part;
    uint4 a[RPT], b[RPT];
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int h = hg + u * groups;
        if (in_range && h < H) {
            a[u] = *reinterpret_cast<const uint4*>(row + (size_t)h * D + l.at0);
            b[u] = *reinterpret_cast<const uint4*>(row + (size_t)h * D + l.at1);
        } else {
            a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const int at = row_of(p, t);
    Angles g;
    load_angles(g, p, l, at);
    uint16_t* to = out + (size_t)t * out_stride + part;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int h = hg + u * groups;
        float x[16];
        turn<DH>(x, a[u], b[u], p, l, g, w);
        if (!in_range || at < 0 || h >= H) continue;
        *reinterpret_cast<uint4*>(to + (size_t)h * D + l.at0) = pack8(x);
        *reinterpret_cast<uint4*>(to + (size_t)h * D + l.at1) = pack8(x + 8);
    }
}

// A token's key row, turned, and value row to their slot of the pools (all lanes together).
template <int D, int DH, bool FP8>
__device__ __forceinline__ void rows_to_pages(const RopeArgs& p, long long i) {
    constexpr int C = D / 16;
    const int c = (int)(i % C);
    const long long item = i / C;
    const bool in_range = item < (long long)p.T * p.Hkv;
    const int t = in_range ? (int)(item / p.Hkv) : p.T - 1;
    const int h = in_range ? (int)(item - (long long)t * p.Hkv) : 0;
    const Lane l = lane_of<DH>(p, c % (DH / 16));
    const int part = c / (DH / 16) * DH;
    const long long slot = p.slots[t];
    const uint16_t* kr = p.k + (size_t)t * p.k_stride + (size_t)h * D + part;
    const uint16_t* vr = p.v + (size_t)t * p.v_stride + (size_t)h * D + c * 16;
    const uint4 a = *reinterpret_cast<const uint4*>(kr + l.at0), b = *reinterpret_cast<const uint4*>(kr + l.at1);
    const uint4 v0 = reinterpret_cast<const uint4*>(vr)[0], v1 = reinterpret_cast<const uint4*>(vr)[1];
    const int at = row_of(p, t);
    Angles g;
    load_angles(g, p, l, at);
    bool live = in_range && at >= 0 && slot >= 0;
    if (live && slot >= (long long)p.num_pages * kTile) {
        atomicOr(&g_status_rope, kStatusBadPage);
        live = false;
    }
    const size_t row = live ? (size_t)((slot / kTile * p.Hkv + h) * kTile + slot % kTile) : 0;
    float x[16];
    turn<DH>(x, a, b, p, l, g, p.k_weight);
    if constexpr (FP8) {
        const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        encode_floats<C>(x, static_cast<uint8_t*>(p.k_pages) + row * D, p.k_scales + row, live, c, part + l.at0,
                         part + l.at1);
        encode_row<C>(v, static_cast<uint8_t*>(p.v_pages) + row * D, p.v_scales + row, live, c);
    } else {
        if (!live) return;
        uint16_t* kp = static_cast<uint16_t*>(p.k_pages) + row * D + part;
        *reinterpret_cast<uint4*>(kp + l.at0) = pack8(x);
        *reinterpret_cast<uint4*>(kp + l.at1) = pack8(x + 8);
        uint4* vp = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_pages) + row * D + c * 16);
        vp[0] = v0;
        vp[1] = v1;
    }
}

enum { kToRows, kToPages, kToPagesFp8 };

// The first q_blocks blocks take the queries, RPT heads a thread, the others the keys (and values).
template <int D, int DH, int TO, int RPT>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs p, unsigned q_blocks, int q_groups, int k_groups) {
    pdl_wait_primary();
    pdl_launch_dependents();
    if (blockIdx.x < q_blocks) {
        rows_to_rows<D, DH, RPT>(p, p.q, p.q_stride, p.q_out, p.q_out_stride, p.q_weight, p.Hq, q_groups,
                                 (long long)blockIdx.x * 256 + threadIdx.x);
        return;
    }
    const long long i = (long long)(blockIdx.x - q_blocks) * 256 + threadIdx.x;
    if constexpr (TO == kToRows)
        rows_to_rows<D, DH, RPT>(p, p.k, p.k_stride, p.k_out, p.k_out_stride, p.k_weight, p.Hkv, k_groups, i);
    else
        rows_to_pages<D, DH, TO == kToPagesFp8>(p, i);
}

template <int D, int DH, int RPT>
cudaError_t launch(const RopeArgs& p, cudaStream_t stream) {
    const int qg = (p.Hq + RPT - 1) / RPT, kg = p.k_pages || p.slots ? p.Hkv : (p.Hkv + RPT - 1) / RPT;
    const auto blocks = [&](int groups) { return ((long long)p.T * groups * (D / 16) + 255) / 256; };
    const unsigned qb = (unsigned)blocks(qg);
    const dim3 grid((unsigned)(qb + blocks(kg)));
    const auto kernel = !p.slots      ? rope_kernel<D, DH, kToRows, RPT>
                        : p.k_scales ? rope_kernel<D, DH, kToPagesFp8, RPT>
                                     : rope_kernel<D, DH, kToPages, RPT>;
    return launch_pdl(kernel, grid, dim3(256), 0, stream, p, qb, qg, kg);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& p, cudaStream_t stream) {
    if (p.T == 0 || p.Hq + p.Hkv == 0) return cudaSuccess;
    if (p.D == 128) return p.halves ? launch<128, 64, 1>(p, stream) : launch<128, 128, 1>(p, stream);
    return p.halves ? launch<64, 32, 1>(p, stream) : launch<64, 64, 1>(p, stream);
}

cudaError_t rope_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_rope, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_rope, &zero, sizeof(unsigned));
}

}  // namespace fd
