// fd_encode.cuh -- e4m3 codes of cache rows on their way into the fp8 cache:
// rows as they come (fd_pages.cu), and rows that were normalised or rotated in
// binary32 before (fd_rope.cu).
#pragma once

#include "fd_device.cuh"

namespace fd {

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

// The row as fd_quantize_kv_fp8 encodes it (the same bytes): s = max |x| / 448,
// codes e4m3(x / s) of the correctly rounded binary32 quotient.  With r = 1 / s
// correctly rounded, q0 = x r and the exact remainder x - q0 s (one fused
// multiply-add), q0 + (x - q0 s) r is that quotient (Markstein's theorem; it
// needs s and 1 / s away from the ends of the range, other rows are divided).
// The kernel carries -q, whose remainder steps keep the sign of a zero, and
// flips the codes' signs.  The maximum skips NaN, as the encoder's does (finite
// scale, NaN codes where the NaNs are); a lane that holds one divides, since a
// flipped sign would show in the NaN's code (the whole test moved into the dividing
// branch: 31.3 us).  C lanes hold a row, 16 channels each: with 8 the pass was bound
// by its instructions (77 us against the 29 us that the bytes of 31K tokens x 8
// heads x 128 need).
template <int C>
__device__ __forceinline__ void encode_row(const uint32_t (&w)[8], uint8_t* codes, float* scale, bool live, int c) {
    // magnitudes of bf16 order like unsigned integers
    uint32_t top = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int e = 1; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    const bool has_nan = __vcmpgtu2(top, 0x7f807f80u) != 0u;
    if (has_nan) {
        top = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t x = w[e] & 0x7fff7fffu;
            top = __vmaxu2(top, x & ~__vcmpgtu2(x, 0x7f807f80u));
        }
    }
#pragma unroll
    for (int o = C / 2; o >= 1; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float amax = __uint_as_float(max(top << 16, top & 0xffff0000u));
    const float s = amax / 448.0f;
    uint32_t out[4];
    if (s > 1e-30f && s < 1e30f && !has_nan) {
        const float r = 1.0f / s;
        const float2 s2 = make_float2(s, s), nr2 = make_float2(-r, -r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = bf16x2_to_float2(w[e]);
            float2 n = f2mul(x, nr2);
            n = f2fma(f2fma(n, s2, x), nr2, n);
            const uint32_t pair = e4m3_pair(n.x, n.y);
            out[e >> 1] = e & 1 ? (out[e >> 1] | pair << 16) ^ 0x80808080u : pair;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = bf16x2_to_float2(w[e]);
            const uint32_t pair = s != 0.f ? e4m3_pair(x.x / s, x.y / s) : 0u;
            out[e >> 1] = e & 1 ? out[e >> 1] | pair << 16 : pair;
        }
    }
    if (!live) return;
    *reinterpret_cast<uint4*>(codes + c * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    if (c == 0) *scale = s;
}

// The same for a row in binary32 (rotated and not yet rounded): one rounding,
// from these values to the codes.  The lane's 16 channels lie in two runs of 8 at
// `at0` and `at1` of the row.  (A NaN's code is NaN with either sign; a row of nothing
// but NaN gets the scale NaN.)  Returns, the same to the row's lanes, whether the row is
// left for the EXACT form, which divides: its scale is near the ends of the range, or
// a lane's x is `worthless`.
template <int C, bool EXACT>
__device__ __forceinline__ bool encode_floats(const float (&x)[16], bool worthless, uint8_t* codes, float* scale,
                                              bool live, int c, int at0, int at1) {
    float amax = !EXACT && worthless ? INFINITY : fabsf(x[0]);
#pragma unroll
    for (int e = 1; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
    for (int o = C / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax / 448.0f;
    if (!EXACT && !(s > 1e-30f && s < 1e30f)) return live;
    uint32_t out[4];
    if constexpr (!EXACT) {
        const float r = 1.0f / s;
        const float2 s2 = make_float2(s, s), nr2 = make_float2(-r, -r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 y = make_float2(x[2 * e], x[2 * e + 1]);
            float2 n = f2mul(y, nr2);
            n = f2fma(f2fma(n, s2, y), nr2, n);
            const uint32_t pair = e4m3_pair(n.x, n.y);
            out[e >> 1] = e & 1 ? (out[e >> 1] | pair << 16) ^ 0x80808080u : pair;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t pair = s != 0.f ? e4m3_pair(x[2 * e] / s, x[2 * e + 1] / s) : 0u;
            out[e >> 1] = e & 1 ? out[e >> 1] | pair << 16 : pair;
        }
    }
    if (!live) return false;
    *reinterpret_cast<uint2*>(codes + at0) = make_uint2(out[0], out[1]);
    *reinterpret_cast<uint2*>(codes + at1) = make_uint2(out[2], out[3]);
    if (c == 0) *scale = s;
    return false;
}

}  // namespace fd
