// fd_diff.cu -- differential attention of one new token per sequence for sm_103a:
// the split-KV pass over a contiguous or paged bf16 cache, and the merge of its
// chunks (and of the parts of differential prompts).
//
// A query or key row of d channels is [first half | second half]; with
// s1_j = scale <q1, k1_j>, s2_j = scale <q2, k2_j>:
//   o = softmax(s1) V - lambda softmax(s2) V,   y = o / sqrt(mean(o^2) + eps) * w  (with a weight w)
// Both maps weigh whole value rows, so a KV head's group of G query heads is 2 G
// columns of scores over one pass through the cache: every key and value is read
// once for both maps and the whole group.  The maps' (m, l, O) stay apart up to the
// end, where their difference is taken in binary32.
#include "fd_device.cuh"
#include "fd_internal.h"
#include "fd_tma.h"

namespace fd {

__device__ unsigned int g_status_diff;

namespace {

struct DiffParams {
    const uint16_t* q;
    const int32_t* seq_lens;
    const int32_t* page_table;
    int max_pages, num_pages;
    int Hq, Hkv, L_max, G;
    float scale_log2;
    int splits, chunk_fixed;
    unsigned long long wait_limit_ns;
    int withhold_tile;
    void* out;
    int out_bf16;
    float* lse;
    float* part_o;
    float* part_ml;
    DiffMix mix;
};

// The difference of a head's two maps: E channels a lane, the warp together.  l1, l2: the maps'
// exp-sums (a head that attended nothing gives 0).
template <int D>
__device__ __forceinline__ void store_difference(const float (&o1)[D / 32], const float (&o2)[D / 32], float l1,
                                                 float l2, const DiffMix& mix, int token, int head, size_t row,
                                                 void* out, int out_bf16, int lane) {
    constexpr int E = D / 32;
    const float lambda = mix.lambda[(size_t)token * mix.lambda_stride + head];
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o1[e] - lambda * o2[e];
    if (mix.weight) {
        const auto squares = [&] {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) sum = fmaf(o[e], o[e], sum);
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            return sum;
        };
        float sum = squares(), eps = mix.eps;
        if (sum == INFINITY) {  // (all lanes) from 2^60 on: o and sqrt(eps) by 2^-96 are in range, whatever o is
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= 0x1p-96f;
            eps = eps * 0x1p-96f * 0x1p-96f;
            sum = squares();
        }
        const float r = rsqrtf(sum * (1.f / D) + eps);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= r * mix.weight[lane * E + e];
    }
    if (l1 == 0.f && l2 == 0.f) {
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
    }
    if (out_bf16) {
        uint32_t* at = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + row * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) at[e / 2] = pack_bf16(o[e], o[e + 1]);
    } else {
        float* at = static_cast<float*>(out) + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) at[e] = o[e];
    }
}

__device__ __forceinline__ float natural_lse(float m, float l) {
    return l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

// One tile of a consumer warp: the online softmax of its 16 rows in NB blocks of 8 columns, and
// O^T += V^T P^T with every V fragment loaded once for all of them.  As mma_softmax_pv with NAN_OUT:
// P as bf16 hi + lo, a NaN or +inf score makes its column NaN.
template <int D, int NB>
__device__ __forceinline__ void softmax_pv(TokAcc<D> (&ac)[NB], const float (&sc)[NB][4], uint32_t vs,
                                           unsigned char* vgen, int warp, int lane, int rows) {
    const int mi = lane >> 3;
    const int ld_row = warp * 16 + 8 * (mi >> 1) + (lane & 7);
    if (warp * 16 + 16 > rows) {
        for (int i = lane; i < 16 * (D / 8); i += 32) {
            const int r = warp * 16 + i / (D / 8);
            if (r >= rows) *reinterpret_cast<uint4*>(vgen + swz(r, i % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
    uint32_t h[NB][2], l[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        float2 mx = make_float2(fmaxf(sc[n][0], sc[n][2]), fmaxf(sc[n][1], sc[n][3]));
        mx = column_max(mx);
        const float m0 = fmaxf(ac[n].m.x, mx.x), m1 = fmaxf(ac[n].m.y, mx.y);
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        const float a0 = m0 == -INFINITY ? 1.f : exp2_approx(ac[n].m.x - m0);
        const float a1 = m1 == -INFINITY ? 1.f : exp2_approx(ac[n].m.y - m1);
        float pr[4];
        pr[0] = exp2_approx(sc[n][0] - z0);
        pr[1] = exp2_approx(sc[n][1] - z1);
        pr[2] = exp2_approx(sc[n][2] - z0);
        pr[3] = exp2_approx(sc[n][3] - z1);
        ac[n].m = make_float2(m0, m1);
        ac[n].l.x = ac[n].l.x * a0 + (pr[0] + pr[2]);
        ac[n].l.y = ac[n].l.y * a1 + (pr[1] + pr[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            split_bf16(pr[2 * i], pr[2 * i + 1], h[n][i], l[n][i]);
            h[n][i] = movmatrix_trans(h[n][i]);
            l[n][i] = movmatrix_trans(l[n][i]);
        }
        if (!__all_sync(0xffffffffu, a0 == 1.f && a1 == 1.f)) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                ac[n].o[mt][0] *= a0;
                ac[n].o[mt][1] *= a1;
                ac[n].o[mt][2] *= a0;
                ac[n].o[mt][3] *= a1;
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        uint32_t v0, v1, v2, v3;
        ldsm_x4_t(vs + swz(ld_row, 2 * mt + (mi & 1)), v0, v1, v2, v3);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            mma_bf16(ac[n].o[mt], v0, v1, v2, v3, h[n][0], h[n][1]);
            mma_bf16(ac[n].o[mt], v0, v1, v2, v3, l[n][0], l[n][1]);
        }
    }
}

// One CTA per (chunk, KV head, sequence): a warp streams the chunk's 64-token tiles through a ring
// in shared memory, CW others take 16 rows of each on mma.sync (S = K Q^T, rows are tokens).
//   NB = 1 (groups of up to 4): one block of 8 columns holds both maps, map 0 in the columns
//     0 .. G - 1 and map 1 behind it; a column takes its scores from its half of the key (its query
//     fragments over the other one are zero, but zero times infinity is not)
//   NB = 2 (groups of 5 to 8): a block a map, each over its half of the key: the same number of
//     products for the scores, twice those of P V
// HBM bounds it.
template <int D, bool PAGED, int NB>
struct DiffGeo {
    static constexpr int CW = 4, COLS = 8 * NB;
    static constexpr int BOXES = D / 64;
    static constexpr int STAGE = 2 * BOXES * kBoxBytes;
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int PITCH = D + 4;  // of a column's output in shared memory (no two banks alike)
    static constexpr int RED = CW * COLS * (PITCH + 2) * 4;
    static constexpr int SMEM = 1024 + STAGES * STAGE + STAGES * 16 + STAGES * 4 + 64;
    static_assert(RED <= STAGES * STAGE, "the combine's scratch must fit in the ring");
};

template <int D, bool PAGED, int NB>
__global__ void __launch_bounds__((DiffGeo<D, PAGED, NB>::CW + 1) * 32, 2)
diff_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const DiffParams p) {
    using Geo = DiffGeo<D, PAGED, NB>;
    constexpr int CW = Geo::CW, COLS = Geo::COLS, BOXES = Geo::BOXES, STAGE = Geo::STAGE, STAGES = Geo::STAGES;
    constexpr int PITCH = Geo::PITCH, E = D / 32;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE);
    uint64_t* empty = full + STAGES;
    int* stage_rows = reinterpret_cast<int*>(empty + STAGES);

    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait_primary();
    const int L = clamped_len(p.seq_lens, b, p.L_max, &g_status_diff);
    const int chunk = chunk_len(L, p.splits, p.chunk_fixed);
    const int t0 = split * chunk, t1 = min(L, t0 + chunk);
    const long long row0 = (long long)b * p.Hq + h * p.G;
    const bool direct = p.splits == 1;
    if (t0 >= t1) {
        pdl_launch_dependents();
        if (direct) {  // an empty sequence (the merge knows the empty chunks by the lengths)
            for (int i = threadIdx.x; i < p.G * D; i += blockDim.x) {
                const size_t o = (size_t)row0 * D + i;
                if (p.out_bf16) static_cast<uint16_t*>(p.out)[o] = 0;
                else static_cast<float*>(p.out)[o] = 0.f;
            }
            if (p.lse && threadIdx.x < 2 * p.G) p.lse[2 * row0 + threadIdx.x] = -INFINITY;
        }
        return;
    }
    const int ntiles = (t1 - t0 + kTile - 1) / kTile;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], CW);
        }
        fence_barrier_init();
    }
    __syncthreads();

    if (warp == CW) {
        if (lane == 0) {
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmv);
            const uint64_t pol = l2_evict_first_policy();
            int t = 0;
            for (; t < ntiles; ++t) {
                const int s = t % STAGES;
                if (!mbar_wait(&empty[s], ((uint32_t)(t / STAGES) & 1u) ^ 1u, p.wait_limit_ns)) {
                    atomicOr(&g_status_diff, kStatusTimeout);
                    break;
                }
                if (t == p.withhold_tile) continue;  // fault injection: no copy, no arrival
                const int tok = t0 + t * kTile;
                int y = (b * p.Hkv + h) * p.L_max + tok;
                bool ok = true;
                if (PAGED) {
                    const int pg = p.page_table[(size_t)b * p.max_pages + tok / kTile];
                    ok = pg >= 0 && pg < p.num_pages;
                    y = (pg * p.Hkv + h) * kTile;
                }
                unsigned char* sk = smem + s * STAGE;
                if (ok) {
                    stage_rows[s] = min(kTile, t1 - tok);
                    mbar_arrive_expect_tx(&full[s], STAGE);
#pragma unroll
                    for (int bx = 0; bx < BOXES; ++bx) {
                        tma_load_box(sk + bx * kBoxBytes, &tmk, 64 * bx, y, &full[s], pol);
                        tma_load_box(sk + (BOXES + bx) * kBoxBytes, &tmv, 64 * bx, y, &full[s], pol);
                    }
                } else {
                    atomicOr(&g_status_diff, kStatusBadPage);
                    stage_rows[s] = 0;
                    mbar_arrive(&full[s]);
                }
            }
            if (t < ntiles || p.withhold_tile >= 0) {
                // the consumers may have stopped early: let every copy in flight land
                for (int u = t - 1; u >= 0 && u >= t - STAGES; --u)
                    if (u != p.withhold_tile) mbar_wait(&full[u % STAGES], (uint32_t)(u / STAGES) & 1u, p.wait_limit_ns);
            }
        }
        pdl_launch_dependents();
        return;
    }

    const int gid = lane >> 2, tig = lane & 3, mi = lane >> 3;
    uint32_t qa0[D / 16], qa2[D / 16];  // B fragments of this lane's column
    {
        const int map = NB == 1 && gid >= p.G ? 1 : 0, g = gid - map * p.G;
        const bool some = g < p.G;
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(p.q + (size_t)(row0 + (some ? g : 0)) * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const bool mine = some && (NB == 2 || (kk >= D / 32) == (map == 1));
            qa0[kk] = mine ? qrow[8 * kk + tig] : 0u;
            qa2[kk] = mine ? qrow[8 * kk + 4 + tig] : 0u;
        }
    }
    TokAcc<D> ac[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) tok_acc_init(ac[n]);
    bool failed = false;
    const int a_row = warp * 16 + 8 * (mi & 1) + (lane & 7);
    const int r0 = warp * 16 + gid;
    for (int t = 0; t < ntiles; ++t) {
        const int s = t % STAGES;
        if (!warp_wait(&full[s], (uint32_t)(t / STAGES) & 1u, p.wait_limit_ns)) {
            atomicOr(&g_status_diff, kStatusTimeout);
            failed = true;
            break;
        }
        const int rows = stage_rows[s];
        unsigned char* sk = smem + s * STAGE;
        const uint32_t ks = smem_u32(sk);
        float s2[2][4] = {}, sc[NB][4];  // the scores by halves of the key
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a0, a1, a2, a3;
            ldsm_x4(ks + swz(a_row, 2 * kk + (mi >> 1)), a0, a1, a2, a3);
            mma_bf16(s2[kk >= D / 32 ? 1 : 0], a0, a1, a2, a3, qa0[kk], qa2[kk]);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = NB == 2 ? s2[n][i] : 2 * tig + (i & 1) < p.G ? s2[0][i] : s2[1][i];
                sc[n][i] = r0 + 8 * (i >> 1) < rows ? x * p.scale_log2 : -INFINITY;
            }
        unsigned char* sv = sk + BOXES * kBoxBytes;
        softmax_pv<D, NB>(ac, sc, smem_u32(sv), sv, warp, lane, rows);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
    }
    pdl_launch_dependents();

    // combine the warps through shared memory (the ring is done with)
    float* red_o = reinterpret_cast<float*>(smem);    // [CW][COLS][PITCH]
    float* red_ml = red_o + CW * COLS * PITCH;        // [CW][COLS][2]
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            ac[n].l.x += __shfl_xor_sync(0xffffffffu, ac[n].l.x, off);
            ac[n].l.y += __shfl_xor_sync(0xffffffffu, ac[n].l.y, off);
        }
    named_barrier(1, CW * 32);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        float* to = red_o + (warp * COLS + 8 * n + 2 * tig) * PITCH;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(i & 1) * PITCH + 16 * mt + gid + 8 * (i >> 1)] = ac[n].o[mt][i];
        if (gid == 0) {
            float* ml = red_ml + 2 * (warp * COLS + 8 * n + 2 * tig);
            ml[0] = failed ? -INFINITY : ac[n].m.x;
            ml[1] = failed ? 0.f : ac[n].l.x;
            ml[2] = failed ? -INFINITY : ac[n].m.y;
            ml[3] = failed ? 0.f : ac[n].l.y;
        }
    }
    named_barrier(1, CW * 32);
    for (int g = warp; g < p.G; g += CW) {
        float o[2][E], l[2];
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            const int col = map * (NB == 1 ? p.G : 8) + g;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < CW; ++w) M = fmaxf(M, red_ml[2 * (w * COLS + col)]);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[map][e] = 0.f;
#pragma unroll
            for (int w = 0; w < CW; ++w) {
                const float* ml = red_ml + 2 * (w * COLS + col);
                const float f = ml[0] == -INFINITY ? 0.f : exp2_approx(ml[0] - M);
                const float* from = red_o + (w * COLS + col) * PITCH + lane * E;
                sum += f * ml[1];
#pragma unroll
                for (int e = 0; e < E; ++e) o[map][e] += f * from[e];
            }
            const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[map][e] *= inv;
            l[map] = sum;
            const size_t row = (size_t)(row0 + g) * 2 + map;
            if (direct) {
                if (lane == 0 && p.lse) p.lse[row] = natural_lse(M, sum);
            } else {
                const size_t rec = row * p.splits + split;
#pragma unroll
                for (int e = 0; e < E; ++e) p.part_o[rec * D + lane * E + e] = o[map][e];
                if (lane == 0) {
                    p.part_ml[2 * rec] = M;
                    p.part_ml[2 * rec + 1] = sum;
                }
            }
        }
        if (direct)
            store_difference<D>(o[0], o[1], l[0], l[1], p.mix, b, h * p.G + g, (size_t)(row0 + g), p.out, p.out_bf16,
                                lane);
    }
}

// Merge: for each row (token, query head) the n records of either map,
// O = sum_i w_i O_i / sum_i w_i with w_i = 2^(m_i - M) l_i, then their difference.  W warps a map:
// 1 with four rows a CTA, or 4 with one.  Prompts (cu): every record is written, l = 0 where
// nothing was attended (its O then need not be).  Decode (cu null): the records of the chunks
// that the length has.
template <int D, int W>
__global__ void __launch_bounds__(256) merge_diff_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml,
                                                         const int32_t* __restrict__ cu, int B, long long rows, int Hq,
                                                         int splits, const int32_t* __restrict__ lens, int L_max,
                                                         int chunk_fixed, void* __restrict__ out, int out_bf16,
                                                         float* __restrict__ lse, const DiffMix mix) {
    constexpr int E = D / 32, AHEAD = 8, ROWS = 4 / W;
    __shared__ float part[8][D + 1];
    __shared__ float second[ROWS][D + 1];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int w0 = warp % W, map = warp / W % 2, r = warp / (2 * W);
    const long long row = (long long)blockIdx.x * ROWS + r;
    bool live = row < rows;
    const int token = live ? (int)(row / Hq) : 0;
    int n = splits;
    if (cu) {
        live = live && token >= cu[0] && token < cu[B];
    } else if (live) {
        const int L = clamped_len(lens, token, L_max, nullptr), chunk = chunk_len(L, splits, chunk_fixed);
        n = min(splits, (L + chunk - 1) / chunk);
    }
    if (!live) n = 0;
    const float2* ml = reinterpret_cast<const float2*>(part_ml) + (row * 2 + map) * splits;
    const float* po = part_o + (row * 2 + map) * splits * D + lane * E;
    auto load = [&](int i, float (&v)[E]) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 x = reinterpret_cast<const float2*>(po + (size_t)i * D)[e / 2];
            v[e] = x.x;
            v[e + 1] = x.y;
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
    const int mine = (n - w0 + W - 1) / W;  // records w0 + W j
    for (int base = 0; base < mine; base += 32) {
        float w = 0.f;
        if (base + lane < mine) {
            const float2 x = ml[w0 + W * (base + lane)];
            if (x.y != 0.f) w = exp2_approx(x.x - top) * x.y;
        }
        const int cnt = 32 - __clz(__ballot_sync(0xffffffffu, w != 0.f));
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
        if (w0 == 0) {
#pragma unroll
            for (int u = 1; u < W; ++u) {
                sum += part[warp + u][D];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += part[warp + u][lane * E + e];
            }
        }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
    if (w0 == 0 && map == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) second[r][lane * E + e] = acc[e];
        if (lane == 0) second[r][D] = sum;
    }
    __syncthreads();
    if (!live || w0 != 0) return;
    if (lane == 0 && lse) lse[row * 2 + map] = natural_lse(M, sum);
    if (map == 0) {
        float o2[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o2[e] = second[r][lane * E + e];
        store_difference<D>(acc, o2, sum, second[r][D], mix, token, (int)(row - (long long)token * Hq), (size_t)row, out,
                            out_bf16, lane);
    }
}

template <int D, bool PAGED, int NB>
struct DiffLauncher {
    using Geo = DiffGeo<D, PAGED, NB>;
    static constexpr auto kernel = diff_kernel<D, PAGED, NB>;
    // Per device: the dynamic shared memory allowed once, and the occupancy for the planner.
    static cudaError_t prepare(int* ctas) {
        static int known[64] = {};
        int dev = 0, n = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= 64 || known[dev] == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::SMEM);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, (Geo::CW + 1) * 32, Geo::SMEM);
            if (e != cudaSuccess) return e;
            if (n < 1) n = 1;
            if (dev < 64) known[dev] = n;
        } else {
            n = known[dev];
        }
        if (ctas) *ctas = n;
        return cudaSuccess;
    }
    static cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p, dim3 grid,
                              cudaStream_t st) {
        const cudaError_t e = prepare(nullptr);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, grid, dim3((Geo::CW + 1) * 32), Geo::SMEM, st, tk, tv, p);
    }
};

template <typename F>
auto dispatch(int D, bool paged, int G, F f) {
    if (D == 128) {
        if (paged) return G <= 4 ? f(DiffLauncher<128, true, 1>()) : f(DiffLauncher<128, true, 2>());
        return G <= 4 ? f(DiffLauncher<128, false, 1>()) : f(DiffLauncher<128, false, 2>());
    }
    if (paged) return G <= 4 ? f(DiffLauncher<64, true, 1>()) : f(DiffLauncher<64, true, 2>());
    return G <= 4 ? f(DiffLauncher<64, false, 1>()) : f(DiffLauncher<64, false, 2>());
}

}  // namespace

int diff_ctas_per_sm(int D, int G, bool paged) {
    int n = 1;
    return dispatch(D, paged, G, [&](auto k) { return k.prepare(&n); }) == cudaSuccess ? n : 1;
}

cudaError_t launch_merge_diff(const float* part_o, const float* part_ml, const int32_t* cu, int B, int tokens, int Hq,
                              int D, int splits, const int32_t* lens, int L_max, int chunk_fixed, void* out,
                              int out_bf16, float* lse, const DiffMix& mix, cudaStream_t stream) {
    const long long rows = (long long)tokens * Hq;
    // A few rows with long lists leave most of the GPU idle with a warp a map (whole calls: 32 rows of 64
    // records 28.4 us with one, 25.9 with four; 64 rows of 76 162 and 157; 1024 rows of 2 27.3 and 29.5).
    const bool wide = splits > 8 && rows < 4096;
    const dim3 grid((unsigned)(wide ? rows : (rows + 3) / 4));
    const auto kernel = D == 128 ? (wide ? merge_diff_kernel<128, 4> : merge_diff_kernel<128, 1>)
                                 : (wide ? merge_diff_kernel<64, 4> : merge_diff_kernel<64, 1>);
    return launch_pdl(kernel, grid, dim3(256), 0, stream, part_o, part_ml, cu, B, rows, Hq, splits, lens, L_max,
                      chunk_fixed, out, out_bf16, lse, mix);
}

cudaError_t launch_decode_diff(const DecodeArgs& a, const DiffMix& mix, cudaStream_t stream) {
    if (a.B == 0) return cudaSuccess;
    const bool paged = a.page_table != nullptr;
    const uint64_t rows = paged ? (uint64_t)a.num_pages * a.Hkv * kTile : (uint64_t)a.B * a.Hkv * a.L_max;
    CUtensorMap tk, tv;
    // (an empty pool or cache: nothing is read, any well-formed map will do)
    if (!make_row_map(&tk, rows ? a.k : a.q, rows ? rows : 1, (uint32_t)a.D * 2) ||
        !make_row_map(&tv, rows ? a.v : a.q, rows ? rows : 1, (uint32_t)a.D * 2))
        return cudaErrorInvalidValue;
    DiffParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.seq_lens = a.seq_lens;
    p.page_table = a.page_table;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.L_max = a.L_max;
    p.G = a.Hq / a.Hkv;
    p.scale_log2 = a.scale * kLog2e;
    p.splits = a.splits;
    p.chunk_fixed = a.chunk_fixed;
    injected_timeout(&p.wait_limit_ns, &p.withhold_tile);
    p.out = a.out;
    p.out_bf16 = a.out_bf16;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_ml = a.part_ml;
    p.mix = mix;
    const dim3 grid((unsigned)a.splits, (unsigned)a.Hkv, (unsigned)a.B);
    const cudaError_t e = dispatch(a.D, paged, p.G, [&](auto k) { return k.launch(tk, tv, p, grid, stream); });
    if (e != cudaSuccess || a.splits == 1) return e;
    return launch_merge_diff(a.part_o, a.part_ml, nullptr, a.B, a.B, a.Hq, a.D, a.splits, a.seq_lens, a.L_max,
                             a.chunk_fixed, a.out, a.out_bf16, a.lse, mix, stream);
}

cudaError_t diff_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_diff, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_diff, &zero, sizeof(unsigned));
}

}  // namespace fd
