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
    int slots_here;  // assign_kernel writes the slots too
    int lens_here;   // and seq_lens
    int in_place;    // an output is an input's buffer: the CTAs are one cluster
};

// What a sequence brings: lengths that the table cannot hold are cut, and
// reported; the tokens cut off keep their place among the slots.
struct Lengths {
    int cached, fresh, end;
    bool bad;
};
__device__ __forceinline__ Lengths lengths_of(const AssignParams& p, int b) {
    const long long cap = (long long)p.max_pages * kTile;
    const int cached = p.cached_lens[b], fresh = p.new_lens[b];
    Lengths l;
    l.bad = cached < 0 || cached > cap || fresh < 0 || fresh > cap - cached;
    l.cached = (int)min(max((long long)cached, 0LL), cap);
    l.fresh = max(fresh, 0);
    l.end = l.cached + (int)min((long long)l.fresh, cap - l.cached);
    return l;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Sequences in groups of 1024, one per thread, with running sums of their new
// tokens and pages.  Every CTA computes the same sums; the table entries and the
// slots of a group are shared out among the CTAs, CTA 0 writes the rest.  Where
// outputs are the inputs' own buffers, the CTAs are one cluster and meet once all
// have read a group's lengths (and the head of the free list before it is
// replaced); apart from that they need nothing of each other.
__global__ void __launch_bounds__(kAssignThreads) assign_kernel(const AssignParams p) {
    __shared__ long long red[64];
    __shared__ int cu_s[kAssignThreads + 1];
    __shared__ int cached_s[kAssignThreads];
    __shared__ int end_s[kAssignThreads];
    __shared__ long long first_s[kAssignThreads];  // pages taken by the group's sequences before this one
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int part = blockIdx.x, parts = gridDim.x;
    long long head = p.free_head ? p.free_head[0] : 0;
    bool bad = false, out_of_pages = false;
    if (head < 0) {
        head = 0;
        bad = true;
    }
    long long tokens = 0, pages = 0;  // before this group
    for (int b0 = 0; b0 < p.B; b0 += kAssignThreads) {
        const int b = b0 + tid, n = min(p.B - b0, kAssignThreads);
        Lengths l = {0, 0, 0, false};
        if (tid < n) l = lengths_of(p, b);
        bad |= l.bad;
        long long tok = l.fresh, pg = pages_of(l.end) - pages_of(l.cached), ttok, tpg;
        block_scan2(tok, pg, ttok, tpg, red);
        cu_s[tid] = (int)min(tokens + tok, (long long)p.total_new);
        cached_s[tid] = l.cached;
        end_s[tid] = l.end;
        first_s[tid] = pg;
        if (tid == 0) cu_s[n] = (int)min(tokens + ttok, (long long)p.total_new);
        if (p.in_place && parts > 1) cluster_sync();
        else __syncthreads();
        if (part == 0 && tid < n) {
            p.cu_new[b] = cu_s[tid];
            if (p.lens_here) p.seq_lens[b] = l.end;
        }
        // the group's new pages, one per thread
        const long long base = head + pages;
        for (long long i = (long long)part * kAssignThreads + tid; i < tpg; i += (long long)parts * kAssignThreads) {
            if (base + i >= p.num_free) out_of_pages = true;
            int lo = 0, hi = n;  // the last sequence with first <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (first_s[mid] <= i) lo = mid;
                else hi = mid;
            }
            p.page_table[(size_t)(b0 + lo) * p.max_pages + pages_of(cached_s[lo]) + (int)(i - first_s[lo])] =
                base + i < p.num_free ? p.free_pages[base + i] : -1;
        }
        if (p.slots_here) {
            const int t0 = cu_s[0], t1 = cu_s[n];
            const int lane0 = part * kAssignThreads + tid, lanes = parts * kAssignThreads;
            auto sequence = [&](int t) {  // the last one with cu <= t
                int lo = 0, hi = n;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (cu_s[mid] <= t) lo = mid;
                    else hi = mid;
                }
                return lo;
            };
            auto page_of = [&](int s, int j) -> int {  // page j of a sequence
                const int old = pages_of(cached_s[s]);
                if (j < old) return p.page_table[(size_t)(b0 + s) * p.max_pages + j];
                const long long at = base + first_s[s] + j - old;
                return at < p.num_free ? p.free_pages[at] : -1;
            };
            auto slot_in = [](int page, unsigned pos) {
                return page < 0 ? (int64_t)-1 : (int64_t)page * kTile + pos % kTile;
            };
            auto slot_of = [&](int t, int s) -> int64_t {
                const unsigned pos = cached_s[s] + (unsigned)(t - cu_s[s]);  // (cut tokens may pass 2^31)
                return pos < (unsigned)end_s[s] ? slot_in(page_of(s, pos / kTile), pos) : -1;
            };
            if (t1 - t0 <= lanes) {
                if (t0 + lane0 < t1) p.slots[t0 + lane0] = slot_of(t0 + lane0, sequence(t0 + lane0));
            } else {
                // four tokens a thread, mostly of one sequence and one or two of its pages
                for (long long four = (long long)(t0 & ~3) + 4 * lane0; four < t1; four += 4LL * lanes) {
                    const int t = (int)four;
                    int s = sequence(max(t, t0));
                    const unsigned pos = cached_s[s] + (unsigned)(t - cu_s[s]);
                    int64_t* to = p.slots + t;
                    if (t >= cu_s[s] && t + 3 < min(cu_s[s + 1], t1) && pos + 3 < (unsigned)end_s[s]) {
                        const int page = page_of(s, pos / kTile);
                        const int next = pos % kTile > kTile - 4 ? page_of(s, pos / kTile + 1) : page;
                        int64_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = slot_in(pos % kTile + e < kTile ? page : next, pos + e);
                        reinterpret_cast<longlong2*>(to)[0] = make_longlong2(x[0], x[1]);
                        reinterpret_cast<longlong2*>(to)[1] = make_longlong2(x[2], x[3]);
                    } else {
#pragma unroll 1
                        for (int e = max(t0 - t, 0); e < 4 && t + e < t1; ++e) {
                            if (t + e >= cu_s[s + 1]) s = sequence(t + e);
                            to[e] = slot_of(t + e, s);
                        }
                    }
                }
            }
        }
        tokens += ttok;
        pages += tpg;
        __syncthreads();
    }
    if (tokens > p.total_new) bad = true;
    if (p.slots_here)
        for (long long t = tokens + part * kAssignThreads + tid; t < p.total_new; t += parts * kAssignThreads)
            p.slots[t] = -1;
    if (p.in_place && parts > 1) cluster_sync();  // free_head is read (B = 0 passes no barrier above)
    else __syncthreads();
    if (part == 0 && tid == 0) {
        p.cu_new[p.B] = (int)min(tokens, (long long)p.total_new);
        p.free_head_out[0] = (int)min(head + pages, (long long)p.num_free);
    }
    if (bad) atomicOr(&g_status_pages, kStatusBadSeqLen);
    if (out_of_pages) atomicOr(&g_status_pages, kStatusOutOfPages);
}

// Slots of many tokens from the finished table: a warp takes kSlotRun tokens in
// a row and finds the sequences of the first and the last by probing 32 places
// of the offsets at a time; a lane searches between them, two tokens at a time
// (one 16-byte store).
constexpr int kSlotRun = 256;

__global__ void __launch_bounds__(256) slots_kernel(const AssignParams p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long run = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kSlotRun;
    if (run >= p.total_new) return;
    // the last sequence in [s, s + n) whose offset is <= t, by the whole warp
    auto search = [&](int s, int n, long long t) {
        while (n > 1) {
            const int step = (n + 31) / 32;
            const bool below = lane * step < n && p.cu_new[s + lane * step] <= t;
            const unsigned votes = __ballot_sync(0xffffffffu, below);
            const int hit = votes ? 31 - __clz(votes) : 0;
            s += hit * step;
            n = min(step, n - hit * step);
        }
        return s;
    };
    int s = search(0, p.B, run);
    const int last = search(s, p.B - s, min(run + kSlotRun, (long long)p.total_new) - 1);
    int start = 0, next = 0, cached = 0, end = 0;
    auto enter = [&](int b) {
        const Lengths l = lengths_of(p, b);
        start = p.cu_new[b];
        next = p.cu_new[b + 1];
        cached = l.cached;
        end = l.end;
    };
    if (p.B > 0) enter(s);
    for (int i = 2 * lane; i < kSlotRun; i += 64) {
        int64_t out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const long long t = run + i + e;
            if (t >= next && s < last) {
                int hi = last + 1;
                while (hi - s > 1) {
                    const int mid = (s + hi) / 2;
                    if (p.cu_new[mid] <= t) s = mid;
                    else hi = mid;
                }
                enter(s);
            }
            out[e] = -1;
            const long long pos = cached + t - start;
            if (t < next && pos < end) {
                const int page = p.page_table[(size_t)s * p.max_pages + pos / kTile];
                if (page >= 0) out[e] = (int64_t)page * kTile + pos % kTile;
            }
        }
        int64_t* to = p.slots + run + i;
        if (run + i + 1 < p.total_new) *reinterpret_cast<longlong2*>(to) = make_longlong2(out[0], out[1]);
        else if (run + i < p.total_new) *to = out[0];
    }
}

// seq_lens in place of cached_lens, once the slots no longer need those.
__global__ void __launch_bounds__(256) lens_kernel(const AssignParams p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b < p.B) p.seq_lens[b] = lengths_of(p, b).end;
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
__device__ __forceinline__ long long pool_row(const AppendParams& p, long long slot, int h) {
    if (slot < 0) return -1;
    if (slot >= (long long)p.num_pages * kTile) {
        atomicOr(&g_status_pages, kStatusBadPage);
        return -1;
    }
    return (slot / kTile * p.Hkv + h) * kTile + slot % kTile;
}

// A thread per 16 bytes of K and of V.  The rows are loaded beside the slot,
// not after it: waiting for the slot first is a second memory latency for the
// same bytes in flight (31K tokens x 8 heads x 128: 41.2 us that way, 38.9 us
// this way, 6.6 TB/s of HBM; a decode step of 256 tokens 1.6 us).
template <int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    constexpr int C = D / 8;  // 16-byte chunks of a row
    pdl_wait_primary();
    pdl_launch_dependents();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)p.T * p.Hkv * C) return;
    const int c = (int)(i % C);
    const unsigned th = (unsigned)(i / C);  // token * Hkv + head
    const int t = (int)(th / (unsigned)p.Hkv), h = (int)(th - (unsigned)t * p.Hkv);
    const long long slot = p.slots[t];
    const uint4 kk = *reinterpret_cast<const uint4*>(p.k + (size_t)t * p.k_stride + (size_t)h * D + c * 8);
    const uint4 vv = *reinterpret_cast<const uint4*>(p.v + (size_t)t * p.v_stride + (size_t)h * D + c * 8);
    const long long row = pool_row(p, slot, h);
    if (row < 0) return;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k_pages) + row * D + c * 8) = kk;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_pages) + row * D + c * 8) = vv;
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

__device__ __forceinline__ void load16(uint32_t (&w)[8], const uint16_t* x) {
    const uint4 a = reinterpret_cast<const uint4*>(x)[0], b = reinterpret_cast<const uint4*>(x)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// HBM bounds it: 31K tokens x 8 heads x 128 in 30.4 us, 6.4 TB/s (29.9 us before it
// looked for NaN; 35.5 us with the rows loaded after their slots).
template <int D>
__global__ void __launch_bounds__(256) append_fp8_kernel(const AppendParams p) {
    constexpr int C = D / 16;
    pdl_wait_primary();
    pdl_launch_dependents();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    // every lane of a warp goes on to the end: the shuffles need them all
    const bool in = i < (long long)p.T * p.Hkv * C;
    const int c = (int)(i % C);
    const unsigned th = in ? (unsigned)(i / C) : 0u;  // token * Hkv + head
    const int t = (int)(th / (unsigned)p.Hkv), h = (int)(th - (unsigned)t * p.Hkv);
    const long long slot = p.slots[t];
    uint32_t k[8], v[8];
    load16(k, p.k + (size_t)t * p.k_stride + (size_t)h * D + c * 16);
    load16(v, p.v + (size_t)t * p.v_stride + (size_t)h * D + c * 16);
    const long long row = in ? pool_row(p, slot, h) : -1;
    encode_row<C>(k, static_cast<uint8_t*>(p.k_pages) + row * D, p.k_scales + row, row >= 0, c);
    encode_row<C>(v, static_cast<uint8_t*>(p.v_pages) + row * D, p.v_scales + row, row >= 0, c);
}

AppendParams append_params(const AppendArgs& a) {
    return AppendParams{static_cast<const uint16_t*>(a.k), static_cast<const uint16_t*>(a.v), a.k_stride, a.v_stride,
                        a.slots, a.T, a.Hkv, a.num_pages, a.k_pages, a.v_pages, a.k_scales, a.v_scales};
}

// Blocks of 256 threads, one piece of work each (a grid of eight blocks per SM
// in turns took 3% longer on 31K tokens x 8 heads).
unsigned append_grid(long long n) { return (unsigned)((n + 255) / 256); }

}  // namespace

// In place, assign_kernel writes the slots itself up to kSlotsHere new tokens; more
// go to slots_kernel on the whole GPU (32768 tokens: 7.1 us here, 8.0 us there; 131072:
// 14.2 and 8.4 us).
constexpr int kSlotsHere = 32768;
// In place, a cluster of eight CTAs shares out more new pages than kPagesAlone and
// more slots than kSlotsAlone, a single CTA writes fewer (256 tokens: 5.5 us with
// eight, 4.7 us alone; 4096: 5.9 and 6.7 us; 4096 pages: 9.3 and 11.2 us, 16384: 11.5
// and 22.6 us).
constexpr int kPagesAlone = 2048, kSlotsAlone = 2048;
// Otherwise a CTA per so many tokens and pages, a thread each, up to one CTA per SM
// (131072 tokens: 4.0 us, 5.6 us with 4096 and 4.0 us with 512 per CTA).  512 prompts
// with a million new tokens take 8.2 us on the GPU (a run of calls in a graph; 8.4 us a
// call into given outputs, 11.7 to 12.2 us when the call allocates them), 11.5 us in the
// two launches of a call in place; their 8.8 MB would pass HBM in 1.3 us; searches and
// page look-ups take 3.5 us of it, the stores 1 us, the launch, lengths and sums 3.7 us
// (two tokens a thread 9.15 us; a run of tokens per CTA that keeps its sequence 9.6 us).
constexpr int kPerCta = 1024;

cudaError_t launch_assign(const AssignArgs& a, cudaStream_t stream) {
    AssignParams p{a.cached_lens, a.new_lens, a.B, a.page_table, a.max_pages, a.free_pages, a.num_free, a.free_head,
                   a.total_new, a.seq_lens, a.cu_new, a.slots, a.free_head_out, 0, 0, 0};
    p.in_place = a.seq_lens == a.cached_lens || a.free_head_out == a.free_head;
    p.slots_here = !p.in_place || a.total_new <= kSlotsHere;
    p.lens_here = p.slots_here || a.seq_lens != a.cached_lens;
    const long long pages = (long long)a.total_new / kTile + a.B;
    unsigned parts = 1;
    if (p.in_place) {
        if (pages > kPagesAlone || (p.slots_here && a.total_new > kSlotsAlone)) parts = 8;
    } else {
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        const long long want = (a.total_new + pages + kPerCta - 1) / kPerCta;
        parts = (unsigned)(want < 1 ? 1 : want < sms ? want : sms);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts);
    cfg.blockDim = dim3(kAssignThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.in_place && parts > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, assign_kernel, p);
    if (e != cudaSuccess || p.slots_here) return e;
    const unsigned blocks = (unsigned)(((long long)a.total_new + 8 * kSlotRun - 1) / (8 * kSlotRun));
    e = launch_pdl(slots_kernel, dim3(blocks), dim3(256), 0, stream, p);
    if (e != cudaSuccess || p.lens_here || a.B == 0) return e;
    return launch_pdl(lens_kernel, dim3((a.B + 255) / 256), dim3(256), 0, stream, p);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    const dim3 grid(append_grid((long long)a.T * a.Hkv * (a.D / 8)));
    return launch_pdl(a.D == 128 ? append_kernel<128> : append_kernel<64>, grid, dim3(256), 0, stream,
                      append_params(a));
}

cudaError_t launch_append_fp8(const AppendArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    const dim3 grid(append_grid((long long)a.T * a.Hkv * (a.D / 16)));
    return launch_pdl(a.D == 128 ? append_fp8_kernel<128> : append_fp8_kernel<64>, grid, dim3(256), 0, stream,
                      append_params(a));
}

cudaError_t pages_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_pages, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_pages, &zero, sizeof(unsigned));
}

}  // namespace fd
