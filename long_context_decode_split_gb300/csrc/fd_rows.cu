// fd_rows.cu -- launches of the rows kernel: whole prompts, prompt tails over a
// paged cache, and the decode of a batch with a shared prefix.
#include <cmath>
#include <type_traits>

#include "fd_rows.cuh"

namespace fd {

namespace {

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
    RowsMaps m;
    if (!rows_setup(a, p, m)) return cudaErrorInvalidValue;
    const bool paged = a.page_table != nullptr;
    const int packed_k = a.cu_k ? a.total_k : -1;
    const bool dual = rows_dual(a.B, a.total_q, p.G, packed_k);
    const long long own_work = a.own_max > 0 ? (long long)a.total_q * a.Hkv * a.own_splits : 0;
    if (own_work > 0) {
        if (dual) return cudaErrorInvalidValue;
        bool ok = make_token_map(&m.own_q, a.q, a.D, a.Hq, a.total_q, a.D, a.q_stride, p.G, 1);
        if (!paged) {
            const long long head = (long long)a.own_max * a.D;
            ok = ok && make_token_map(&m.own_k, a.own_k, a.D, a.total_q * a.Hkv, a.own_max, head, a.D, 1, kBlock) &&
                 make_token_map(&m.own_v, a.own_v, a.D, a.total_q * a.Hkv, a.own_max, head, a.D, 1, kBlock);
        }
        if (!ok) return cudaErrorInvalidValue;
    }
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
    p.shared_work = (int)(tiles * a.Hkv * a.splits);
    const dim3 grid((unsigned)(p.shared_work + own_work));
    const auto launch = [&](auto d, auto pages) {
        constexpr int D = decltype(d)::value;
        constexpr bool P = decltype(pages)::value;
        if (dual) return a.fine ? launch_kernel<D, P, kTwoTiles, true>(m, p, grid, stream)
                                : launch_kernel<D, P, kTwoTiles, false>(m, p, grid, stream);
        return a.fine ? launch_kernel<D, P, kOneTile, true>(m, p, grid, stream)
                      : launch_kernel<D, P, kOneTile, false>(m, p, grid, stream);
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
