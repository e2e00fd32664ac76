// fd_rows_diff.cu -- differential attention of packed query rows: whole prompts, and
// prompt tails over a paged cache.  The rows kernel with a map to each pipeline
// (kTwoMaps): both read the same tile of queries and the same blocks of keys and
// values, each its half of the query and key rows.
#include <type_traits>

#include "fd_rows.cuh"

namespace fd {

long long rows_diff_tiles(int B, int total_q, int G) { return (long long)total_q / rows_tok(G) + B; }
int rows_diff_tokens(int G) { return rows_tok(G); }

cudaError_t launch_rows_diff(const RowsArgs& a, const DiffMix& mix, cudaStream_t stream) {
    if (a.total_q == 0 || a.B == 0) return cudaSuccess;
    RowsParams p;
    RowsMaps m;
    if (!rows_setup(a, p, m)) return cudaErrorInvalidValue;
    p.mix = mix;
    // The norm's sum of d squares: values may be as large as 2^80, of which 2^-24 is in range.  With eps by 2^-48
    // still far above the smallest numbers, what small squares lose does not show beside it.  (A test of the sum and
    // a second pass over large ones instead: 1% slower on ragged prompts, 2% on tails.)
    if (mix.weight && mix.eps >= 0x1p-60f) {
        p.shrink = 0x1p-24f;
        p.mix.eps = mix.eps * 0x1p-48f;
    }
    p.tiles = (int)rows_diff_tiles(a.B, a.total_q, p.G);
    p.shared_work = (int)((long long)p.tiles * a.Hkv * a.splits);
    const dim3 grid((unsigned)p.shared_work);
    const auto launch = [&](auto d, auto pages) {
        constexpr int D = decltype(d)::value;
        constexpr bool P = decltype(pages)::value;
        return a.fine ? launch_kernel<D, P, kTwoMaps, true>(m, p, grid, stream)
                      : launch_kernel<D, P, kTwoMaps, false>(m, p, grid, stream);
    };
    using std::integral_constant;
    const bool paged = a.page_table != nullptr;
    if (a.D == 128) return paged ? launch(integral_constant<int, 128>(), std::true_type())
                                 : launch(integral_constant<int, 128>(), std::false_type());
    return paged ? launch(integral_constant<int, 64>(), std::true_type())
                 : launch(integral_constant<int, 64>(), std::false_type());
}

cudaError_t rows_diff_status_read(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_status_rows, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_status_rows, &zero, sizeof(unsigned));
}

}  // namespace fd
