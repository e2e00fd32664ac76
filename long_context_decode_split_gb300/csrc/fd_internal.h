// fd_internal.h -- host-side interface between the C-ABI layer (fd_api.cu)
// and the kernel translation units.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>
#include <cuda_runtime.h>

namespace fd {

constexpr int kTile = 64;  // tokens per pipeline stage; also the page size

#ifdef __CUDACC__
#define FD_HD __host__ __device__
#else
#define FD_HD
#endif

// Chunk length in tokens for a sequence of length L: `chunk_fixed` when the
// plan fixed one, else ceil(L / splits) rounded up to whole 64-token tiles.
FD_HD inline int chunk_len(int L, int splits, int chunk_fixed) {
    if (chunk_fixed > 0) return chunk_fixed;
    int c = (L + splits - 1) / splits;
    c = (c + kTile - 1) / kTile * kTile;
    return c > 0 ? c : kTile;
}

// Inputs and outputs of one split-KV decode launch (dense or paged).
struct DecodeArgs {
    const void* q;            // [B, Hq, D] bf16
    const void* k;            // contiguous [B, Hkv, L_max, D] or pool [P, Hkv, 64, D]
    const void* v;
    const void* k_scales;     // fp8 cache: [rows] binary32 row scales; fp4 cache: [rows, D/32] u8 block
    const void* v_scales;     // exponents (of K and of V)
    const int32_t* seq_lens;  // [B] or null (= L_max)
    const int32_t* page_table;// [B, max_pages] when paged, else null
    int max_pages, num_pages;
    int B, Hq, Hkv, L_max, D;
    float scale;
    int splits;               // chunks per sequence = grid.x
    int chunk_fixed;          // > 0: every sequence uses this chunk (tokens)
    void* out;                // [B, Hq, D]
    int out_bf16;
    float* lse;               // [B, Hq] or null
    float* part_o;            // workspace: [B, Hq, splits, D]
    float* part_ml;           // workspace: [B, Hq, splits, 2]
    int unified;              // bf16 cache only: unified-max variant with fixed max value `phi`
    float phi;                // (natural-log units of the scaled score)
    // bf16 cache only: chunks written as part of a longer list of partials
    // (the shared-prefix decode).  list_splits > 0: no merge follows; chunk i
    // goes to record rec0 + i of list_splits, empty chunks are marked, and the
    // first skip_tokens tokens of every sequence belong to someone else
    // (page_table then points at the first own page of row 0).
    int list_splits, rec0, skip_tokens;
};

// Workspace bytes for `splits` chunks (0 when splits == 1).
size_t decode_workspace_bytes(int B, int Hq, int D, int splits);

// Occupancy (resident CTAs per SM) of the partial-pass kernel for this shape.
int decode_ctas_per_sm(int D, int G, bool paged);

// Enqueue the partial pass (+ merge when splits > 1).  Returns a cudaError_t.
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);

// Device status words, one per translation unit that owns kernels.
cudaError_t decode_status_read(unsigned* bits, bool clear);

// Fault injection for the bf16 dense/paged pass and the prompt rows (fd_debug_inject_wait_timeout).
void inject_wait_timeout(unsigned long long wait_limit_ns, int withhold_tile);
void injected_timeout(unsigned long long* wait_limit_ns, int* withhold_tile);  // what a launch has to use

struct QuantArgs {
    const void* k;            // [B, Hkv, L_max, D] bf16
    const int32_t* seq_lens;
    int B, Hkv, L_max, D;
    uint8_t* codes;
    void* mn_scale;
    int8_t* res;
    void* res_scale;
};
cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t stream);

struct TopDeltaArgs {
    const void* q;
    const uint8_t* codes;
    const void* mn_scale;
    const int8_t* res;
    const void* res_scale;
    const void* v;
    const int32_t* seq_lens;
    int B, Hq, Hkv, L_max, D;
    float scale, delta;
    int n_sink, window;
    int splits, chunk_fixed;
    int group_union;
    void* out;
    int out_bf16;
    float* lse;
    uint32_t* sel_mask;
    int32_t* sel_count;
    float* part_o;
    float* part_ml;
};
int topdelta_ctas_per_sm(int D, int G);
cudaError_t launch_topdelta(const TopDeltaArgs& a, cudaStream_t stream);
cudaError_t topdelta_status_read(unsigned* bits, bool clear);

// fp8 (e4m3) KV cache: encoder and decode (DecodeArgs with k/v = codes,
// k_scales/v_scales = row scales; same workspace layout as the bf16 path).
struct Fp8QuantArgs {
    const void* x;            // [B, H, L_max, D] bf16
    const int32_t* seq_lens;
    int B, H, L_max, D;
    uint8_t* codes;           // [B, H, L_max, D]
    float* scales;            // [B, H, L_max]
};
cudaError_t launch_quantize_fp8(const Fp8QuantArgs& a, cudaStream_t stream);
int fp8_ctas_per_sm(int D, bool paged);
cudaError_t launch_decode_fp8(const DecodeArgs& a, cudaStream_t stream);
cudaError_t fp8_status_read(unsigned* bits, bool clear);

// fp4 (e2m1, power-of-two block scales) KV cache: encoder and decode.
struct Fp4QuantArgs {
    const void* x;            // [B, H, L_max, D] bf16
    const int32_t* seq_lens;
    int B, H, L_max, D;
    uint8_t* codes;           // [B, H, L_max, D/2] (channel pairs), or [B, H, (L_max+1)/2, D] (token pairs)
    uint8_t* scales;          // [B, H, L_max, D/32]
    int token_pairs;          // the value-cache layout: one byte = one channel of tokens 2p, 2p + 1
};
cudaError_t launch_quantize_fp4(const Fp4QuantArgs& a, cudaStream_t stream);
int fp4_ctas_per_sm(int D, bool paged);
cudaError_t launch_decode_fp4(const DecodeArgs& a, cudaStream_t stream);
cudaError_t fp4_status_read(unsigned* bits, bool clear);

// Attention of packed query rows (fd_rows.cu): prompts, prompt tails, and the
// shared part of a shared-prefix decode.  Sequence s owns the query tokens
// cu_q[s] .. cu_q[s + 1] - 1 (cu_q null: one sequence of total_q tokens) and
// Lk keys; its query i sees keys [0, Lk - Lq + i] (causal) or [0, Lk).
struct RowsArgs {
    const void* q;            // [total_q, Hq, D] bf16, tokens q_stride elements apart
    long long q_stride;
    const void* k;            // contiguous: token t of head h at t * k_stride + h * k_head_stride;
    const void* v;            // or pools [num_pages, Hkv, 64, D]
    long long k_stride, v_stride, k_head_stride, v_head_stride;
    const int32_t* cu_q;      // [B + 1] or null
    const int32_t* cu_k;      // contiguous keys: [B + 1] or null (sequence 0 has all total_k)
    const int32_t* seq_lens;  // pages: [B] keys of each sequence or null (max_pages * 64)
    const int32_t* row_lens;  // [total_q] or null: a further limit on the keys of a query
    const int32_t* page_table;// [B, table_stride] when paged, else null
    int max_pages, num_pages; // entries of a row that may be read; pages in the pool
    long long table_stride;
    int B, total_q, total_k, Hq, Hkv, D;
    int max_k;                // bound on Lk
    float scale;
    int causal;
    int splits, chunk;        // equal parts of a tile's keys, of at least `chunk` (both multiples of 128)
    void* out;                // splits == 1: [total_q, Hq, D] and lse [total_q, Hq] or null
    int out_bf16;
    float* lse;
    float* part_o;            // else record rec0 + chunk of rec_stride: [total_q, Hq, rec_stride, D]
    float* part_ml;           // and [total_q, Hq, rec_stride, 2]
    int rec0, rec_stride;     // (every record of a query row is written; empty ones get l = 0 and may lack O)
    int direct;               // write out/lse instead of records
    int fine;                 // weights in two bf16 terms (float32 results)
    // Own tokens of a shared-prefix decode, beside the work of single tiles: query token b also attends
    // own_lens[b] - own_skip tokens of its own, in chunks written to the records own_rec0 + chunk.
    const void* own_k;        // contiguous [total_q, Hkv, own_max, D]; paged: the pools above
    const void* own_v;
    const int32_t* own_lens;  // [total_q] or null (own_max)
    const int32_t* own_table; // paged: [total_q, own_table_stride]
    long long own_table_stride;
    int own_max, own_skip;    // own_max: most own tokens of a sequence
    int own_splits, own_chunk, own_rec0;  // equal parts of at least own_chunk; own_splits == 0: they are someone else's
};
// Whether the tokens of this call take one tile per CTA (own tokens are then part of its work).
// packed_k: the keys of a packed call (RowsArgs::cu_k given), -1 for others.
bool rows_single(int B, int total_q, int G, int packed_k);
// Tiles of `total_q` tokens: how many tokens one takes, and how many tiles there are at most
// (B sequences by offsets) or exactly (one sequence).
int rows_tokens(int B, int total_q, int G, int packed_k);
long long rows_tiles(int B, int total_q, int G, int packed_k, bool offsets);
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t stream);
cudaError_t rows_status_read(unsigned* bits, bool clear);
// Merge (fd_merge.cu) of n records per row, all of them written (l = 0: nothing attended).
// lens (or null): [tokens], an entry outside [0, len_most] is recorded in the device status.
// cu (or null: all): only the tokens cu[0] .. cu[B] - 1 have records and results.
cudaError_t launch_merge_list(const float* part_o, const float* part_ml, const int32_t* cu, int B, int tokens, int Hq,
                              int D, int n, void* out, int out_bf16, float* lse, cudaStream_t stream,
                              const int32_t* lens = nullptr, int len_most = 0);
cudaError_t merge_status_read(unsigned* bits, bool clear);

// Differential attention (fd_diff.cu, fd_rows_diff.cu): what joins a head's two maps.
struct DiffMix {
    const float* lambda;      // of token t, query head h: lambda[t * lambda_stride + h]
    long long lambda_stride;  // 0: the same for all tokens
    const float* weight;      // [D] norm of the difference, or null
    float eps;
};
// Decode with DecodeArgs as above (bf16 cache, lse [B, Hq, 2]); records of both maps:
// part_o [B, Hq, 2, splits, D], part_ml [B, Hq, 2, splits, 2].
int diff_ctas_per_sm(int D, int G, bool paged);
cudaError_t launch_decode_diff(const DecodeArgs& a, const DiffMix& mix, cudaStream_t stream);
// Prompts with RowsArgs as above (sequences by offsets; no row_lens, no own tokens); lse and records
// [total_q, Hq, 2, ..].  A tile has rows_diff_tokens tokens.
int rows_diff_tokens(int G);
long long rows_diff_tiles(int B, int total_q, int G);
cudaError_t launch_rows_diff(const RowsArgs& a, const DiffMix& mix, cudaStream_t stream);
// Merge of `splits` records per row and map.  cu given: prompts, every record of the tokens
// cu[0] .. cu[B] - 1 is written.  cu null: a decode's chunks, as many as the lengths have.
cudaError_t launch_merge_diff(const float* part_o, const float* part_ml, const int32_t* cu, int B, int tokens, int Hq,
                              int D, int splits, const int32_t* lens, int L_max, int chunk_fixed, void* out,
                              int out_bf16, float* lse, const DiffMix& mix, cudaStream_t stream);
cudaError_t diff_status_read(unsigned* bits, bool clear);
cudaError_t rows_diff_status_read(unsigned* bits, bool clear);

// Norms and rotation (fd_rope.cu): of rows to rows, or (slots given) with the keys and values on
// their way into the pages, which hold bf16, or e4m3 codes with the row scales.
struct RopeArgs {
    const uint16_t* q;        // [T, Hq, D], tokens the stride apart (elements); likewise the others
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride;
    int T, Hq, Hkv, D;
    const float* cos_sin;     // [max_pos, rot]: cosines, then sines
    int max_pos, rot, interleaved, halves;
    const int32_t* positions; // [T], or null: from cu [B + 1] and lens [B]
    const int32_t* cu;
    const int32_t* lens;
    int B;
    const float* q_weight;    // [D], or [D / 2] with halves; or null
    const float* k_weight;
    float eps;
    uint16_t* q_out;
    uint16_t* k_out;
    long long q_out_stride, k_out_stride;
    const int64_t* slots;     // [T]
    int num_pages;
    void* k_pages;
    void* v_pages;
    float* k_scales;
    float* v_scales;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t rope_status_read(unsigned* bits, bool clear);

// Page assignment and cache append (fd_pages.cu).
struct AssignArgs {
    const int32_t* cached_lens;
    const int32_t* new_lens;
    int B;
    int32_t* page_table;
    int max_pages;
    const int32_t* free_pages;
    int num_free;
    const int32_t* free_head;  // [1] or null (0)
    int total_new;
    int32_t* seq_lens;
    int32_t* cu_new;
    int64_t* slots;
    int32_t* free_head_out;
};
cudaError_t launch_assign(const AssignArgs& a, cudaStream_t stream);

struct AppendArgs {
    const void* k;            // [T, Hkv, D] bf16, tokens k_stride elements apart
    const void* v;
    long long k_stride, v_stride;
    const int64_t* slots;     // [T]
    int T, Hkv, D, num_pages;
    void* k_pages;            // bf16, or e4m3 codes with the row scales below
    void* v_pages;
    float* k_scales;
    float* v_scales;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_append_fp8(const AppendArgs& a, cudaStream_t stream);
cudaError_t pages_status_read(unsigned* bits, bool clear);

// Launch with programmatic stream serialization: the grid may be scheduled
// while the previous kernel in the stream is still running, so the kernel
// must execute griddepcontrol.wait before it touches global memory (every
// kernel launched this way does so first).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Merge of per-chunk partials (shared by the dense and top-delta paths).
cudaError_t launch_merge(const float* part_o, const float* part_ml, const int32_t* seq_lens,
                         int B, int Hq, int L_max, int D, int splits, int chunk_fixed,
                         void* out, int out_bf16, float* lse, cudaStream_t stream);

}  // namespace fd
