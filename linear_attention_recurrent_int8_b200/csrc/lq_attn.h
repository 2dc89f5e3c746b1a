// lq_attn.h -- internal interface between the C-ABI layer of the
// softmax-attention operators (lq_attn_api.cu) and their kernel launchers.
// Not installed; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lq {

constexpr unsigned int kErrBadPage = 4u;  // device error word: block_table entry out of range

constexpr int kMaxAttnBatch = 4096;  // sequences of one attention call

// Norm, rotation and (with `append`) the write into the paged cache.
struct RowsArgs {
    const void *q, *k, *v;              // q may be nullptr (Hq is then 0)
    long long q_stride, k_stride, v_stride;  // elements between tokens
    const float *q_weight, *k_weight;   // [D] or nullptr
    const float *cos_sin;               // [table_len][rot]
    void *q_out, *k_out;                // dense outputs (k_out: without append)
    const int32_t *positions;           // without append: [tokens] or nullptr
    // append
    void *k_pages, *v_pages;
    const int32_t *block_table, *pos, *cu;
    int B, num_pages, page_size, page_shift, max_pages;
    int tokens, Hq, Hkv;
    int norm, rot, table_len;
    float eps;
};
cudaError_t launch_rows(const RowsArgs &a, int D, bool bf16, bool adjacent, bool append,
                        cudaStream_t stream);

// Attention over the paged cache.
struct AttnArgs {
    const void *k_pages, *v_pages;
    const int32_t *block_table, *pos, *cu;
    const void *q;
    void *o;
    unsigned char *ws;
    int B, Hq, Hkv, num_pages, page_size, page_shift, max_pages;
    int tokens;  // prefill: rows of q and o
    int window;
    float scale, softcap;
};
size_t attn_decode_workspace_bytes(int B, int Hq, int Hkv, int D, bool bf16, cudaError_t *err);
cudaError_t launch_attn_decode(const AttnArgs &a, int D, bool bf16, cudaStream_t stream);
cudaError_t launch_attn_prefill(const AttnArgs &a, int D, bool bf16, cudaStream_t stream);

}  // namespace lq
