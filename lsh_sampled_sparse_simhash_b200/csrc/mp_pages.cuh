// Shapes and launchers of the exact-attention calls: prompts, the paged
// key-value cache, decode over it and the operations on its pages.
#pragma once

#include "mp_kernels.cuh"

namespace mp {

constexpr int kPagesMaxBatch = 4096;  // the page plans keep one word per sequence in shared memory

struct PromptShape {
    int B, Hq, Hkv, G, T;
    int64_t qs, ks, vs;  // elements from one token's row to the next
};

struct PagesShape {
    int B, Hq, Hkv, G, P, S, M;
};

int validate_prompt_shape(const mp_prompt_shape *in, PromptShape &s);
int validate_pages_shape(const mp_pages_shape *in, PagesShape &s);

cudaError_t launch_prompt(const PromptShape &s, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                          const int32_t *cu_lens, uint16_t *out, float *lse, int32_t *status, cudaStream_t st);

size_t paged_workspace_bytes(const PagesShape &s, int max_len);
cudaError_t launch_paged_attend(const PagesShape &s, const uint16_t *q, const uint16_t *kp, const uint16_t *vp,
                                const int32_t *table, const int32_t *lens, int max_len, float *out, float *lse,
                                void *workspace, int32_t *status, cudaStream_t st);
cudaError_t launch_paged_append(const PagesShape &s, const uint16_t *k_new, const uint16_t *v_new, int64_t ks, int64_t vs,
                                const int32_t *cu_new, int n_rows, int advance, const int32_t *table, int32_t *lens,
                                uint16_t *kp, uint16_t *vp, int32_t *status, cudaStream_t st);

cudaError_t launch_pages_reserve(const PagesShape &s, const int32_t *n_new, int32_t *table, const int32_t *lens,
                                 int32_t *refs, int32_t *status, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesShape &s, const int32_t *src, const int32_t *dst, int n, int32_t *table,
                              int32_t *lens, int32_t *refs, int32_t *copies, int32_t *status, cudaStream_t st);
cudaError_t launch_pages_free(const PagesShape &s, const int32_t *seqs, int n, int32_t *table, int32_t *lens,
                              int32_t *refs, int32_t *status, cudaStream_t st);
cudaError_t launch_pages_compact(const PagesShape &s, int32_t *table, int32_t *refs, int32_t *copies, int32_t *status,
                                 cudaStream_t st);
cudaError_t launch_pages_copy(const PagesShape &s, const int32_t *copies, int max_copies, uint16_t *kp, uint16_t *vp,
                              int32_t *status, cudaStream_t st);

}  // namespace mp
