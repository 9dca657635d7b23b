// sketchssm_prefill: which form a call takes (prefill_common.h has the chunked one).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "prefill_common.h"

namespace skssm {

namespace {

// Whether a call takes the chunked kernels, else the recurrent one.  A chunk of 32
// tokens costs nearly the same however many of them there are, the recurrent form
// pays for each; three terms make the chunk dearer.  us chunked and recurrent at 16
// and 24 tokens of 128 sequences: GDN, 32 heads of 128, 197, 196 and 202, 270; Mamba-2,
// 128 heads of 80, 408, 383 and 422, 498; at 24 and 32 tokens: GDN with float32 keys
// 276, 270 and 293, 344; KDA 339, 289 and 346, 371.  One sequence crosses at about the
// same lengths (GDN, 16 and 20 tokens: 14.1, 17.8 and 14.4, 21.6).
bool chunked(const sketchssm_shape& sh, int max_len, int total) {
    const bool one_term = sh.qkv == SKSSM_BF16 && sh.kind != SKSSM_KDA;
    return std::min(max_len, total) > (one_term ? 16 : 28);
}

}  // namespace

}  // namespace skssm

using namespace skssm;

extern "C" size_t sketchssm_prefill_workspace(const sketchssm_shape* shape, int32_t n_seqs, int32_t total_tokens,
                                              int32_t max_len) {
    if (check_shape(shape) != SKSSM_OK || n_seqs <= 0 || total_tokens < 0 || max_len < 0) return 0;
    if (!chunked(*shape, max_len, total_tokens)) return 0;
    return walk_workspace(*shape, n_seqs, total_tokens, max_len);
}

extern "C" sketchssm_status sketchssm_prefill(const sketchssm_shape* shape, const float* S0, int32_t n_rows0,
                                              const int32_t* rows0, float* S, const int32_t* rows,
                                              const int32_t* offsets, int32_t n_seqs, int32_t total_tokens,
                                              int32_t max_len, const void* q, const void* k, const void* v,
                                              const float* a, const float* beta, float* y, void* workspace,
                                              size_t workspace_bytes, void* stream) {
    RaggedArgs A;
    const sketchssm_status st = ragged_args(shape, S0, n_rows0, rows0, S, rows, offsets, n_seqs, total_tokens, max_len,
                                            q, k, v, a, beta, y, &A);
    if (st != SKSSM_OK) return st;
    if (workspace && !aligned16(workspace)) return SKSSM_EALIGN;
    if (n_seqs == 0) return SKSSM_OK;
    const size_t need = sketchssm_prefill_workspace(shape, n_seqs, total_tokens, max_len);
    if (need && !workspace) return SKSSM_EINVAL;
    if (workspace_bytes < need) return SKSSM_ESHAPE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (!chunked(*shape, max_len, total_tokens)) e = launch_recur(*shape, A, s);
    else e = launch_walk(*shape, A, static_cast<char*>(workspace), s);
    if (e == hipErrorInvalidConfiguration) return SKSSM_ESHAPE;  // more threads than a launch takes
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
