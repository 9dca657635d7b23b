// Prefill of ragged prompts for gfx950.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "ragged.h"
#include "sketchssm_internal.h"

using namespace skssm;

extern "C" size_t sketchssm_prefill_workspace(const sketchssm_shape* shape, int32_t n_seqs, int32_t total_tokens,
                                              int32_t max_len) {
    (void)shape, (void)n_seqs, (void)total_tokens, (void)max_len;
    return 0;
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
    const hipError_t e = launch_recur(*shape, A, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
