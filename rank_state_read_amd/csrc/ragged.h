// Ragged batches: which state rows and tokens a sequence of a call stands for.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "sketchssm_internal.h"

namespace skssm {

// What the ragged entry points (sketchssm_rmw_seq, sketchssm_prefill) share.
struct RaggedArgs {
    const float* S0;         // first states, or null: every sequence starts from zero
    float* S;                // last states
    const int32_t* rows0;    // state row of S0 per sequence (negative: zero), or null: as rows
    const int32_t* rows;     // state row of S per sequence, or null: sequence i is row i
    const int32_t* offsets;  // [n_seqs + 1] first token of each sequence
    const void* q;
    const void* k;
    const void* v;
    const float* a;
    const float* beta;
    float* y;
    int B0, B, n_seqs, total, max_len;
    int H, Hk, share;  // key/query heads; each serves `share` consecutive heads
    uint32_t* firsts;  // chunked form: each sequence's first slot of the workspace
};

struct SeqSpan {
    int row, row0;  // row0 < 0: start from zero
    int t0, len;
    bool live;
};

// Sequence i of the call.  The lists live on the device, so what they hold is
// checked here: a sequence with a row, a first token or a length out of range
// is idle, nothing of it is read or written.
__device__ __forceinline__ SeqSpan seq_span(const RaggedArgs& A, int i) {
    SeqSpan s;
    const int t1 = A.offsets[i + 1];
    s.t0 = A.offsets[i];
    s.row = A.rows ? A.rows[i] : i;
    s.row0 = !A.S0 ? -1 : A.rows0 ? A.rows0[i] : s.row;
    s.live = s.t0 >= 0 && t1 >= s.t0 && t1 <= A.total && s.row >= 0 && s.row < A.B && s.row0 < A.B0;
    s.len = s.live ? t1 - s.t0 : 0;
    if (s.len > A.max_len) s.live = false;
    return s;
}

// The same where every lane asks for one sequence.  What lanes share is moved to
// scalar registers: a buffer resource built from vector registers costs a loop
// over their values at each access.
__device__ __forceinline__ SeqSpan seq_span_uniform(const RaggedArgs& A, int i) {
    SeqSpan s = seq_span(A, __builtin_amdgcn_readfirstlane(i));
    s.row = __builtin_amdgcn_readfirstlane(s.row);
    s.row0 = __builtin_amdgcn_readfirstlane(s.row0);
    s.t0 = __builtin_amdgcn_readfirstlane(s.t0);
    s.len = __builtin_amdgcn_readfirstlane(s.len);
    s.live = __builtin_amdgcn_readfirstlane(int(s.live)) != 0;
    return s;
}

// How many lanes below this one are set in a ballot's mask.  (Not by a shift of the mask by the lane's number: on
// gfx950 a 64-bit shift has taken another amount than its own where that lay in the wave's last vector register.)
__device__ __forceinline__ int lanes_below(unsigned long long m) {
    return int(__builtin_amdgcn_mbcnt_hi(uint32_t(m >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m), 0u)));
}

// The sequence that the r-th group of blocks takes where those of more than twice
// the mean length go first, so that the last blocks to start are short ones.
__device__ __forceinline__ int seq_long_first(const RaggedArgs& A, int r, int lane) {
    const int bar = 2 * (A.total / A.n_seqs);
    auto is_long = [&](int i) {
        const int at = min(i, A.n_seqs - 1);
        return long(A.offsets[at + 1]) - A.offsets[at] > bar;
    };
    int n = 0;
    for (int c = 0; c < A.n_seqs; c += 64) n += __popcll(__ballot(c + lane < A.n_seqs && is_long(c + lane)));
    const bool first = r < n;
    if (!first) r -= n;
    for (int c = 0; c < A.n_seqs; c += 64) {
        const bool in = c + lane < A.n_seqs && is_long(c + lane) == first;
        const unsigned long long m = __ballot(in);
        n = __popcll(m);
        if (r < n) return c + __ffsll(__ballot(in && lanes_below(m) == r)) - 1;
        r -= n;
    }
    return 0;  // r >= n_seqs: no such group
}

// Checks the arguments of a ragged entry point (host) and fills `out`.
sketchssm_status ragged_args(const sketchssm_shape* shape, const float* S0, int32_t n_rows0, const int32_t* rows0,
                             float* S, const int32_t* rows, const int32_t* offsets, int32_t n_seqs,
                             int32_t total_tokens, int32_t max_len, const void* q, const void* k, const void* v,
                             const float* a, const float* beta, float* y, RaggedArgs* out);

// The recurrent form's launch (recur.hip).
hipError_t launch_recur(const sketchssm_shape& sh, const RaggedArgs& a, hipStream_t s);

}  // namespace skssm
