// Recurrent form for listed state rows on gfx950: a few tokens of each of n
// sequences, one after the other, on a state held in registers.  Per (b, h)
// and token
//   S <- M S + beta k v^T,   y = S^T q
// with Mamba-2 M = a I (beta = 1), GDN M = a (I - beta k k^T),
// KDA M = (I - beta k k^T) diag(a).
//
// The state is read once and written once whatever the number of tokens, so a
// call of one to a few tokens is bound by those 2 K V 4 bytes per item.  One
// block per (sequence, head) with V/16 waves; wave w holds value columns
// 16w..16w+15 for all 128 key rows in registers (lane l, register (kt, r) <->
// key row 16 kt + 4 (l/16) + r, column 16 w + l % 16).  Both sums over keys are
// a per-lane sum over the lane's 32 rows plus two exchanges between
// quarter-waves.  Tokens are staged in LDS eight at a time as fp32, so the
// token loop has no barrier inside.
//
// Measured: 192 sequences of a Mamba-2 layer (128 heads of 80, 500 tokens) 378 us, 5.4
// TB/s of states and tokens; 96 of a KDA layer (32 heads of 128, 480 tokens, one
// sequence of 57) 98 us, 4.4 TB/s; float32 tokens 383 and 112 us.  A plain stream that
// writes as much as it reads runs at 5.9 to 6.2 TB/s (torch's copy at 4.8 to 5.3).  One
// token of one GDN layer's row takes 5.6 us, the latency of its loads.  Registers: 72,
// six waves per SIMD (budgets of 5 and 4 with k kept between its two uses ran the same).
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "ragged.h"
#include "sketchssm_internal.h"
#include "state_tiles.h"

namespace skssm {

namespace {

constexpr int kTB = 8;  // tokens staged at a time

template <int KIND, int V>
struct RecurLds {
    static constexpr bool kda = KIND == SKSSM_KDA;
    static constexpr int ks = 0;
    static constexpr int qs = ks + kTB * kK;
    static constexpr int al = qs + kTB * kK;             // KDA: decays [kTB][K], else [kTB]
    static constexpr int be = al + (kda ? kTB * kK : kTB);
    static constexpr int vs = be + kTB;
    static constexpr int tokens = vs + kTB * V;
    static constexpr int tiles = 2 * 16 * (V + 4);       // the state on its way out, over the tokens
    static constexpr int total = tokens > tiles ? tokens : tiles;
};

__device__ __forceinline__ float recur_quarter_sum(float x) {
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    return x;
}

// Long sequences, of more than a 16th of the tokens, start before all others, in
// `kFront` groups of blocks in front of the grid.
constexpr int kFront = 15;

__device__ __forceinline__ bool is_long(const RaggedArgs& A, int i) {
    const int t0 = A.offsets[i], t1 = A.offsets[i + 1];
    return t0 >= 0 && t1 <= A.total && t1 > t0 && t1 - t0 > A.total / 16;
}

// How many of them have an index below `seq`.
__device__ __forceinline__ int longs_before(const RaggedArgs& A, int seq, int lane) {
    int n = 0;
    for (int c = 0; c < seq; c += 64) n += __popcll(__ballot(c + lane < seq && is_long(A, min(c + lane, seq))));
    return n;
}

// The r-th one, or -1.
__device__ __forceinline__ int long_sequence(const RaggedArgs& A, int r, int lane) {
    for (int c = 0; c < A.n_seqs; c += 64) {
        const bool mine = c + lane < A.n_seqs && is_long(A, min(c + lane, A.n_seqs - 1));
        const unsigned long long m = __ballot(mine);
        if (r < __popcll(m)) return c + __ffsll(__ballot(mine && __popcll(m & ((1ull << lane) - 1)) == r)) - 1;
        r -= __popcll(m);
    }
    return -1;
}

}  // namespace

template <int KIND, int V, typename QT>
__global__ __launch_bounds__(V / 16 * 64) __attribute__((amdgpu_waves_per_eu(6)))
void recur_kernel(RaggedArgs A, int front) {
    constexpr int K = kK;
    constexpr int NT = V / 16 * 64;
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    constexpr bool KDA = KIND == SKSSM_KDA;
    typedef RecurLds<KIND, V> L;
    __shared__ __align__(16) float lds[L::total];
    float* ks = lds + L::ks;
    float* qs = lds + L::qs;
    float* al = lds + L::al;
    float* be = lds + L::be;
    float* vs = lds + L::vs;

    const int tid = threadIdx.x;
    const int w = tid >> 6;
    const int lane = tid & 63;
    const int lr = lane & 15;
    const int lq = lane >> 4;
    const int v0 = 16 * w;
    const int group = blockIdx.x / A.H;
    const int h = blockIdx.x - group * A.H;
    const int seq = group < front ? long_sequence(A, group, lane) : group - front;
    if (seq < 0) return;
    const int hk = h / A.share;
    const SeqSpan sp = seq_span_uniform(A, seq);
    if (!sp.live) return;
    if (front && group >= front && is_long(A, seq) && longs_before(A, seq, lane) < front) return;  // in front

    f32x4 s[8];
    const int svo = (4 * lq * V + v0 + lr) * 4;
    if (sp.row0 >= 0) {
        const __amdgpu_buffer_rsrc_t s0 = buffer_rsrc(A.S0 + (size_t(sp.row0) * A.H + h) * (K * V), K * V * 4);
#pragma unroll
        for (int kt = 0; kt < 8; ++kt)
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) s[kt][rr] = buffer_load_f32(s0, svo, (16 * kt + rr) * V * 4);
    } else {
#pragma unroll
        for (int kt = 0; kt < 8; ++kt) s[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    for (int tb = 0; tb < sp.len; tb += kTB) {
        const int nb = min(kTB, sp.len - tb);
        const size_t t0 = size_t(sp.t0) + tb;
        if (tb) __syncthreads();  // the tokens before are read
        for (int i = tid; i < nb * (K / 8); i += NT) {
            const int j = i / (K / 8), c = 8 * (i - j * (K / 8));
            const size_t e = ((t0 + j) * A.Hk + hk) * K + c;
            float f[8];
            Vec8<QT>::unpack(Vec8<QT>::load(A.k, e), f);
            store8f(ks + j * K + c, f);
            Vec8<QT>::unpack(Vec8<QT>::load(A.q, e), f);
            store8f(qs + j * K + c, f);
            if (KDA) {
                load8f(A.a + ((t0 + j) * A.H + h) * K + c, f);
                store8f(al + j * K + c, f);
            }
        }
        for (int i = tid; i < nb * (V / 8); i += NT) {
            const int j = i / (V / 8), c = 8 * (i - j * (V / 8));
            float f[8];
            Vec8<QT>::unpack(Vec8<QT>::load(A.v, ((t0 + j) * A.H + h) * V + c), f);
            store8f(vs + j * V + c, f);
        }
        if (tid < nb) {
            if (!KDA) al[tid] = A.a[(t0 + tid) * A.H + h];
            be[tid] = DELTA ? A.beta[(t0 + tid) * A.H + h] : 1.f;
        }
        __syncthreads();

        for (int j = 0; j < nb; ++j) {
            const float* kj = ks + j * K + 4 * lq;
            const float* qj = qs + j * K + 4 * lq;
            const float* aj = al + j * K + 4 * lq;  // KDA only
            const float a_s = KDA ? 1.f : al[j];
            const float bt = be[j];
            const float vc = vs[j * V + v0 + lr];
            // erase term of this lane's column: k^T S (GDN), k^T diag(a) S (KDA, whose
            // state takes its decays here)
            float wc = 0.f;
            if (DELTA) {
#pragma unroll
                for (int kt = 0; kt < 8; ++kt) {
                    const f32x4 k4 = *reinterpret_cast<const f32x4*>(kj + 16 * kt);
                    if (KDA) s[kt] *= *reinterpret_cast<const f32x4*>(aj + 16 * kt);
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) wc = fmaf(k4[rr], s[kt][rr], wc);
                    __builtin_amdgcn_sched_barrier(0);
                }
                wc = recur_quarter_sum(wc);
            }
            const float u = KDA ? bt * (vc - wc) : DELTA ? bt * (vc - a_s * wc) : vc;
            float yc = 0.f;
#pragma unroll
            for (int kt = 0; kt < 8; ++kt) {
                const f32x4 k4 = *reinterpret_cast<const f32x4*>(kj + 16 * kt);
                const f32x4 q4 = *reinterpret_cast<const f32x4*>(qj + 16 * kt);
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    s[kt][rr] = fmaf(k4[rr], u, KDA ? s[kt][rr] : a_s * s[kt][rr]);
                    yc = fmaf(q4[rr], s[kt][rr], yc);
                }
                // one tile's operands at a time: within the register budget
                __builtin_amdgcn_sched_barrier(0);
            }
            yc = recur_quarter_sum(yc);
            if (lq == 0) A.y[((t0 + j) * A.H + h) * V + v0 + lr] = yc;
        }
    }
    const __amdgpu_buffer_rsrc_t so = buffer_rsrc(A.S + (size_t(sp.row) * A.H + h) * (K * V), K * V * 4);
    store_state_tiles<V>(s, lds, so, tid);
}

template <int KIND, int V, typename QT>
static hipError_t launch_recur_t(const RaggedArgs& a, hipStream_t s) {
    // Where there can be a long sequence and more waves are to come than the CUs hold:
    // us without and with, 96 sequences of a KDA layer, 480 tokens, one of 57: 138, 98;
    // 192 of a Mamba-2 layer, 500 tokens, one of 99 that starts early anyway: 372, 379.
    const int front = long(a.max_len) * 16 > a.total && long(a.n_seqs) * a.H * (V / 16) > 256 * 24 ? kFront : 0;
    if (!launch_fits(double(a.n_seqs + front) * a.H, V / 16 * 64)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((recur_kernel<KIND, V, QT>), dim3((a.n_seqs + front) * a.H), dim3(V / 16 * 64), 0, s, a, front);
    return hipGetLastError();
}

template <int KIND, typename QT>
static hipError_t launch_recur_v(int V, const RaggedArgs& a, hipStream_t s) {
    switch (V) {
        case 64: return launch_recur_t<KIND, 64, QT>(a, s);
        case 80: return launch_recur_t<KIND, 80, QT>(a, s);
        case 96: return launch_recur_t<KIND, 96, QT>(a, s);
        case 112: return launch_recur_t<KIND, 112, QT>(a, s);
        case 128: return launch_recur_t<KIND, 128, QT>(a, s);
    }
    return hipErrorInvalidValue;
}

template <typename QT>
static hipError_t launch_recur_k(int kind, int V, const RaggedArgs& a, hipStream_t s) {
    switch (kind) {
        case SKSSM_MAMBA2: return launch_recur_v<SKSSM_MAMBA2, QT>(V, a, s);
        case SKSSM_GDN: return launch_recur_v<SKSSM_GDN, QT>(V, a, s);
        case SKSSM_KDA: return launch_recur_v<SKSSM_KDA, QT>(V, a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_recur(const sketchssm_shape& sh, const RaggedArgs& a, hipStream_t s) {
    return sh.qkv == SKSSM_BF16 ? launch_recur_k<Bf16Tag>(sh.kind, sh.V, a, s)
                                : launch_recur_k<F32Tag>(sh.kind, sh.V, a, s);
}

sketchssm_status ragged_args(const sketchssm_shape* shape, const float* S0, int32_t n_rows0, const int32_t* rows0,
                             float* S, const int32_t* rows, const int32_t* offsets, int32_t n_seqs,
                             int32_t total_tokens, int32_t max_len, const void* q, const void* k, const void* v,
                             const float* a, const float* beta, float* y, RaggedArgs* out) {
    const sketchssm_status st = check_shape(shape);
    if (st != SKSSM_OK) return st;
    if (n_seqs < 0 || total_tokens < 0 || max_len < 0) return SKSSM_EINVAL;
    if (!S || !offsets || (!S0 && rows0)) return SKSSM_EINVAL;
    if (S0 && n_rows0 < 1) return SKSSM_ESHAPE;
    if (total_tokens > 0) {
        if (!q || !k || !v || !a || !y) return SKSSM_EINVAL;
        if ((shape->kind != SKSSM_MAMBA2) != (beta != nullptr)) return SKSSM_EINVAL;
    }
    // block indices, and elements of the first states, stay below 2^31
    if ((double(n_seqs) + kFront) * shape->H >= 2147483648.0) return SKSSM_ESHAPE;
    if (S0 && double(n_rows0) * shape->H * shape->K * shape->V >= 2147483648.0) return SKSSM_ESHAPE;
    const void* ptrs[] = {S0, S, rows0, rows, offsets, q, k, v, a, beta, y};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return SKSSM_EALIGN;
    RaggedArgs& A = *out;
    A.S0 = S0;
    A.S = S;
    A.rows0 = rows0;
    A.rows = rows;
    A.offsets = offsets;
    A.q = q;
    A.k = k;
    A.v = v;
    A.a = a;
    A.beta = beta;
    A.y = y;
    A.B0 = n_rows0;
    A.B = shape->B;
    A.n_seqs = n_seqs;
    A.total = total_tokens;
    A.max_len = max_len;
    A.H = shape->H;
    A.Hk = kq_heads_of(*shape);
    A.share = shape->H / A.Hk;
    A.firsts = nullptr;
    return SKSSM_OK;
}

}  // namespace skssm

using namespace skssm;

extern "C" sketchssm_status sketchssm_rmw_seq(const sketchssm_shape* shape, const float* S0, int32_t n_rows0,
                                              const int32_t* rows0, float* S, const int32_t* rows,
                                              const int32_t* offsets, int32_t n_seqs, int32_t total_tokens,
                                              int32_t max_len, const void* q, const void* k, const void* v,
                                              const float* a, const float* beta, float* y, void* stream) {
    RaggedArgs A;
    const sketchssm_status st = ragged_args(shape, S0, n_rows0, rows0, S, rows, offsets, n_seqs, total_tokens, max_len,
                                            q, k, v, a, beta, y, &A);
    if (st != SKSSM_OK) return st;
    if (n_seqs == 0) return SKSSM_OK;
    const hipError_t e = launch_recur(*shape, A, static_cast<hipStream_t>(stream));
    if (e == hipErrorInvalidConfiguration) return SKSSM_ESHAPE;  // more threads than a launch takes
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
