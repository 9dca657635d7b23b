// Trees of drafted tokens over a row's cache on gfx950.  Per (sequence, head) a
// node n with ancestors (itself included) and the row's held-back window tokens
// before them:
//   walk, from n to the root and then from the window's last slot to its first:
//     s = k . x,  acc += beta s v,  x <- M^T x          (x = q_n at the start)
//   y = acc + S^T x (dense head)  |  acc + Z^T (F x) (sketch head)
// with Mamba-2 M = a I (beta = 1), GDN M = a (I - beta k k^T),
// KDA M = (I - beta k k^T) diag(a).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "sketchssm_internal.h"

namespace skssm {

namespace {

struct TreeArgs {
    const float* S;
    const float* Z;
    const float* frames;
    const void* kbuf;
    const void* vbuf;
    const float* abuf;
    const float* bbuf;
    const int32_t* pos;      // held-back tokens per state row, or null: none
    const int32_t* rows;     // state row of each sequence, or null: sequence i is row i
    const int32_t* offsets;  // [n_seqs + 1]
    const int32_t* parents;  // [total]
    const void* q;
    const void* k;
    const void* v;
    const float* a;
    const float* beta;
    float* y;
    int B, n_seqs, total, max_nodes;
    int H, Hk, share;
    int n_dense;  // dense heads lead the head table
};

// A sequence of the call; what the lists hold is checked here.
struct TreeSpan {
    int row, p, t0, len;
    bool live;
};

__device__ __forceinline__ TreeSpan tree_span(const TreeArgs& A, int i) {
    TreeSpan s;
    const int t1 = A.offsets[i + 1];
    s.t0 = A.offsets[i];
    s.row = A.rows ? A.rows[i] : i;
    s.live = s.t0 >= 0 && t1 > s.t0 && t1 <= A.total && s.row >= 0 && s.row < A.B;
    s.len = s.live ? t1 - s.t0 : 0;
    if (s.len > A.max_nodes) s.live = false;
    s.p = s.live && A.pos ? A.pos[s.row] : 0;
    if (s.p < 0 || s.p > kW) s.live = false;
    return s;
}

// One token past the carried query of a 16-lane row (lane l owns key elements
// 8l .. 8l+7 and, for l < V/8, value elements 8l .. 8l+7).
template <int KIND, int V, typename QT>
__device__ __forceinline__ void walk_token(const void* kp, size_t ke, const void* vp, size_t ve, const float* ap,
                                           size_t ae, float beta, int l, float (&x)[8], float (&acc)[8]) {
    constexpr bool KDA = KIND == SKSSM_KDA;
    float kf[8], vf[8], af[8];
    Vec8<QT>::unpack(Vec8<QT>::load(kp, ke + 8 * l), kf);
    Vec8<QT>::unpack(Vec8<QT>::load(vp, ve + (l < V / 8 ? 8 * l : 0)), vf);
    if (KDA) load8f(ap + ae * kK + 8 * l, af);
    else af[0] = ap[ae];
    const float s = beta * row_sum16(dot8(kf, x));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] = fmaf(s, vf[e], acc[e]);
        if (KIND != SKSSM_MAMBA2) x[e] = fmaf(-s, kf[e], x[e]);
        x[e] *= KDA ? af[e] : af[0];
    }
}

// Walks node n of a sequence back to the last flush; false if its path holds a
// parent that is none (the node is then left alone).
template <int KIND, int V, typename QT>
__device__ __forceinline__ bool walk(const TreeArgs& A, const TreeSpan& sp, int n, int h, int l, float (&x)[8],
                                     float (&acc)[8]) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    const int hk = h / A.share;
    Vec8<QT>::unpack(Vec8<QT>::load(A.q, (size_t(sp.t0 + n) * A.Hk + hk) * kK + 8 * l), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    bool ok = true;
    for (int m = n; m >= 0;) {
        const size_t t = size_t(sp.t0) + m;
        const size_t th = t * A.H + h;
        walk_token<KIND, V, QT>(A.k, (t * A.Hk + hk) * kK, A.v, th * V, A.a, th, DELTA ? A.beta[th] : 1.f, l, x, acc);
        const int up = A.parents[t];
        ok = ok && up < m && up >= -1;
        m = ok ? up : -1;
    }
    for (int j = sp.p - 1; j >= 0; --j) {
        const size_t at = (size_t(j) * A.H + h) * A.B + sp.row;
        walk_token<KIND, V, QT>(A.kbuf, ((size_t(j) * A.Hk + hk) * A.B + sp.row) * kK, A.vbuf, at * V, A.abuf, at,
                                DELTA ? A.bbuf[at] : 1.f, l, x, acc);
    }
    return ok;
}

}  // namespace

// Sketch heads: a 16-lane row per node, 16 nodes of one sequence and head per block.
template <int KIND, int V, typename QT>
__global__ __launch_bounds__(256) void tree_sketch_kernel(TreeArgs A, HeadTable T, int tiles) {
    const int seq = blockIdx.x / tiles % A.n_seqs;
    const int tile = blockIdx.x % tiles;
    const int at = A.n_dense + blockIdx.x / tiles / A.n_seqs;
    const int h = T.head[at], r = T.rank[at];
    const int l = threadIdx.x & 15, n = 16 * tile + (threadIdx.x >> 4);
    const TreeSpan sp = tree_span(A, seq);
    if (!sp.live || n >= sp.len) return;
    float x[8], acc[8];
    if (!walk<KIND, V, QT>(A, sp, n, h, l, x, acc)) return;
    const float* F = A.frames + size_t(T.frow[at]) * kK;
    const float* Z = A.Z + (size_t(T.zrow[at]) * A.B + size_t(sp.row) * r) * V;
    for (int i = 0; i < r; ++i) {
        float f[8], z[8];
        load8f(F + i * kK + 8 * l, f);
        load8f(Z + i * V + (l < V / 8 ? 8 * l : 0), z);
        const float c = row_sum16(dot8(f, x));
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(c, z[e], acc[e]);
    }
    if (l < V / 8) store8f(A.y + (size_t(sp.t0 + n) * A.H + h) * V + 8 * l, acc);
}

// Dense heads: a block per (sequence, head), MT tiles of 16 nodes.  The block's four
// waves take 32 key rows of the state each, in registers; x of all nodes goes through
// LDS to the fp32 matrix instruction, the waves' sums through LDS to the nodes' rows.
template <int KIND, int V, typename QT, int MT>
__global__ __launch_bounds__(256) void tree_dense_kernel(TreeArgs A, HeadTable T) {
    constexpr int CT = V / 16;  // column tiles
    constexpr int R = CT - 4;   // those past column 64
    constexpr int XS = kK + 4;
    constexpr int kX = MT * 16 * XS, kRed = 4 * 16 * V;
    __shared__ __align__(16) float lds[kX > kRed ? kX : kRed];
    const int seq = blockIdx.x % A.n_seqs;
    const int h = T.head[blockIdx.x / A.n_seqs];
    const TreeSpan sp = tree_span(A, seq);
    if (!sp.live) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int j = lane & 15, kk = lane >> 4;
    float s[8][CT];
    const float* S = A.S + (size_t(sp.row) * A.H + h) * (kK * V) + (32 * w + 8 * kk) * V;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float4 c = *reinterpret_cast<const float4*>(S + t * V + 4 * j);
        s[t][0] = c.x; s[t][1] = c.y; s[t][2] = c.z; s[t][3] = c.w;
#pragma unroll
        for (int i = 0; i < R; ++i) s[t][4 + i] = S[t * V + 64 + R * j + i];
    }
    const int rrow = threadIdx.x >> 4, l = threadIdx.x & 15;
    float acc[MT][8];
    bool ok[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int n = 16 * m + rrow;
        ok[m] = false;
        if (n < sp.len) {
            float x[8];
            ok[m] = walk<KIND, V, QT>(A, sp, n, h, l, x, acc[m]);
            store8f(lds + n * XS + 8 * l, x);
        }
    }
    __syncthreads();
    f32x4 d[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int c = 0; c < CT; ++c) d[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (16 * m >= sp.len) continue;
        float x[8];
        load8f(lds + (16 * m + j) * XS + 32 * w + 8 * kk, x);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) d[m][c] = mfma_16x16x4(x[t], s[t][c], d[m][c]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= sp.len) break;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float* to = lds + (w * 16 + 4 * kk + i) * V;
            *reinterpret_cast<float4*>(to + 4 * j) = make_float4(d[m][0][i], d[m][1][i], d[m][2][i], d[m][3][i]);
#pragma unroll
            for (int c = 0; c < R; ++c) to[64 + R * j + c] = d[m][4 + c][i];
        }
        __syncthreads();
        if (ok[m] && l < V / 8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float f[8];
                load8f(lds + (u * 16 + rrow) * V + 8 * l, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[m][e] += f[e];
            }
            store8f(A.y + (size_t(sp.t0 + 16 * m + rrow) * A.H + h) * V + 8 * l, acc[m]);
        }
    }
}

// The path to each sequence's accepted node, its tokens to the row's next window
// slots.  A block takes one sequence and some heads; the last block writes the new
// positions.
namespace {

struct AcceptArgs {
    void* kbuf;
    void* vbuf;
    float* abuf;
    float* bbuf;
    const int32_t* pos;
    int32_t* new_pos;
    const int32_t* rows;
    const int32_t* offsets;
    const int32_t* parents;
    const int32_t* accepted;
    const void* k;
    const void* v;
    const float* a;
    const float* beta;
    int B, n_seqs, total;
    int H, Hk, share, V, kda;
};

constexpr int kAcceptHeads = 8;

// The path of sequence i from its first token on, and its length; 0 where nothing
// is accepted or anything is out of range.
__device__ __forceinline__ int accept_path(const AcceptArgs& A, int i, int& row, int& t0, int (&path)[kW]) {
    const int t1 = A.offsets[i + 1];
    t0 = A.offsets[i];
    row = A.rows ? A.rows[i] : i;
    if (!(t0 >= 0 && t1 > t0 && t1 <= A.total && row >= 0 && row < A.B)) return 0;
    const int p = A.pos[row];
    int m = A.accepted[i];
    if (p < 0 || p > kW || m >= t1 - t0) return 0;
    int n = 0;
    while (m >= 0) {
        if (p + n >= kW) return 0;
        path[n++] = m;
        const int up = A.parents[t0 + m];
        if (up >= m || up < -1) return 0;
        m = up;
    }
    return n;
}

}  // namespace

template <typename QT>
__global__ __launch_bounds__(256) void tree_accept_kernel(AcceptArgs A, int groups) {
    __shared__ int path[kW], info[3];
    const int seq = blockIdx.x / groups, group = blockIdx.x % groups;
    if (seq == A.n_seqs) {  // positions: every row's old one, then those that grew
        for (int b = threadIdx.x; b < A.B; b += 256) A.new_pos[b] = A.pos[b];
        __syncthreads();
        for (int i = threadIdx.x; i < A.n_seqs; i += 256) {
            int pt[kW], row, t0;
            const int n = accept_path(A, i, row, t0, pt);
            if (n) A.new_pos[row] = A.pos[row] + n;
        }
        return;
    }
    if (threadIdx.x == 0) {
        int pt[kW], row, t0;
        const int n = accept_path(A, seq, row, t0, pt);
        for (int i = 0; i < n; ++i) path[i] = pt[n - 1 - i];
        info[0] = n;
        info[1] = row;
        info[2] = t0;
    }
    __syncthreads();
    const int n = info[0], row = info[1];
    const int h0 = group * kAcceptHeads, nh = min(kAcceptHeads, A.H - h0);
    if (n == 0) return;
    const int p = A.pos[row];
    const int VC = A.V / 8, KC = kK / 8;
    for (int i = 0; i < n; ++i) {
        const size_t t = size_t(info[2]) + path[i];
        const size_t slot = size_t(p + i);
        for (int e = threadIdx.x; e < nh * VC; e += 256) {
            const int h = h0 + e / VC, c = 8 * (e % VC);
            Vec8<QT>::store(A.vbuf, ((slot * A.H + h) * A.B + row) * A.V + c,
                            Vec8<QT>::load(A.v, (t * A.H + h) * A.V + c));
        }
        for (int e = threadIdx.x; e < nh * KC; e += 256) {
            const int h = h0 + e / KC, c = 8 * (e % KC);
            if (h % A.share == 0) {
                const int hk = h / A.share;
                Vec8<QT>::store(A.kbuf, ((slot * A.Hk + hk) * A.B + row) * kK + c,
                                Vec8<QT>::load(A.k, (t * A.Hk + hk) * kK + c));
            }
            if (A.kda) {
                float f[8];
                load8f(A.a + (t * A.H + h) * kK + c, f);
                store8f(A.abuf + ((slot * A.H + h) * A.B + row) * kK + c, f);
            }
        }
        for (int e = threadIdx.x; e < nh; e += 256) {
            const size_t to = (slot * A.H + h0 + e) * A.B + row, from = t * A.H + h0 + e;
            if (!A.kda) A.abuf[to] = A.a[from];
            if (A.bbuf) A.bbuf[to] = A.beta[from];
        }
    }
}

namespace {

template <int KIND, int V, typename QT, int MT>
hipError_t launch_dense(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    if (!launch_fits(double(a.n_seqs) * a.n_dense, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((tree_dense_kernel<KIND, V, QT, MT>), dim3(a.n_seqs * a.n_dense), dim3(256), 0, s, a, t);
    return hipGetLastError();
}

template <int KIND, int V, typename QT>
hipError_t launch_tree_t(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    const int tiles = (a.max_nodes + 15) / 16;
    const int sketch = a.H - a.n_dense;
    if (!launch_fits(double(a.n_seqs) * sketch * tiles, 256)) return hipErrorInvalidConfiguration;
    if (a.n_dense) {
        const hipError_t e = tiles == 1 ? launch_dense<KIND, V, QT, 1>(a, t, s)
                             : tiles == 2 ? launch_dense<KIND, V, QT, 2>(a, t, s)
                                          : launch_dense<KIND, V, QT, 4>(a, t, s);
        if (e != hipSuccess) return e;
    }
    if (sketch)
        hipLaunchKernelGGL((tree_sketch_kernel<KIND, V, QT>), dim3(a.n_seqs * sketch * tiles), dim3(256), 0, s, a, t,
                           tiles);
    return hipGetLastError();
}

template <int KIND, typename QT>
hipError_t launch_tree_v(int V, const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    switch (V) {
        case 64: return launch_tree_t<KIND, 64, QT>(a, t, s);
        case 80: return launch_tree_t<KIND, 80, QT>(a, t, s);
        case 96: return launch_tree_t<KIND, 96, QT>(a, t, s);
        case 112: return launch_tree_t<KIND, 112, QT>(a, t, s);
        case 128: return launch_tree_t<KIND, 128, QT>(a, t, s);
    }
    return hipErrorInvalidValue;
}

template <typename QT>
hipError_t launch_tree(int kind, int V, const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    switch (kind) {
        case SKSSM_MAMBA2: return launch_tree_v<SKSSM_MAMBA2, QT>(V, a, t, s);
        case SKSSM_GDN: return launch_tree_v<SKSSM_GDN, QT>(V, a, t, s);
        case SKSSM_KDA: return launch_tree_v<SKSSM_KDA, QT>(V, a, t, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

}  // namespace skssm

using namespace skssm;

extern "C" sketchssm_status sketchssm_tree_read(const sketchssm_plan* plan, const float* S, const float* Z,
                                                const float* frames, const void* kbuf, const void* vbuf,
                                                const float* abuf, const float* bbuf, const int32_t* pos,
                                                const int32_t* rows, const int32_t* offsets, int32_t n_seqs,
                                                int32_t total_nodes, int32_t max_nodes, const int32_t* parents,
                                                const void* q, const void* k, const void* v, const float* a,
                                                const float* beta, float* y, void* stream) {
    if (!plan) return SKSSM_EINVAL;
    const sketchssm_shape& sh = plan->shape;
    const bool delta = sh.kind != SKSSM_MAMBA2;
    if (n_seqs < 0 || total_nodes < 0 || max_nodes < 0) return SKSSM_EINVAL;
    if (max_nodes > kMaxNodes) return SKSSM_ESHAPE;
    if (!offsets || (plan->n_dense > 0 && !S)) return SKSSM_EINVAL;
    if (plan->n_dense < sh.H && (!Z || !frames)) return SKSSM_EINVAL;
    if (pos && (!kbuf || !vbuf || !abuf || (delta && !bbuf))) return SKSSM_EINVAL;
    if (!delta && (bbuf || beta)) return SKSSM_EINVAL;
    if (total_nodes > 0 && (!parents || !q || !k || !v || !a || !y || (delta && !beta))) return SKSSM_EINVAL;
    const void* ptrs[] = {S, Z, frames, kbuf, vbuf, abuf, bbuf, pos, rows, offsets, parents, q, k, v, a, beta, y};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return SKSSM_EALIGN;
    if (double(n_seqs) * sh.H * 4 >= 2147483648.0) return SKSSM_ESHAPE;  // block indices stay below 2^31
    if (n_seqs == 0 || total_nodes == 0 || max_nodes == 0) return SKSSM_OK;
    TreeArgs A;
    A.S = S;
    A.Z = Z;
    A.frames = frames;
    A.kbuf = kbuf;
    A.vbuf = vbuf;
    A.abuf = abuf;
    A.bbuf = bbuf;
    A.pos = pos;
    A.rows = rows;
    A.offsets = offsets;
    A.parents = parents;
    A.q = q;
    A.k = k;
    A.v = v;
    A.a = a;
    A.beta = beta;
    A.y = y;
    A.B = sh.B;
    A.n_seqs = n_seqs;
    A.total = total_nodes;
    A.max_nodes = max_nodes;
    A.H = sh.H;
    A.Hk = kq_heads_of(sh);
    A.share = sh.H / A.Hk;
    A.n_dense = plan->n_dense;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = sh.qkv == SKSSM_BF16 ? launch_tree<Bf16Tag>(sh.kind, sh.V, A, plan->table, s)
                                              : launch_tree<F32Tag>(sh.kind, sh.V, A, plan->table, s);
    if (e == hipErrorInvalidConfiguration) return SKSSM_ESHAPE;  // more threads than a launch takes
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}

extern "C" sketchssm_status sketchssm_tree_accept(const sketchssm_shape* shape, void* kbuf, void* vbuf, float* abuf,
                                                  float* bbuf, const int32_t* pos, int32_t* new_pos,
                                                  const int32_t* rows, const int32_t* offsets, int32_t n_seqs,
                                                  int32_t total_nodes, const int32_t* parents,
                                                  const int32_t* accepted, const void* k, const void* v,
                                                  const float* a, const float* beta, void* stream) {
    const sketchssm_status st = check_shape(shape);
    if (st != SKSSM_OK) return st;
    const bool delta = shape->kind != SKSSM_MAMBA2;
    if (n_seqs < 0 || total_nodes < 0) return SKSSM_EINVAL;
    if (!kbuf || !vbuf || !abuf || !pos || !new_pos || pos == new_pos || !offsets) return SKSSM_EINVAL;
    if (delta != (bbuf != nullptr)) return SKSSM_EINVAL;
    if (n_seqs > 0 && !accepted) return SKSSM_EINVAL;
    if (total_nodes > 0 && (!parents || !k || !v || !a || delta != (beta != nullptr))) return SKSSM_EINVAL;
    const void* ptrs[] = {kbuf, vbuf, abuf, bbuf, pos, new_pos, rows, offsets, parents, accepted, k, v, a, beta};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return SKSSM_EALIGN;
    const int groups = (shape->H + kAcceptHeads - 1) / kAcceptHeads;
    if (!launch_fits((double(n_seqs) + 1) * groups, 256)) return SKSSM_ESHAPE;
    AcceptArgs A;
    A.kbuf = kbuf;
    A.vbuf = vbuf;
    A.abuf = abuf;
    A.bbuf = bbuf;
    A.pos = pos;
    A.new_pos = new_pos;
    A.rows = rows;
    A.offsets = offsets;
    A.parents = parents;
    A.accepted = accepted;
    A.k = k;
    A.v = v;
    A.a = a;
    A.beta = beta;
    A.B = shape->B;
    A.n_seqs = total_nodes > 0 ? n_seqs : 0;
    A.total = total_nodes;
    A.H = shape->H;
    A.Hk = kq_heads_of(*shape);
    A.share = A.H / A.Hk;
    A.V = shape->V;
    A.kda = shape->kind == SKSSM_KDA;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(A.n_seqs * groups + 1);  // the last block: positions
    if (shape->qkv == SKSSM_BF16) hipLaunchKernelGGL((tree_accept_kernel<Bf16Tag>), grid, dim3(256), 0, s, A, groups);
    else hipLaunchKernelGGL((tree_accept_kernel<F32Tag>), grid, dim3(256), 0, s, A, groups);
    return hipGetLastError() == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
