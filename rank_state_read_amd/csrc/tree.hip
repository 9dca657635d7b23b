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

// A tree's tokens as rows: 0 .. 15 the window's slots, 16 + n node n.  `up` of a row is
// the row before it on a path, -1 at the window's start, kNoRow where a parent is none.
constexpr int kNoRow = -2;

// Rows of CH 16-byte chunks on their way to LDS, through registers.  Rows behind the
// window's or the tree's last one repeat that one: nothing points to them.
template <int CH, int MT>
struct RowRegs {
    static constexpr int PER = 256 / CH;  // rows per load of the block
    static constexpr int N = 16 * (1 + MT) / PER;
    u32x4 r[N];

    __device__ __forceinline__ void load(const char* win, size_t wstride, int p, const char* node, size_t nstride,
                                         int len) {
        const int row = threadIdx.x / CH;
        const size_t c = 16 * (threadIdx.x % CH);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r[i] = u32x4{0u, 0u, 0u, 0u};
            if (i * PER < 16) {
                if (i * PER < p) r[i] = *reinterpret_cast<const u32x4*>(win + min(i * PER + row, p - 1) * wstride + c);
            } else if (i * PER - 16 < len) {
                r[i] = *reinterpret_cast<const u32x4*>(node + min(i * PER - 16 + row, len - 1) * nstride + c);
            }
        }
    }
    __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<u32x4*>(lds + (i * 256 + threadIdx.x) * 16) = r[i];
    }
};

// One lane's part of a matrix operand whose rows are V wide: of one row the columns
// 4j .. 4j+3 (column tiles 0 .. 3) and, of those past 64, R j .. R j + R-1 (tiles 4 ..),
// so that a row's first 64 values are one load of 16 lanes.
template <int V>
__device__ __forceinline__ void load_cols(const float* p, int j, float (&f)[V / 16]) {
    constexpr int R = V / 16 - 4;
    const float4 c = *reinterpret_cast<const float4*>(p + 4 * j);
    f[0] = c.x; f[1] = c.y; f[2] = c.z; f[3] = c.w;
#pragma unroll
    for (int i = 0; i < R; ++i) f[4 + i] = p[64 + R * j + i];
}

// The same of a row of the qkv dtype, as it is stored.
template <int V, typename QT>
struct ValueCols;
template <int V>
struct ValueCols<V, F32Tag> {
    float f[V / 16];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < V / 16; ++c) f[c] = 0.f;
    }
    __device__ __forceinline__ void load(const void* base, size_t e, int j) {
        load_cols<V>(static_cast<const float*>(base) + e, j, f);
    }
    __device__ __forceinline__ float get(int c) const { return f[c]; }
    __device__ __forceinline__ void drop(int c) { f[c] = 0.f; }
};
template <int V>
struct ValueCols<V, Bf16Tag> {
    static constexpr int R = V / 16 - 4;
    uint32_t u[2 + (R + 1) / 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < 2 + (R + 1) / 2; ++c) u[c] = 0u;
    }
    __device__ __forceinline__ void load(const void* base, size_t e, int j) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + e;
        const uint2 c = *reinterpret_cast<const uint2*>(p + 4 * j);
        u[0] = c.x;
        u[1] = c.y;
        p += 64 + R * j;
        if constexpr (R == 4) {
            const uint2 d = *reinterpret_cast<const uint2*>(p);
            u[2] = d.x;
            u[3] = d.y;
        } else if constexpr (R == 2) {
            u[2] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (R > 0) {
            u[2] = p[0];
            if constexpr (R == 3) {
                u[2] |= uint32_t(p[1]) << 16;
                u[3] = p[2];
            }
        }
    }
    __device__ __forceinline__ float get(int c) const {
        return __uint_as_float(c % 2 ? u[c / 2] & 0xffff0000u : u[c / 2] << 16);
    }
    __device__ __forceinline__ void drop(int c) { u[c / 2] &= c % 2 ? 0xffffu : 0xffff0000u; }
};

template <int KIND, int V, typename QT, int MT>
struct TreeLds {
    static constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    static constexpr bool KDA = KIND == SKSSM_KDA;
    static constexpr int NT = 16 * MT, L = 16 + NT;
    static constexpr int LP = L + 4;   // row of P; 4 rows apart in the banks
    static constexpr int XS = kK + 4;  // row of x
    static constexpr int kKeyBytes = kK * Vec8<QT>::kElemBytes;
    // what the walk uses, then the waves' sums over it
    static constexpr int keys = 0;
    static constexpr int dec = keys + (DELTA ? L * kKeyBytes : 0);
    static constexpr int x = dec + (KDA ? L * kK * 4 : 0);
    static constexpr int gram = x;                                             // Mamba-2
    static constexpr int cs = DELTA ? keys : x + NT * LP * 4;                  // coefficients of 16 ranks
    static constexpr int cs_end = cs + 4 * 16 * 20 * 4;
    static constexpr int x_end = x + NT * XS * 4;
    static constexpr int walk_end = DELTA ? x_end : cs_end;
    static constexpr int red_end = 4 * 16 * V * 4;
    static constexpr int p = walk_end > red_end ? walk_end : red_end;
    static constexpr int a = p + NT * LP * 4;  // decays; Mamba-2: its window's become products
    static constexpr int beta = a + L * 4;
    static constexpr int up = beta + L * 4;
    static constexpr int g = up + L * 4;       // per node: Mamba-2's product of decays
    static constexpr int flag = g + NT * 4;
    static constexpr int bytes = flag + 16;
    static_assert(!DELTA || cs_end <= x, "the coefficients' sums fit the keys' place");
};

}  // namespace

// A block per (sequence, head), MT tiles of 16 nodes; dense heads first.
template <int KIND, int V, typename QT, int MT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(MT == 1 ? (V <= 96 ? 4 : 3) : 2)))
void tree_kernel(TreeArgs A, HeadTable T) {
    typedef TreeLds<KIND, V, QT, MT> Lds;
    constexpr bool DELTA = Lds::DELTA, KDA = Lds::KDA;
    constexpr int CT = V / 16, R = CT - 4, E = Vec8<QT>::kElemBytes;
    constexpr int L = Lds::L, LP = Lds::LP, XS = Lds::XS, NT = Lds::NT;
    extern __shared__ __align__(16) char lds[];
    float* red = reinterpret_cast<float*>(lds);
    float* xs = reinterpret_cast<float*>(lds + Lds::x);
    float* gram = reinterpret_cast<float*>(lds + Lds::gram);
    float* ps = reinterpret_cast<float*>(lds + Lds::p);
    float* as = reinterpret_cast<float*>(lds + Lds::a);
    float* bs = reinterpret_cast<float*>(lds + Lds::beta);
    int* up = reinterpret_cast<int*>(lds + Lds::up);
    float* gs = reinterpret_cast<float*>(lds + Lds::g);
    int* flag = reinterpret_cast<int*>(lds + Lds::flag);

    const int seq = blockIdx.x % A.n_seqs, at = blockIdx.x / A.n_seqs;
    const int h = T.head[at], rank = T.rank[at], hk = h / A.share;
    const TreeSpan sp = tree_span(A, seq);
    if (!sp.live) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int j = lane & 15, kk = lane >> 4;
    const int rrow = tid >> 4, l = tid & 15;

    // ---- loads, in the order of their use --------------------------------------
    const size_t win = size_t(h) * A.B + sp.row, wslot = size_t(A.H) * A.B;  // an item's window entry, a slot
    const size_t node = size_t(sp.t0) * A.H + h;
    const size_t kwin = size_t(hk) * A.B + sp.row, kslot = size_t(A.Hk) * A.B;
    const size_t knode = size_t(sp.t0) * A.Hk + hk;
    float a_r = 1.f, b_r = 1.f;
    int up_r = kNoRow;
    if (tid < 16) {
        if (tid < sp.p) {
            if (!KDA) a_r = A.abuf[win + tid * wslot];
            if (DELTA) b_r = A.bbuf[win + tid * wslot];
            up_r = tid - 1;
        }
    } else if (tid < L && tid - 16 < sp.len) {
        const int n = tid - 16;
        if (!KDA) a_r = A.a[node + size_t(n) * A.H];
        if (DELTA) b_r = A.beta[node + size_t(n) * A.H];
        const int up = A.parents[sp.t0 + n];
        up_r = up >= n || up < -1 ? kNoRow : up < 0 ? sp.p - 1 : 16 + up;
    }
    RowRegs<kK * E / 16, MT> kr;
    RowRegs<kK * 4 / 16, MT> ar;
    typename Vec8<QT>::raw_t qr[MT];
    if constexpr (DELTA) {
        kr.load(static_cast<const char*>(A.kbuf) + kwin * kK * E, kslot * kK * E, sp.p,
                static_cast<const char*>(A.k) + knode * kK * E, size_t(A.Hk) * kK * E, sp.len);
        if constexpr (KDA)
            ar.load(reinterpret_cast<const char*>(A.abuf) + win * kK * 4, wslot * kK * 4, sp.p,
                    reinterpret_cast<const char*>(A.a) + node * kK * 4, size_t(A.H) * kK * 4, sp.len);
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (16 * m < sp.len)
                qr[m] = Vec8<QT>::load(A.q, (knode + size_t(min(16 * m + rrow, sp.len - 1)) * A.Hk) * kK + 8 * l);
    }
    // values: of each 16 rows this wave takes 4
    ValueCols<V, QT> vr[1 + MT];
#pragma unroll
    for (int u = 0; u <= MT; ++u) {
        const int row = 4 * w + kk + 16 * (u > 0 ? u - 1 : 0);
        const bool on = row < (u ? sp.len : sp.p);
        vr[u].zero();
        if (on)
            vr[u].load(u ? A.v : A.vbuf, (u ? node + size_t(row) * A.H : win + row * wslot) * V, j);
    }
    float s[8][CT];
    if (rank == 0) {
        const float* S = A.S + (size_t(sp.row) * A.H + h) * (kK * V) + (32 * w + 8 * kk) * V;
#pragma unroll
        for (int t = 0; t < 8; ++t) load_cols<V>(S + t * V, j, s[t]);
    }
    __builtin_amdgcn_sched_barrier(0);

    // ---- to LDS --------------------------------------------------------------------
    if (tid < L) {
        as[tid] = a_r;
        bs[tid] = b_r;
        up[tid] = up_r;
    }
    if (tid == 0) *flag = 0;
    for (int i = tid; i < NT * LP; i += 256) ps[i] = 0.f;
    if constexpr (DELTA) {
        kr.store(lds + Lds::keys);
        if constexpr (KDA) ar.store(lds + Lds::dec);
    } else {  // products q k of all nodes and rows
        for (int tile = w; tile < MT * (1 + MT); tile += 4) {
            const int m = tile / (1 + MT), u = tile % (1 + MT);
            if (16 * m >= sp.len || (u ? 16 * (u - 1) >= sp.len : sp.p == 0)) continue;
            const size_t qe = (knode + size_t(min(16 * m + j, sp.len - 1)) * A.Hk) * kK + 8 * kk;
            const void* kb = u ? A.k : A.kbuf;
            const size_t ke = (u ? knode + size_t(min(16 * (u - 1) + j, sp.len - 1)) * A.Hk
                                 : kwin + min(j, sp.p - 1) * kslot) * kK + 8 * kk;
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const auto qv = Vec8<QT>::load(A.q, qe + 32 * c);
                const auto kv = Vec8<QT>::load(kb, ke + 32 * c);
                if constexpr (E == 2) {
                    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, qv.w),
                                                                __builtin_bit_cast(bf16x8, kv.w), d, 0, 0, 0);
                } else {
                    float qf[8], kf[8];
                    Vec8<QT>::unpack(qv, qf);
                    Vec8<QT>::unpack(kv, kf);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d = mfma_16x16x4(qf[e], kf[e], d);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) gram[(16 * m + 4 * kk + i) * LP + 16 * u + j] = d[i];
        }
    }
    __syncthreads();

    // a value that is no number must not meet the zeros of other nodes' rows: it is
    // left out of the products and joins the nodes below it at the end
    bool odd = false;
#pragma unroll
    for (int u = 0; u <= MT; ++u)
#pragma unroll
        for (int c = 0; c < CT; ++c)
            if (!isfinite(vr[u].get(c))) {
                odd = true;
                vr[u].drop(c);
            }
    if (odd) *flag = 1;

    // ---- the walk --------------------------------------------------------------------
    bool ok[MT];
    if constexpr (DELTA) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int n = 16 * m + rrow;
            ok[m] = false;
            if (n < sp.len) {
                float x[8], g = 1.f;
                Vec8<QT>::unpack(qr[m], x);
                int row = 16 + n;
                while (row >= 0) {
                    float kf[8];
                    Vec8<QT>::unpack(Vec8<QT>::load(lds + Lds::keys, row * kK + 8 * l), kf);
                    const float c = bs[row] * row_sum16(dot8(kf, x));
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = fmaf(-c, kf[e], x[e]);
                    if constexpr (KDA) {
                        float af[8];
                        load8f(reinterpret_cast<const float*>(lds + Lds::dec) + row * kK + 8 * l, af);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= af[e];
                    }
                    if (l == 0) ps[n * LP + row] = g * c;
                    if constexpr (!KDA) g *= as[row];
                    row = up[row];
                }
                ok[m] = row == -1;
                if constexpr (!KDA) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= g;
                }
                store8f(xs + n * XS + 8 * l, x);
            }
        }
    } else {
        if (tid < sp.len) {  // the nodes of the path
            float g = 1.f;
            int row = 16 + tid;
            while (row >= 16) {
                ps[tid * LP + row] = g * gram[tid * LP + row];
                g *= as[row];
                row = up[row];
            }
            gs[tid] = g;
            if (row == kNoRow) up[16 + tid] = kNoRow;  // (a walk that meets this entry meets the other one too)
        }
    }
    __syncthreads();
    f32x4 d[MT][CT];
    if constexpr (!DELTA) {
#pragma unroll
        for (int m = 0; m < MT; ++m) ok[m] = 16 * m + rrow < sp.len && up[16 + 16 * m + rrow] != kNoRow;
    }
    // products of the decays from each slot's successor to the window's end
    float after = 1.f, all = 1.f;
    if constexpr (!DELTA) {
        for (int i = sp.p - 1; i >= 0; --i) {
            if (i == 4 * w + kk) after = all;
            all *= as[i];
        }
    }

    // ---- the state, or the sketch ----------------------------------------------------
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) d[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto x_of = [&](int m, float (&x)[8]) {  // node 16 m + j, key elements 32 w + 8 kk ..
        if constexpr (DELTA) load8f(xs + (16 * m + j) * XS + 32 * w + 8 * kk, x);
        else Vec8<QT>::unpack(Vec8<QT>::load(A.q, (knode + size_t(min(16 * m + j, sp.len - 1)) * A.Hk) * kK + 32 * w + 8 * kk), x);
    };
    if (rank == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (16 * m >= sp.len) continue;
            float x[8];
            x_of(m, x);
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int c = 0; c < CT; ++c) d[m][c] = mfma_16x16x4(x[t], s[t][c], d[m][c]);
        }
    } else {
        const float* F = A.frames + size_t(T.frow[at]) * kK;
        const float* Z = A.Z + (size_t(T.zrow[at]) * A.B + size_t(sp.row) * rank) * V;
        f32x4 c[MT];
#pragma unroll 1
        for (int r0 = 0; r0 < rank; r0 += 16) {
            float f[8], z[CT];
            load8f(F + min(r0 + j, rank - 1) * kK + 32 * w + 8 * kk, f);
#pragma unroll
            for (int i = 0; i < CT; ++i) z[i] = 0.f;
            if (r0 + 4 * w + kk < rank) load_cols<V>(Z + (r0 + 4 * w + kk) * V, j, z);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                c[m] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (16 * m >= sp.len) continue;
                float x[8];
                x_of(m, x);
#pragma unroll
                for (int t = 0; t < 8; ++t) c[m] = mfma_16x16x4(x[t], f[t], c[m]);
            }
            // c's sums over the waves' keys
            float* cs = reinterpret_cast<float*>(lds + Lds::cs);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (16 * m >= sp.len) break;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) cs[(w * 16 + 4 * kk + i) * 20 + j] = c[m][i];
                __syncthreads();
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) y += cs[(i * 16 + j) * 20 + 4 * w + kk];
                if (r0 + 4 * w + kk >= rank) y = 0.f;
#pragma unroll
                for (int i = 0; i < CT; ++i) d[m][i] = mfma_16x16x4(y, z[i], d[m][i]);
            }
        }
    }

    // ---- the path's values, the waves' sums ---------------------------------------
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= sp.len) break;
        if constexpr (!DELTA) {  // what the state gave decays over the whole path
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = all * gs[16 * m + 4 * kk + i];
#pragma unroll
                for (int c = 0; c < CT; ++c) d[m][c][i] *= g;
            }
        }
#pragma unroll
        for (int u = 0; u <= MT; ++u) {
            if (u ? 16 * (u - 1) >= sp.len : sp.p == 0) continue;
            const int n = 16 * m + j, row = 16 * u + 4 * w + kk;
            float pv;
            if (!DELTA && u == 0) {
                pv = row < sp.p && n < sp.len ? gs[n] * after * gram[n * LP + row] : 0.f;
                ps[n * LP + row] = pv;
            } else {
                pv = ps[n * LP + row];
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) d[m][c] = mfma_16x16x4(pv, vr[u].get(c), d[m][c]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= sp.len) break;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float* to = red + (w * 16 + 4 * kk + i) * V;
            *reinterpret_cast<float4*>(to + 4 * j) = make_float4(d[m][0][i], d[m][1][i], d[m][2][i], d[m][3][i]);
#pragma unroll
            for (int c = 0; c < R; ++c) to[64 + R * j + c] = d[m][4 + c][i];
        }
        __syncthreads();
        if (ok[m] && l < V / 8) {
            const int n = 16 * m + rrow;
            float y[8];
            load8f(red + rrow * V + 8 * l, y);
#pragma unroll
            for (int u = 1; u < 4; ++u) {
                float f[8];
                load8f(red + (u * 16 + rrow) * V + 8 * l, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += f[e];
            }
            if (*flag) {
                for (int row = 16 + n; row >= 0; row = up[row]) {
                    float f[8];
                    Vec8<QT>::unpack(row < 16 ? Vec8<QT>::load(A.vbuf, (win + row * wslot) * V + 8 * l)
                                              : Vec8<QT>::load(A.v, (node + size_t(row - 16) * A.H) * V + 8 * l), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!isfinite(f[e])) y[e] = fmaf(ps[n * LP + row], f[e], y[e]);
                }
            }
            store8f(A.y + (node + size_t(n) * A.H) * V + 8 * l, y);
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
hipError_t launch_tree_m(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    constexpr int bytes = TreeLds<KIND, V, QT, MT>::bytes;
    if (!launch_fits(double(a.n_seqs) * a.H, 256)) return hipErrorInvalidConfiguration;
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(tree_kernel<KIND, V, QT, MT>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((tree_kernel<KIND, V, QT, MT>), dim3(a.n_seqs * a.H), dim3(256), bytes, s, a, t);
    return hipGetLastError();
}

template <int KIND, int V, typename QT>
hipError_t launch_tree_t(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    if (a.max_nodes <= 16) return launch_tree_m<KIND, V, QT, 1>(a, t, s);
    if (a.max_nodes <= 32) return launch_tree_m<KIND, V, QT, 2>(a, t, s);
    return launch_tree_m<KIND, V, QT, 4>(a, t, s);
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
