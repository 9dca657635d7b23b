// Trees of drafted tokens over a row's cache on gfx950.  Per (sequence, head) a
// node n with ancestors (itself included) and the row's held-back window tokens
// before them:
//   walk, from n to the root and then from the window's last slot to its first:
//     s = k . x,  acc += beta s v,  x <- M^T x          (x = q_n at the start)
//   y = acc + S^T x (dense head)  |  acc + Z^T (F x) (sketch head)
// with Mamba-2 M = a I (beta = 1), GDN M = a (I - beta k k^T),
// KDA M = (I - beta k k^T) diag(a).  The products beta s make a matrix P, nodes by
// rows (window slots and nodes, 0 off a node's path), so that acc = P v is a matrix
// product, as is the state's or the sketch's part.
//
// Every float32 operand keeps its 24 bits: products are fp32, or bf16 with the
// float32 factor in three terms.  All sums are fp32.  Errors of y grow with the path, as its roundings' squares
// add up: in the 2-norm 10 of 2^-24 by that count for 80 tokens on a path, 3.9 measured.  On calls of some 10 nodes a
// path y was within 1.3e-7 of the same sums in 64 bits, relative to a call's largest y.
//
// Two kernels: the delta rule changes x at every token, so GDN and KDA walk
// (tree_kernel); Mamba-2 only scales it, so that s = decays times (q k) and all of it is
// products (tree_scan_kernel).
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
    int H, Hk;
    uint32_t per_share;  // 2^16 / (heads of a key head), rounded up: h / share is h per_share >> 16 below 256
    bool sketch;  // whether any head has one
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

// A tree's tokens as rows: 0 .. 15 the window's slots, 16 + n node n, and behind them
// two that end a path: `rows` behind the window's first slot, `rows` + 1 where a parent
// is none.  Every row says which one stands before it on a path.
struct __align__(16) RowInfo {
    int up;
    float beta, a;
    int pad;
};

// The delta rule's blocks: four waves, two by two, wave (wk, wc) with keys 64 wk .. 64 wk + 63
// and half wc of the columns.
constexpr int kTreeThreads = 256;

// A load at a per-lane 32-bit byte offset from a base that all lanes share.
template <typename T>
__device__ __forceinline__ T load_at(const void* base, uint32_t off) {
    return *reinterpret_cast<const T*>(static_cast<const char*>(base) + off);
}

// A block's rows of CH 16-byte chunks, through registers to LDS.  All loads are made,
// without a branch to wait behind (loads of existing rows alone have not been measured
// beside it): rows behind the window's or the tree's last one repeat it, and nothing
// points to them.
template <int CH, int MT>
struct RowRegs {
    static constexpr int PER = kTreeThreads / CH;  // rows per load of the block
    static constexpr int W = 16 / PER, N = W * (1 + MT);
    u32x4 r[N];

    __device__ __forceinline__ void load(const void* node, uint32_t nstep, int len, const void* win, uint32_t wstep,
                                         int p) {
        const int row = threadIdx.x / CH;
        const uint32_t c = 16 * (threadIdx.x % CH);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i < W) r[i] = load_at<u32x4>(win, max(min(i * PER + row, p - 1), 0) * wstep + c);
            else r[i] = load_at<u32x4>(node, min(i * PER - 16 + row, len - 1) * nstep + c);
        }
    }
    __device__ __forceinline__ void store(char* lds, int rows) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (int(i * PER + threadIdx.x / CH) < rows)
                *reinterpret_cast<u32x4*>(lds + (i * kTreeThreads + threadIdx.x) * 16) = r[i];
    }
};

// A matrix operand whose rows are V wide goes to lanes by columns: a wave has half of
// them, lane j of 16 columns C j .. C j + C-1 of that half, each in a column tile of its
// own, so that a row is one contiguous load.  Columns past V repeat others; their
// results are not stored.
template <int V>
struct Cols {
    static constexpr int C = (V / 16 + 1) / 2;
    static constexpr bool kFull = 2 * 16 * C == V;
    __device__ static __forceinline__ int first(int wc, int j) { return 16 * C * wc + C * j; }
    __device__ static __forceinline__ bool stored(int wc, int j, int c) { return kFull || first(wc, j) + c < V; }

    // of the row at element e of a shared base
    __device__ static __forceinline__ void load(const float* base, uint32_t e, int wc, int j, float (&f)[C]) {
        const int at = first(wc, j);
        if constexpr (C == 4) {
            const float4 v = load_at<float4>(base, 4 * (e + (kFull ? at : min(at, V - 4))));
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        } else if constexpr (C == 2) {
            const float2 v = load_at<float2>(base, 4 * (e + at));
            f[0] = v.x; f[1] = v.y;
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) f[c] = load_at<float>(base, 4 * (e + (kFull ? at + c : min(at + c, V - 1))));
        }
    }
    // from a buffer whose reads past the end give 0
    __device__ static __forceinline__ void load_buf(__amdgpu_buffer_rsrc_t rs, int voff, int soff, float (&f)[C]) {
        if constexpr (C == 4) {
            const uint4 v = buffer_load_u4_nt(rs, voff, soff);
            f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
            f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        } else if constexpr (C == 3) {
            typedef unsigned u32x3 __attribute__((ext_vector_type(3)));
            const u32x3 v = __builtin_bit_cast(u32x3, __builtin_amdgcn_raw_buffer_load_b96(rs, voff, soff, 2));
            f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z);
        } else {
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, voff, soff, 2));
            f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        }
    }
    __device__ static __forceinline__ void store(float* p, int wc, int j, const float (&f)[C]) {
        const int at = first(wc, j);
        if constexpr (C == 4) {
            if (stored(wc, j, 0)) *reinterpret_cast<float4*>(p + at) = make_float4(f[0], f[1], f[2], f[3]);
        } else if constexpr (C == 2) {
            *reinterpret_cast<float2*>(p + at) = make_float2(f[0], f[1]);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (stored(wc, j, c)) p[at + c] = f[c];
        }
    }
};

// The same columns of a row of values, as they are stored.
template <int V, typename QT>
struct ValueCols;
template <int V>
struct ValueCols<V, F32Tag> {
    static constexpr int C = Cols<V>::C;
    float f[C];
    __device__ __forceinline__ void load(const void* base, uint32_t e, int wc, int j) {
        Cols<V>::load(static_cast<const float*>(base), e, wc, j, f);
    }
    __device__ __forceinline__ float get(int c) const { return f[c]; }
    __device__ __forceinline__ void drop(int c) { f[c] = 0.f; }
    __device__ __forceinline__ void keep(bool on) {
#pragma unroll
        for (int c = 0; c < C; ++c) f[c] = on ? f[c] : 0.f;
    }
};
template <int V>
struct ValueCols<V, Bf16Tag> {
    static constexpr int C = Cols<V>::C;
    uint32_t u[(C + 1) / 2];
    __device__ __forceinline__ void keep(bool on) {
#pragma unroll
        for (int c = 0; c < (C + 1) / 2; ++c) u[c] = on ? u[c] : 0u;
    }
    __device__ __forceinline__ void load(const void* base, uint32_t e, int wc, int j) {
        const int at = Cols<V>::first(wc, j);
        if constexpr (C == 4) {
            const uint2 c = load_at<uint2>(base, 2 * (e + (Cols<V>::kFull ? at : min(at, V - 4))));
            u[0] = c.x;
            u[1] = c.y;
        } else if constexpr (C == 2) {
            u[0] = load_at<uint32_t>(base, 2 * (e + at));
        } else {
            auto one = [&](int c) { return uint32_t(load_at<uint16_t>(base, 2 * (e + min(at + c, V - 1)))); };
            u[0] = one(0) | one(1) << 16;
            u[1] = one(2);
        }
    }
    __device__ __forceinline__ float get(int c) const {
        return __uint_as_float(c % 2 ? u[c / 2] & 0xffff0000u : u[c / 2] << 16);
    }
    __device__ __forceinline__ void drop(int c) { u[c / 2] &= c % 2 ? 0xffffu : 0xffff0000u; }
};

// LDS of a block, by the call's largest tree.
template <int KIND, int V, typename QT>
struct TreeLds {
    static constexpr bool KDA = KIND == SKSSM_KDA;
    static constexpr int XS = kK + 4;  // row of x
    static constexpr int CS = 20;      // row of a sketch's coefficients
    static constexpr int kKey = kK * Vec8<QT>::kElemBytes;
    static constexpr int kCoef = 4 * 16 * CS * 4;
    static constexpr int kRed = 2 * 2 * Cols<V>::C * 64 * 8;
    int rows;  // window slots and nodes, a multiple of 4
    int lp;    // row of P, 4 apart in the banks from the next one
    int keys, dec, x, red, cs, p, info, good, flag, bytes;

    __host__ __device__ __forceinline__ TreeLds(int max_nodes, bool sketch) {
        rows = 16 + (max_nodes + 3) / 4 * 4;
        lp = 16 + (max_nodes + 15) / 16 * 16 + 4;
        keys = 0;
        dec = keys + (rows + 1) * kKey;
        x = dec + (KDA ? (rows + 1) * kK * 4 : 0);
        red = x + (KDA ? 0 : 16 * XS * 4);  // KDA: the sums take x's place
        cs = red + (KDA && 16 * XS * 4 > kRed ? 16 * XS * 4 : kRed);
        p = cs + (sketch ? kCoef : 0);
        info = p + (16 * lp + 4) * 4;
        good = info + (rows + 2) * int(sizeof(RowInfo));
        flag = good + (rows - 16) * 4;
        bytes = flag + 16;
    }
};

}  // namespace

// GDN and KDA: a block per (sequence, head), the heads of a sequence in turn, so that heads that
// share keys run side by side.  Per tile of 16 nodes: the walk, 16 lanes a node with 8 of the 128
// key elements each, its tokens from LDS; then x S (or F x, Z^T) and P v on the fp32 matrix units, keys
// halved over two waves and columns over the other two, the halves joined through LDS.
//   The state is read once, with streaming loads that are made before the walk and stay in
// registers over all tiles; three waves per SIMD hold it (plain loads and two waves: 102 us for the first
// call below, then 99.5).  Behind the walk, with four waves, they make no call faster.
//   Values go to P v behind the walk, two groups of 16 rows on their way.  Any that is no number is
// zeroed there and joins the nodes below it at the end, since 0 times it would not be 0.
//   Measured (calls behind each other, bf16 but where named; a kernel trace, which lets none overlap the
// next, has the first at 98 us): gdn, 128 trees of 16 nodes, 32 heads of 128 on the
// state: 92 us, 3.8 TB/s (loads of the state alone 51 us, everything but them 59: they overlap
// little, a block's loads and its walk take turns at three blocks per CU), kda 101; kda, 160 trees of 10 nodes on
// sketches of rank 10: 80 us, 2.3 TB/s, of which the walk's vector and LDS instructions take about 50
// (vector units busy 42%, LDS 23%), gdn 74, kda in float32 104; gdn, float32 chains of 8, 40 x 32 heads of 96: 23.5 us,
// 3.8 TB/s.
//   Without gain: eight waves a block, several heads a block with the next one's loads in flight (137 us
// for the gdn call), fp32 keys in LDS, blocks of a head on one XCD.
template <int KIND, int V, typename QT, int MT>
__global__ __launch_bounds__(kTreeThreads) __attribute__((amdgpu_waves_per_eu(3)))
void tree_kernel(TreeArgs A, HeadTable T) {
    typedef TreeLds<KIND, V, QT> Lds;
    typedef Cols<V> Co;
    typedef typename Vec8<QT>::raw_t Raw;
    constexpr bool KDA = Lds::KDA;
    constexpr int C = Co::C, E = Vec8<QT>::kElemBytes, XS = Lds::XS, CS = Lds::CS;
    extern __shared__ __align__(16) char lds[];
    const Lds Y(A.max_nodes, A.sketch);
    float* xs = reinterpret_cast<float*>(lds + Y.x);
    float* ps = reinterpret_cast<float*>(lds + Y.p);
    RowInfo* info = reinterpret_cast<RowInfo*>(lds + Y.info);
    int* flag = reinterpret_cast<int*>(lds + Y.flag);
    int* good = reinterpret_cast<int*>(lds + Y.good);  // whether a node has a path
    const int LP = Y.lp;

    const int seq = blockIdx.x / A.H, h = blockIdx.x % A.H;
    const int rank = T.rank[h], hk = int(uint32_t(h) * A.per_share >> 16);
    const TreeSpan sp = tree_span(A, seq);
    if (!sp.live) return;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, kk = lane >> 4;
    const int wk = w & 1, wc = w >> 1;
    const int rrow = tid >> 4, l = tid & 15;

    // ---- tokens to LDS ---------------------------------------------------------------
    // bases of this item's window entries and nodes, which all lanes share, and the
    // 32-bit strides of a slot and a node (a window array is below 2^32 bytes for every shape)
    const size_t win = size_t(h) * A.B + sp.row, kwin = size_t(hk) * A.B + sp.row;
    const size_t node = size_t(sp.t0) * A.H + h, knode = size_t(sp.t0) * A.Hk + hk;
    const uint32_t slot = uint32_t(A.H) * A.B, kslot = uint32_t(A.Hk) * A.B, step = A.H, kstep = A.Hk;
    const auto at_elem = [](const void* p, size_t e, int bytes) -> const void* {
        return static_cast<const char*>(p) + e * bytes;
    };
    const bool held = sp.p > 0;  // without a window its loads read the first node's
    const void* k_n = at_elem(A.k, knode * kK, E);
    const void* q_n = at_elem(A.q, knode * kK, E);
    const void* v_n = at_elem(A.v, node * V, E);
    const void* k_w = held ? at_elem(A.kbuf, kwin * kK, E) : k_n;
    const void* v_w = held ? at_elem(A.vbuf, win * V, E) : v_n;
    const float* a_n = A.a + node * (KDA ? kK : 1);
    const float* a_w = held ? A.abuf + win * (KDA ? kK : 1) : a_n;
    float s[16][C];  // keys 64 wk + 8 kk + (t < 8 ? t : 24 + t)
    {
        RowInfo in = {Y.rows + 1, 1.f, 1.f, 0};
        const int in_n = max(min(tid - 16, sp.len - 1), 0);
        const uint32_t in_off = 4 * (tid < 16 ? min(tid, max(sp.p - 1, 0)) * slot : in_n * step);
        const int par = load_at<int>(A.parents + sp.t0, 4 * in_n);
        const bool first16 = tid < 16 && held;
        if constexpr (!KDA) in.a = load_at<float>(first16 ? a_w : a_n, in_off);
        in.beta = load_at<float>(first16 ? A.bbuf + win : A.beta + node, in_off);
        RowRegs<kK * E / 16, MT> kr;
        RowRegs<kK * 4 / 16, MT> ar;
        kr.load(k_n, kstep * kK * E, sp.len, k_w, kslot * kK * E, sp.p);
        if constexpr (KDA) ar.load(a_n, step * kK * 4, sp.len, a_w, slot * kK * 4, sp.p);
        // the state is on its way while the first tile's queries are carried back
        if (rank == 0) {
            const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(A.S + (size_t(sp.row) * A.H + h) * (kK * V), kK * V * 4);
            const int voff = ((64 * wk + 8 * kk) * V + Co::first(wc, j)) * 4;
#pragma unroll
            for (int t = 0; t < 16; ++t) Co::load_buf(rs, voff, (t < 8 ? t : 24 + t) * V * 4, s[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (tid < Y.rows + 2) {
            // paths end behind slot 0, or at once without a window
            if (tid < 16) in.up = tid > 0 ? tid - 1 : Y.rows;
            else if (tid < Y.rows)
                in.up = par >= in_n || par < -1 ? Y.rows + 1 : par >= 0 ? 16 + par : held ? sp.p - 1 : Y.rows;
            else in = {tid, 0.f, 1.f, 0};
            info[tid] = in;
        }
        if (tid == 0) *flag = 0;
        kr.store(lds + Y.keys, Y.rows);
        if (tid < Lds::kKey / 16)
            *reinterpret_cast<u32x4*>(lds + Y.keys + Y.rows * Lds::kKey + 16 * tid) = u32x4{0u, 0u, 0u, 0u};
        if constexpr (KDA) {
            ar.store(lds + Y.dec, Y.rows);
            if (tid < kK) reinterpret_cast<float*>(lds + Y.dec)[Y.rows * kK + tid] = 1.f;
        }
    }
    __syncthreads();

    const int j_lane = j, kk_lane = kk;
#pragma unroll 1
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= sp.len) break;
        const int n0 = 16 * m, left = sp.len - n0;
        // a tile's addresses are formed anew: kept from tile to tile they take the registers
        // of another wave
        int j = j_lane, kk = kk_lane;
        if constexpr (MT > 1) asm volatile("" : "+v"(j), "+v"(kk));
        {
            // ---- the walk: 16 lanes a node, a wave's four until the last one ends --------
            const int n = n0 + min(rrow, left - 1), end = Y.rows;
            float x[8], g = 1.f;
            Vec8<QT>::unpack(load_at<Raw>(q_n, (n * kstep * kK + 8 * l) * E), x);
            float* pr = ps + rrow * LP;
            for (int i = l; i < LP; i += 16) pr[i] = 0.f;
            // a row's operands are read while the one before is in use; the rows that end
            // paths have the key 0 and lead to themselves
            struct Step {
                RowInfo in;
                Raw k;
                float a[8];
            };
            auto read = [&](Step& t, int row) {
                const int r = min(row, end);
                t.in = info[row];
                t.k = Vec8<QT>::load(lds + Y.keys, r * kK + 8 * l);
                if constexpr (KDA) load8f(reinterpret_cast<const float*>(lds + Y.dec) + r * kK + 8 * l, t.a);
            };
            auto take = [&](const Step& t, int row) {
                float k[8];
                Vec8<QT>::unpack(t.k, k);
                const bool on = row < end;
                const float c = on ? t.in.beta * row_sum16(dot8(k, x)) : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = fmaf(-c, k[e], x[e]);
                    if constexpr (KDA) x[e] *= t.a[e];
                }
                // lane 0 notes the product; the others, and ended paths, write behind P
                ps[on && l == 0 ? rrow * LP + row : 16 * LP] = g * c;
                if constexpr (!KDA) g *= t.in.a;
            };
            int row = rrow < left ? 16 + n : end;
            Step s0, s1;
            read(s0, row);
            while (__any(row < end)) {
                const int r1 = s0.in.up;
                read(s1, r1);
                take(s0, row);
                row = s1.in.up;
                read(s0, row);
                take(s1, r1);
            }
            if (l == 0 && rrow < left) good[n] = row == end;
            if constexpr (!KDA) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= g;
            }
            store8f(xs + rrow * XS + 8 * l, x);
        }
        __syncthreads();

        // ---- values: of each 16 rows 8 wk + 4 i + kk, i = 0, 1; NB groups on their way ---
        constexpr int NB = 2;
        ValueCols<V, QT> vr[NB][2];
        auto load_values = [&](int u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * wk + 4 * i + kk;
                if (u == 0) vr[u % NB][i].load(v_w, max(min(row, sp.p - 1), 0) * (slot * V), wc, j);
                else vr[u % NB][i].load(v_n, min(16 * (u - 1) + row, sp.len - 1) * (step * V), wc, j);
            }
        };
#pragma unroll
        for (int u = 0; u < NB; ++u) load_values(u);

        // ---- the state, or the sketch ------------------------------------------------
        f32x4 d[C];
#pragma unroll
        for (int c = 0; c < C; ++c) d[c] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (rank == 0) {
#pragma unroll
            for (int t8 = 0; t8 < 2; ++t8) {
                float x[8];
                load8f(xs + j * XS + 64 * wk + 32 * t8 + 8 * kk, x);
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int c = 0; c < C; ++c) d[c] = mfma_16x16x4(x[t], s[8 * t8 + t][c], d[c]);
            }
        } else {
            const float* F = A.frames + size_t(T.frow[h]) * kK;
            const float* Z = A.Z + (size_t(T.zrow[h]) * A.B + size_t(sp.row) * rank) * V;
            float x[8];  // node n0 + j, key elements 32 w + 8 kk ..
            load8f(xs + j * XS + 32 * w + 8 * kk, x);
            float* cs = reinterpret_cast<float*>(lds + Y.cs);
#pragma unroll 1
            for (int r0 = 0; r0 < rank; r0 += 16) {
                float z[2][C];
                const uint32_t fe = 4 * (min(r0 + j, rank - 1) * kK + 32 * w + 8 * kk);
                const f32x4 f0 = load_at<f32x4>(F, fe), f1 = load_at<f32x4>(F, fe + 16);
#pragma unroll
                for (int i = 0; i < 2; ++i) Co::load(Z, min(r0 + 8 * wk + 4 * i + kk, rank - 1) * V, wc, j, z[i]);
                f32x4 q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < 8; ++t) q = mfma_16x16x4(x[t], t < 4 ? f0[t & 3] : f1[t & 3], q);
                if (r0) __syncthreads();  // the coefficients before are read
#pragma unroll
                for (int i = 0; i < 4; ++i) cs[(w * 16 + 4 * kk + i) * CS + j] = q[i];
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 8 * wk + 4 * i + kk;
                    float y = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y += cs[(e * 16 + j) * CS + r];
                    const bool on = r0 + r < rank;
                    y = on ? y : 0.f;
#pragma unroll
                    for (int c = 0; c < C; ++c) d[c] = mfma_16x16x4(y, on ? z[i][c] : 0.f, d[c]);
                }
            }
        }

        // ---- the path's values ---------------------------------------------------------
        // a value that is no number must not meet the zeros of other nodes' rows: it is
        // left out of the products and joins the nodes below it at the end
        bool odd = false;
#pragma unroll
        for (int u = 0; u <= MT; ++u) {
            if (u > m + 1) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ValueCols<V, QT>& vu = vr[u % NB][i];
                vu.keep(8 * wk + 4 * i + kk + 16 * (u ? u - 1 : 0) < (u ? sp.len : sp.p));
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (!isfinite(vu.get(c))) {
                        odd = true;
                        vu.drop(c);
                    }
                const float pv = u || held ? ps[j * LP + 16 * u + 8 * wk + 4 * i + kk] : 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c) d[c] = mfma_16x16x4(pv, vu.get(c), d[c]);
            }
            if (u + NB <= MT && u + NB <= m + 1) load_values(u + NB);
        }
        if (odd) *flag = 1;
        // ---- the two halves of the keys: each wave keeps nodes 4 kk + 2 wk + i -------
        if constexpr (KDA) __syncthreads();  // x is read
        float* red = reinterpret_cast<float*>(lds + Y.red) + wc * (2 * C * 64 * 2) + 2 * lane;
#pragma unroll
        for (int c = 0; c < C; ++c)
            *reinterpret_cast<float2*>(red + (wk * C + c) * 128) =
                wk ? make_float2(d[c][0], d[c][1]) : make_float2(d[c][2], d[c][3]);
        __syncthreads();
        float y[2][C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float2 o = *reinterpret_cast<const float2*>(red + ((1 - wk) * C + c) * 128);
            y[0][c] = (wk ? d[c][2] : d[c][0]) + o.x;
            y[1][c] = (wk ? d[c][3] : d[c][1]) + o.y;
        }
        const bool fix = *flag;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rn = 4 * kk + 2 * wk + i, n = n0 + rn;
            if (rn < left && good[n]) {
                if (fix) {
                    for (int row = 16 + n; row < Y.rows; row = info[row].up) {
                        ValueCols<V, QT> f;
                        f.load(row < 16 ? v_w : v_n, (row < 16 ? row * slot : (row - 16) * step) * V, wc, j);
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            if (!isfinite(f.get(c))) y[i][c] = fmaf(ps[rn * LP + row], f.get(c), y[i][c]);
                    }
                }
                Co::store(A.y + (node + size_t(n) * A.H) * V, wc, j, y[i]);
            }
        }
        // KDA: the next x takes the sums' place; all: P is read above
        if (KDA || fix) __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Mamba-2: a wave per (sequence, head), up to 16 MT nodes.  Queries are not changed on
// the way but for the decays, so there is no walk over keys: y = g (q S) + P v with P the
// products q k times the decays between two tokens of a path, one path to a lane.  Nothing is
// shared by the waves of a block, so that none waits for another.
//   bf16 activations: q S, q F^T and P v are bf16 products of 32 keys or rows (16 cycles) with S, F
// and P in three terms (fp32 products take 32 cycles for 4 keys); Z, float32 on both sides, and
// float32 activations take the fp32 ones.
//   Bound by the latency of four loads that follow each other (lists, decays and frame, keys and values)
// at four waves per SIMD, beside vector units that are busy 40% of the time.  Measured: 192 trees
// of 8 nodes, 128 heads of 80 on sketches of rank 6: 83 us, 2.3 TB/s (68 us with its operands in the
// last-level cache); 64 trees of 47 nodes on the state: 161 us, 3.4 TB/s.  The same in float32, whose products are
// all fp32 ones: 148 and 322 us.
// A block per head as for the delta rule took 210 and 285 us; three waves with the keys loaded ahead of the
// sketch 106 where four without took 89.
// ---------------------------------------------------------------------------
namespace {

// What this lane wrote to LDS may be read by the wave's other lanes.
__device__ __forceinline__ void wave_lds() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight floats as three vectors of bf16 whose sum they are: the first 8 bits of each, the
// next 8 and the rest.  Products with bf16 numbers are then exact before they are summed.
__device__ __forceinline__ void split3(const float (&f)[8], bf16x8 (&out)[3]) {
    uint32_t u[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[2][3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = f[2 * i + e];
            a[e][0] = __float_as_uint(x);
            const float r = x - __uint_as_float(a[e][0] & 0xffff0000u);
            a[e][1] = __float_as_uint(r);
            a[e][2] = __float_as_uint(r - __uint_as_float(a[e][1] & 0xffff0000u));
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) u[s][i] = __builtin_amdgcn_perm(a[1][s], a[0][s], 0x07060302u);  // the upper halves
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) out[s] = __builtin_bit_cast(bf16x8, (u32x4{u[s][0], u[s][1], u[s][2], u[s][3]}));
}

// All V columns of a row for 16 lanes: lane j has 4j .. 4j+3 (tiles 0 .. 3) and, of those
// past 64, R j .. R j + R-1 (tiles 4 ..).
template <int V>
struct AllCols {
    static constexpr int CT = V / 16, R = CT - 4;
    __device__ static __forceinline__ void load(const float* base, uint32_t e, int j, float (&f)[CT]) {
        const f32x4 c = load_at<f32x4>(base, 4 * (e + 4 * j));
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = c[i];
        if constexpr (R == 4) {
            const f32x4 d = load_at<f32x4>(base, 4 * (e + 64 + 4 * j));
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 + i] = d[i];
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) f[4 + i] = load_at<float>(base, 4 * (e + 64 + R * j + i));
        }
    }
    __device__ static __forceinline__ void load(const uint16_t* base, uint32_t e, int j, float (&f)[CT]) {
        const uint2 c = load_at<uint2>(base, 2 * (e + 4 * j));
        const uint32_t u[2] = {c.x, c.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(i % 2 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
        if constexpr (R == 4) {
            const uint2 d = load_at<uint2>(base, 2 * (e + 64 + 4 * j));
            const uint32_t v[2] = {d.x, d.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 + i] = __uint_as_float(i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                f[4 + i] = __uint_as_float(uint32_t(load_at<uint16_t>(base, 2 * (e + 64 + R * j + i))) << 16);
        }
    }
    __device__ static __forceinline__ void store(float* p, int j, const float (&f)[CT]) {
        *reinterpret_cast<float4*>(p + 4 * j) = make_float4(f[0], f[1], f[2], f[3]);
        if constexpr (R == 4) {
            *reinterpret_cast<float4*>(p + 64 + 4 * j) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) p[64 + R * j + i] = f[4 + i];
        }
    }
};

// The same columns of a row of bf16 values, as they are stored.
template <int V>
struct PackedCols {
    static constexpr int CT = V / 16, R = CT - 4;
    static constexpr bool kPairs = R % 2 == 0;
    static constexpr int X = kPairs ? R / 2 : R;
    uint32_t w[2], x[X > 0 ? X : 1];
    __device__ __forceinline__ void load(const uint16_t* base, uint32_t e, int j) {
        const uint2 c = load_at<uint2>(base, 2 * (e + 4 * j));
        w[0] = c.x;
        w[1] = c.y;
        const uint32_t at = 2 * (e + 64 + R * j);
        if constexpr (R == 4) {
            const uint2 d = load_at<uint2>(base, at);
            x[0] = d.x;
            x[1] = d.y;
        } else if constexpr (R == 2) {
            x[0] = load_at<uint32_t>(base, at);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) x[i] = load_at<uint16_t>(base, at + 2 * i);
        }
    }
    __device__ __forceinline__ void clear() {
        w[0] = w[1] = 0u;
#pragma unroll
        for (int i = 0; i < X; ++i) x[i] = 0u;
    }
    // column tile c of two rows, the first one's in the lower half
    __device__ static __forceinline__ uint32_t pair(const PackedCols& a, const PackedCols& b, int c) {
        const bool tail = c >= 4;
        const int i = tail ? (kPairs ? (c - 4) / 2 : c - 4) : c / 2;
        const bool upper = tail && !kPairs ? false : c % 2 != 0;
        return __builtin_amdgcn_perm(tail ? b.x[i] : b.w[i], tail ? a.x[i] : a.w[i], upper ? 0x07060302 : 0x05040100);
    }
};

// LDS of one wave.
template <int MT>
struct ScanLds {
    static constexpr int ROWS = 16 + 16 * MT;
    static constexpr int CS = 20;  // row of a sketch's coefficients
    // P of tile m: its 16 nodes by the window and the nodes of tiles 0 .. m; rows 4 apart in the banks
    __host__ __device__ static constexpr int row_p(int m) { return 16 * m + 36; }
    __host__ __device__ static constexpr int tile_p(int m) { return 128 * m * (m - 1) + 576 * m; }
    float p[tile_p(MT)];
    float c[16 * CS];
    float a[ROWS];
    int up[ROWS];  // the row before on a path: -1 none, -2 no path
    float ws[16];  // decays behind each window slot
    float gs[16 * MT];  // a node's decays to the tree's root
    // the nodes of its path.  Two words, and 32-bit shifts wherever they are read: a 64-bit shift
    // by a lane's amount that lay in the wave's last vector register has shifted by another one.
    uint2 path[16 * MT];
};

}  // namespace

// Waves of a block: their LDS stays below 64 KB.
__host__ __device__ constexpr int scan_waves(int MT) { return MT == 4 ? 2 : 4; }

// Waves per SIMD the registers are made for: the sums take MT V / 4 of them and the loads in flight
// V / 2 more.  Chosen by time, which is mostly, but not always, one wave fewer where that would spill: at four waves
// and up to 16 nodes V = 80 keeps 9 registers in scratch (float32 13, and 3 at V = 96).  Measured with 64 heads in
// bf16; float32 goes by the same rule, not measured for itself (us, more | fewer waves):
// 12 nodes on the sketch V = 128 67 | 47, V = 112 81 | 52, V = 96 40 | 40, V = 80 38 | 41; 31 nodes on the state V = 128
// 121 | 77, V = 96 78 | 53, V = 80 44.5 | 46; 64 nodes V = 128 140 | 124, V = 112 154 | 123, V = 96 95 | 105.
__host__ __device__ constexpr int scan_per_simd(int V, int MT) {
    return MT == 1 ? (V <= 96 ? 4 : 3) : MT == 2 ? (V <= 80 ? 3 : 2) : V <= 96 ? 2 : 1;
}

template <int V, typename QT, int MT>
__global__ __launch_bounds__(64 * scan_waves(MT)) __attribute__((amdgpu_waves_per_eu(scan_per_simd(V, MT))))
void tree_scan_kernel(TreeArgs A, HeadTable T) {
    typedef AllCols<V> Co;
    typedef typename Vec8<QT>::raw_t Raw;
    typedef typename std::conditional<std::is_same<QT, Bf16Tag>::value, uint16_t, float>::type Elem;
    constexpr int CT = Co::CT, E = Vec8<QT>::kElemBytes, CS = ScanLds<MT>::CS;
    constexpr bool BF = E == 2;
    __shared__ __align__(16) ScanLds<MT> lds[scan_waves(MT)];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    ScanLds<MT>& Y = lds[w];
    const int item = blockIdx.x * scan_waves(MT) + w;
    const int seq = item / A.H, h = item - seq * A.H;
    if (seq >= A.n_seqs) return;
    const TreeSpan sp = tree_span(A, seq);
    if (!sp.live) return;
    const int rank = T.rank[h], hk = int(uint32_t(h) * A.per_share >> 16);
    const int j = lane & 15, kk = lane >> 4;
    const bool held = sp.p > 0;
    const uint32_t slot = uint32_t(A.H) * A.B, kslot = uint32_t(A.Hk) * A.B, step = A.H, kstep = A.Hk;
    const size_t win = size_t(h) * A.B + sp.row, node = size_t(sp.t0) * A.H + h;
    const size_t kwin = size_t(hk) * A.B + sp.row, knode = size_t(sp.t0) * A.Hk + hk;
    const char* q_n = static_cast<const char*>(A.q) + knode * kK * E;
    const char* k_n = static_cast<const char*>(A.k) + knode * kK * E;
    const char* k_w = held ? static_cast<const char*>(A.kbuf) + kwin * kK * E : k_n;
    const Elem* v_n = static_cast<const Elem*>(A.v) + node * V;
    const Elem* v_w = held ? static_cast<const Elem*>(A.vbuf) + win * V : v_n;

    Raw q0[4];  // the first tile's queries
    if constexpr (MT == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            q0[c] = load_at<Raw>(q_n, (uint32_t(min(j, sp.len - 1)) * kstep * kK + 32 * c + 8 * kk) * E);
    }
    // ---- rows: decays, and which one stands before --------------------------------------
#pragma unroll
    for (int r0 = 0; r0 < 16 * (1 + MT); r0 += 64) {
        const int r = r0 + lane;
        const int n = max(min(r - 16, sp.len - 1), 0);
        const bool in_w = r < 16 && held;
        const float a = load_at<float>(in_w ? A.abuf + win : A.a + node,
                                       4 * (r < 16 ? min(r, max(sp.p - 1, 0)) * slot : n * step));
        const int par = load_at<int>(A.parents + sp.t0, 4 * n);
        if (r < 16 * (1 + MT)) {
            Y.a[r] = a;
            Y.up[r] = par >= n || par < -1 ? -2 : par < 0 ? -1 : 16 + par;
        }
    }

    // ---- decays behind each window slot and of the whole window; between a node, a lane
    // each, and its ancestors ------------------------------------------------------------
    wave_lds();
    float all = 1.f;
    for (int i = sp.p - 1; i >= 0; --i) {
        if (lane == 0) Y.ws[i] = all;
        all *= Y.a[i];
    }
    if (lane < 16 * MT) {
        float* pr = Y.p + ScanLds<MT>::tile_p(lane >> 4) + j * ScanLds<MT>::row_p(lane >> 4);
        float g = 1.f;
        uint2 path = make_uint2(0u, 0u);
        int row = lane < sp.len ? 16 + lane : -2;
        while (row >= 0) {
            pr[row] = g;
            const uint32_t bit = 1u << (row - 16 & 31);
            path.x |= row < 48 ? bit : 0u;
            path.y |= row < 48 ? 0u : bit;
            g *= Y.a[row];
            row = Y.up[row];
        }
        Y.gs[lane] = g;
        Y.path[lane] = row == -1 ? path : make_uint2(0u, 0u);
    }

    // ---- q times the state, or the sketch ----------------------------------------------
    f32x4 d[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) d[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto q_at = [&](int m, int key) {  // node 16 m + j, key elements key + 8 kk ..
        return load_at<Raw>(q_n, (uint32_t(min(16 * m + j, sp.len - 1)) * kstep * kK + key + 8 * kk) * E);
    };
    // d += q f^T over 32 keys
    auto multiply = [&](const Raw& q, const float (&f)[8], f32x4 d) {
        if constexpr (BF) {
            bf16x8 t[3];
            split3(f, t);
#pragma unroll
            for (int s = 0; s < 3; ++s)
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, q.w), t[s], d, 0, 0, 0);
        } else {
            float x[8];
            Vec8<QT>::unpack(q, x);
#pragma unroll
            for (int t = 0; t < 8; ++t) d = mfma_16x16x4(x[t], f[t], d);
        }
        return d;
    };
    if (rank == 0) {
        const float* S = A.S + (size_t(sp.row) * A.H + h) * (kK * V);
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            float s[8][CT];
#pragma unroll
            for (int t = 0; t < 8; ++t) Co::load(S, (32 * b + 8 * kk + t) * V, j, s[t]);
            Raw q[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) q[m] = q_at(m, 32 * b);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < CT; ++c) {  // one column tile's terms at a time
                float f[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) f[t] = s[t][c];
                if constexpr (BF) {
                    bf16x8 t[3];
                    split3(f, t);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        if (16 * m < sp.len)
#pragma unroll
                            for (int e = 0; e < 3; ++e)
                                d[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, q[m].w), t[e],
                                                                                  d[m][c], 0, 0, 0);
                } else {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        if (16 * m < sp.len) d[m][c] = multiply(q[m], f, d[m][c]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else {
        const float* F = A.frames + size_t(T.frow[h]) * kK;
        const float* Z = A.Z + (size_t(T.zrow[h]) * A.B + size_t(sp.row) * rank) * V;
#pragma unroll 1
        for (int r0 = 0; r0 < rank; r0 += 16) {
            float f[4][8], z[4][CT];
            const uint32_t fe = 4 * (min(r0 + j, rank - 1) * kK + 8 * kk);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const f32x4 f0 = load_at<f32x4>(F, fe + 128 * b), f1 = load_at<f32x4>(F, fe + 128 * b + 16);
#pragma unroll
                for (int t = 0; t < 8; ++t) f[b][t] = t < 4 ? f0[t & 3] : f1[t & 3];
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) Co::load(Z, min(r0 + 4 * s + kk, rank - 1) * V, j, z[s]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (16 * m >= sp.len) continue;
                __builtin_amdgcn_sched_barrier(0);
                f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    c = multiply(MT == 1 ? q0[b] : q_at(m, 32 * b), f[b], c);
                    __builtin_amdgcn_sched_barrier(0);
                }
                wave_lds();
#pragma unroll
                for (int i = 0; i < 4; ++i) Y.c[(4 * kk + i) * CS + j] = c[i];
                wave_lds();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (r0 + 4 * s >= rank) continue;
                    const bool on = r0 + 4 * s + kk < rank;
                    const float y = on ? Y.c[j * CS + 4 * s + kk] : 0.f;
#pragma unroll
                    for (int t = 0; t < CT; ++t) d[m][t] = mfma_16x16x4(y, on ? z[s][t] : 0.f, d[m][t]);
                }
            }
        }
    }

#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int n0 = 16 * m, left = sp.len - n0;
        if (left <= 0) break;
        float* pt = Y.p + ScanLds<MT>::tile_p(m);
        const int LP = ScanLds<MT>::row_p(m);
        wave_lds();
        float gr[4];
        uint2 pa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gr[i] = Y.gs[n0 + 4 * kk + i];
            pa[i] = Y.path[n0 + 4 * kk + i];
            const float g = all * gr[i];
#pragma unroll
            for (int c = 0; c < CT; ++c) d[m][c][i] *= g;
        }
        // ---- P: products q k, each with the decays between its tokens -----------------------
        Raw qf[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) qf[c] = MT == 1 ? q0[c] : q_at(m, 32 * c);
        // group u: the window's slots, then the tiles' nodes
        auto k_at = [&](int u, int c) {
            const uint32_t r = u ? min(16 * (u - 1) + j, sp.len - 1) * kstep : max(min(j, sp.p - 1), 0) * kslot;
            return load_at<Raw>(u ? k_n : k_w, (r * kK + 32 * c + 8 * kk) * E);
        };
        auto note = [&](int u, const f32x4& g) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float& p = pt[(4 * kk + i) * LP + 16 * u + j];
                const int r = 16 * (u - 1) + j;
                const float f = u ? p * g[i] : gr[i] * Y.ws[j] * g[i];
                p = (u == 0 ? j < sp.p : ((r < 32 ? pa[i].x : pa[i].y) >> (r & 31) & 1u) != 0u) ? f : 0.f;
            }
        };
        // ... and times the values.  One that is no number must not meet the zeros of other
        // nodes' rows: it is left out here and joins the nodes below it afterwards
        bool odd = false;
        if constexpr (BF) {
            // two groups at a time: their 32 rows are one product's, with P in three terms
#pragma unroll
            for (int s = 0; s < (MT + 2) / 2; ++s) {
                if (2 * s > m + 1) break;
                const bool two = 2 * s < m + 1;
                __builtin_amdgcn_sched_barrier(0);
                Raw kf[2][4];
                PackedCols<V> v[8];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (!e || two) kf[e][c] = k_at(2 * s + e, c);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int u = 2 * s + t / 4, r = 4 * kk + t % 4;
                    if (t >= 4 && !two) v[t].clear();
                    else if (u) v[t].load(v_n, min(16 * (u - 1) + r, sp.len - 1) * (step * V), j);
                    else v[t].load(v_w, max(min(r, sp.p - 1), 0) * (slot * V), j);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e && !two) continue;
                    f32x4 g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, qf[c].w),
                                                                    __builtin_bit_cast(bf16x8, kf[e][c].w), g, 0, 0, 0);
                    note(2 * s + e, g);
                }
                wave_lds();
                const float* pr = pt + j * LP + 32 * s + 4 * kk;
                const f32x4 p0 = *reinterpret_cast<const f32x4*>(pr);
                const f32x4 p1 = two ? *reinterpret_cast<const f32x4*>(pr + 16) : f32x4{0.f, 0.f, 0.f, 0.f};
                const float pv[8] = {p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]};
                bf16x8 a[3];
                split3(pv, a);
                u32x4 b[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int t = 0; t < 4; ++t) b[c][t] = PackedCols<V>::pair(v[2 * t], v[2 * t + 1], c);
                // times zeros they add up to no number if any is none
                f32x4 nul = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    nul = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, (u32x4{0u, 0u, 0u, 0u})),
                                                                  __builtin_bit_cast(bf16x8, b[c]), nul, 0, 0, 0);
                if (__any(!(nul[0] == 0.f))) {
                    odd = true;
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t u = b[c][t];
                            b[c][t] = ((u & 0x7f80u) == 0x7f80u ? 0u : u & 0xffffu) |
                                      ((u & 0x7f800000u) == 0x7f800000u ? 0u : u & 0xffff0000u);
                        }
                }
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        d[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[e], __builtin_bit_cast(bf16x8, b[c]), d[m][c],
                                                                          0, 0, 0);
            }
        } else {
#pragma unroll
            for (int u = 0; u <= m + 1; ++u) {
                if (u == 0 && !held) continue;
                __builtin_amdgcn_sched_barrier(0);
                const int rows = u ? min(16, sp.len - 16 * (u - 1)) : sp.p;
                Raw kf[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) kf[c] = k_at(u, c);
                float v[4][CT];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = min(4 * s + kk, rows - 1);
                    if (u) Co::load(v_n, (16 * (u - 1) + r) * (step * V), j, v[s]);
                    else Co::load(v_w, r * (slot * V), j, v[s]);
                }
                f32x4 g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float k[8];
                    Vec8<QT>::unpack(kf[c], k);
                    g = multiply(qf[c], k, g);
                }
                note(u, g);
                wave_lds();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (4 * s >= rows) continue;
                    const bool on = 4 * s + kk < rows;
                    const float pv = pt[j * LP + 16 * u + 4 * s + kk];
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const bool fin = isfinite(v[s][c]);
                        odd = odd || !fin;
                        d[m][c] = mfma_16x16x4(pv, on && fin ? v[s][c] : 0.f, d[m][c]);
                    }
                }
            }
        }
        const bool fix = __any(odd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rn = 4 * kk + i, n = n0 + rn;
            if (rn >= left || !(pa[i].x | pa[i].y)) continue;
            float y[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) y[c] = d[m][c][i];
            if (fix) {
                auto join = [&](int row) {
                    float f[CT];
                    if (row < 16) Co::load(v_w, row * (slot * V), j, f);
                    else Co::load(v_n, (row - 16) * (step * V), j, f);
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        if (!isfinite(f[c])) y[c] = fmaf(pt[rn * LP + row], f[c], y[c]);
                };
                for (int row = 16 + n; row >= 0; row = Y.up[row]) join(row);
                for (int row = 0; row < sp.p; ++row) join(row);
            }
            Co::store(A.y + (node + size_t(n) * A.H) * V, j, y);
        }
    }
}

// The path to each sequence's accepted node, its tokens to the row's next window slots: copies,
// exact.  A block takes one sequence and 8 heads; the first block, whose paths take longest, writes the
// new positions.
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
constexpr int kStaged = 256;  // parents of a tree's first nodes, in LDS

// The path to accepted node m of a tree of len nodes, last node first, and its length; 0 where
// nothing is accepted, anything is out of range or the window has no room behind p tokens.
template <typename Parent>
__device__ __forceinline__ int accept_path(int m, int len, int p, Parent&& parent, int* path) {
    if (p < 0 || p > kW || m >= len) return 0;
    int n = 0;
    while (m >= 0) {
        if (p + n >= kW) return 0;
        if (path) path[n] = m;
        ++n;
        const int up = parent(m);
        if (up >= m || up < -1) return 0;
        m = up;
    }
    return n;
}

struct AcceptSpan {
    int row, t0, len;  // len 0: idle
};

__device__ __forceinline__ AcceptSpan accept_span(const AcceptArgs& A, int i) {
    AcceptSpan s;
    const int t1 = A.offsets[i + 1];
    s.t0 = A.offsets[i];
    s.row = A.rows ? A.rows[i] : i;
    s.len = s.t0 >= 0 && t1 > s.t0 && t1 <= A.total && s.row >= 0 && s.row < A.B ? t1 - s.t0 : 0;
    return s;
}

}  // namespace

// Bound by latency: the path has to be known before its tokens can be read.  A tree's parents
// come to LDS in one load, and a block's threads take all tokens of its heads at once.  192 sequences, 128 heads of
// 80, 4 of 8 tokens each (17 MB): 10.0 us on the GPU, one sequence of 32 KDA heads 3.9 us.  Heads a block, for
// those two, measured beside each other on another day: 4 10.6 and 3.4, 8 9.9 and 3.4, 16 9.2 and 4.1.
template <typename QT>
__global__ __launch_bounds__(256) void tree_accept_kernel(AcceptArgs A, int groups) {
    __shared__ int path[kW], staged[kStaged], n_path;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {  // positions: every row's old one, then those that grew
        for (int b = tid; b < A.B; b += 256) A.new_pos[b] = A.pos[b];
        __syncthreads();
        for (int i = tid; i < A.n_seqs; i += 256) {
            const AcceptSpan sp = accept_span(A, i);
            if (!sp.len) continue;
            const int n = accept_path(A.accepted[i], sp.len, A.pos[sp.row],
                                      [&](int m) { return A.parents[sp.t0 + m]; }, nullptr);
            if (n) A.new_pos[sp.row] = A.pos[sp.row] + n;
        }
        return;
    }
    const int seq = (blockIdx.x - 1) / groups, group = (blockIdx.x - 1) % groups;
    const AcceptSpan sp = accept_span(A, seq);
    if (!sp.len) return;
    const int row = sp.row, p = A.pos[row], last = A.accepted[seq];
    if (tid < sp.len) staged[tid] = A.parents[sp.t0 + tid];
    __syncthreads();
    if (tid == 0)
        n_path = accept_path(last, sp.len, p, [&](int m) { return m < kStaged ? staged[m] : A.parents[sp.t0 + m]; }, path);
    __syncthreads();
    const int n = n_path;
    if (n == 0) return;
    const int h0 = group * kAcceptHeads, nh = min(kAcceptHeads, A.H - h0);
    const auto token = [&](int i) { return size_t(sp.t0) + path[n - 1 - i]; };  // the path's i-th from the root
    const int VC = A.V / 8, KC = kK / 8;
    for (int e = tid; e < n * nh * VC; e += 256) {
        const int i = e / (nh * VC), r = e - i * (nh * VC), h = h0 + r / VC, c = 8 * (r % VC);
        Vec8<QT>::store(A.vbuf, ((size_t(p + i) * A.H + h) * A.B + row) * A.V + c,
                        Vec8<QT>::load(A.v, (token(i) * A.H + h) * A.V + c));
    }
    for (int e = tid; e < n * nh * KC; e += 256) {
        const int i = e / (nh * KC), r = e - i * (nh * KC), h = h0 + r / KC, c = 8 * (r % KC);
        const size_t t = token(i), slot = size_t(p + i);
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
    for (int e = tid; e < n * nh; e += 256) {
        const int i = e / nh, h = h0 + e - i * nh;
        const size_t to = (size_t(p + i) * A.H + h) * A.B + row, from = token(i) * A.H + h;
        if (!A.kda) A.abuf[to] = A.a[from];
        if (A.bbuf) A.bbuf[to] = A.beta[from];
    }
}

namespace {

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

template <int KIND, int V, typename QT, int MT>
hipError_t launch_tree_m(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    const int bytes = TreeLds<KIND, V, QT>(a.max_nodes, a.sketch).bytes;
    if (!launch_fits(double(a.n_seqs) * a.H, kTreeThreads)) return hipErrorInvalidConfiguration;
    if (bytes > 65536) {
        // the kernel's limit is shared with calls of other threads: the most it ever takes, so that none lowers it
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(tree_kernel<KIND, V, QT, MT>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 TreeLds<KIND, V, QT>(16 * MT, true).bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((tree_kernel<KIND, V, QT, MT>), dim3(a.n_seqs * a.H), dim3(kTreeThreads), bytes, s, a, t);
    return hipGetLastError();
}

template <int V, typename QT, int MT>
hipError_t launch_scan_m(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    constexpr int waves = scan_waves(MT);
    const double blocks = (double(a.n_seqs) * a.H + waves - 1) / waves;
    if (!launch_fits(blocks, 64 * waves)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((tree_scan_kernel<V, QT, MT>), dim3(uint32_t(blocks)), dim3(64 * waves), 0, s, a, t);
    return hipGetLastError();
}

// Forms for up to 16, 32 and 64 nodes, by the caller's bound: registers and LDS go by it.  What a bound
// above the largest tree costs (us by bound): Mamba-2 sketch, 12 nodes, 16 66, 32 84, 64 112; KDA sketch, 17 nodes,
// 17 78, 32 94, 64 161 (tokens in LDS); GDN chains of 12, 16 24.8, 32 27.4, 64 31.6; GDN on the state, 25
// nodes, 32 98, 64 98.
template <int KIND, int V, typename QT>
hipError_t launch_tree_t(const TreeArgs& a, const HeadTable& t, hipStream_t s) {
    if constexpr (KIND == SKSSM_MAMBA2) {
        if (a.max_nodes <= 16) return launch_scan_m<V, QT, 1>(a, t, s);
        if (a.max_nodes <= 32) return launch_scan_m<V, QT, 2>(a, t, s);
        return launch_scan_m<V, QT, 4>(a, t, s);
    } else {
        if (a.max_nodes <= 16) return launch_tree_m<KIND, V, QT, 1>(a, t, s);
        if (a.max_nodes <= 32) return launch_tree_m<KIND, V, QT, 2>(a, t, s);
        return launch_tree_m<KIND, V, QT, 4>(a, t, s);
    }
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
    // a node's y may be written before another one's inputs are read
    const size_t T = total_nodes, elem = sh.qkv == SKSSM_BF16 ? 2 : 4, y_bytes = T * sh.H * sh.V * 4;
    const size_t k_bytes = T * kq_heads_of(sh) * kK * elem, a_elems = T * sh.H * (sh.kind == SKSSM_KDA ? kK : 1);
    if (overlap(y, y_bytes, q, k_bytes) || overlap(y, y_bytes, k, k_bytes) ||
        overlap(y, y_bytes, v, T * sh.H * sh.V * elem) || overlap(y, y_bytes, a, a_elems * 4) ||
        overlap(y, y_bytes, beta, beta ? T * sh.H * 4 : 0))
        return SKSSM_EINVAL;
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
    const uint32_t share = uint32_t(sh.H / A.Hk);
    A.per_share = (65536 + share - 1) / share;
    A.sketch = plan->n_dense < sh.H;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = sh.qkv == SKSSM_BF16 ? launch_tree<Bf16Tag>(sh.kind, sh.V, A, plan->by_head, s)
                                              : launch_tree<F32Tag>(sh.kind, sh.V, A, plan->by_head, s);
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
    if (!kbuf || !vbuf || !abuf || !pos || !new_pos || !offsets) return SKSSM_EINVAL;
    if (delta != (bbuf != nullptr)) return SKSSM_EINVAL;
    if (n_seqs > 0 && !accepted) return SKSSM_EINVAL;
    if (total_nodes > 0 && (!parents || !k || !v || !a || delta != (beta != nullptr))) return SKSSM_EINVAL;
    const void* ptrs[] = {kbuf, vbuf, abuf, bbuf, pos, new_pos, rows, offsets, parents, accepted, k, v, a, beta};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return SKSSM_EALIGN;
    if (overlap(pos, size_t(shape->B) * 4, new_pos, size_t(shape->B) * 4)) return SKSSM_EINVAL;
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
    const dim3 grid(A.n_seqs * groups + 1);  // the first block: positions
    if (shape->qkv == SKSSM_BF16) hipLaunchKernelGGL((tree_accept_kernel<Bf16Tag>), grid, dim3(256), 0, s, A, groups);
    else hipLaunchKernelGGL((tree_accept_kernel<F32Tag>), grid, dim3(256), 0, s, A, groups);
    return hipGetLastError() == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
