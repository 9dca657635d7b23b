// Prefill of ragged prompts for gfx950: the state update in chunks of C = 32
// tokens on the matrix cores.
//
// Per sequence and head, within a chunk that starts at state S, with gamma_i the
// decays' product up to token i, gamma_ij that after j up to i and sigma_j that
// after j to the chunk's end:
//   A_ij = beta_i gamma_ij (k_i . k_j)  (j < i),   P_ij = gamma_ij (q_i . k_j)  (j <= i)
//   T    = (I + A)^-1 diag(beta)                    (Mamba-2: w = v instead)
//   w    = T (v - gamma K S),   y = gamma Q S + P w,   S <- gamma_C S + K^T (sigma w)
//
// Two launches.  T and P depend on a chunk's own tokens alone, so the first
// forms them for all chunks of all heads at once and leaves them in the
// workspace; the second walks a sequence's chunks in order with the state in
// registers.  Value columns are independent of each other: one wave owns 16 of
// them for all 128 key rows, and nothing it computes has to reach another wave.
//
// Products run on the bf16 matrix instruction (16x16x32, fp32 sums) and keep
// fp32 precision: an fp32 operand x is written as hi + mid + lo, three bf16
// numbers of 8 significant bits each.  q, k, v in bf16 are exact operands, so
// their products with an fp32 operand take three instructions, products of two
// fp32 operands six (the terms below 2^-24 are left out).  The fp32 matrix
// instruction has 1/16 of the bf16 rate.
//
// The accumulator layout (lane l, register r <-> row 4 (l/16) + r, column l % 16)
// becomes the next product's B operand (lane l <-> 8 consecutive rows from
// 8 (l/16), column l % 16) without leaving the lane: rows 4 q + r of the two
// tiles of a 32-row group stand for group rows 8 q + r and 8 q + 4 + r, which the
// A operand's rows follow.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "ragged.h"
#include "sketchssm_internal.h"

namespace skssm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kC = 32;                       // tokens per chunk
constexpr int kFrag = 64 * 16;               // one A operand of a wave, bytes
constexpr int kTri = 3 * 2 * kFrag;          // T or P: three terms, two row tiles
constexpr int kGam = 2 * kC * 4;             // gamma, sigma

__device__ __forceinline__ f32x4 mfma_bf16(const uint4& a, const uint4& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// x = t[0] + t[1] + t[2], each of 8 consecutive values rounded to bf16.
struct Split3 {
    uint4 t[3];
};

__device__ __forceinline__ Split3 split3(const float* f) {
    uint32_t u[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x0 = f[2 * i], x1 = f[2 * i + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x0, x1}), bf16x2));
            u[p][i] = h;
            x0 -= __uint_as_float(h << 16);
            x1 -= __uint_as_float(h & 0xffff0000u);
        }
    }
    Split3 s;
#pragma unroll
    for (int p = 0; p < 3; ++p) s.t[p] = make_uint4(u[p][0], u[p][1], u[p][2], u[p][3]);
    return s;
}

// Row i of row tile m of a 32-row group (see above).
__device__ __forceinline__ int tile_row(int m, int i) { return 8 * (i >> 2) + 4 * m + (i & 3); }

// A workspace record: P, then T (delta rule), then gamma and sigma.
template <int KIND>
struct Record {
    static constexpr bool delta = KIND != SKSSM_MAMBA2;
    static constexpr int p = 0;
    static constexpr int t = kTri;
    static constexpr int g = delta ? 2 * kTri : kTri;
    static constexpr int bytes = g + kGam;
};

__host__ __device__ inline long prefill_slots(long total, int n_seqs) { return total / kC + n_seqs; }

// Chunk c of a sequence has slot off / C + seq + c of the workspace: a sequence
// of len tokens has at most (off + len) / C - off / C + 1 chunks, so sequences
// that do not overlap never share a slot.
__device__ __forceinline__ long first_slot(int t0, int seq) { return long(t0) / kC + seq; }

}  // namespace

// ---------------------------------------------------------------------------
// T and P of every chunk and head: one wave per (slot, head).
// ---------------------------------------------------------------------------
constexpr int kPrepWaves = 4;
constexpr int kGS = kC + 4;  // row stride of a C x C tile in LDS, floats

template <int KIND>
__global__ __launch_bounds__(kPrepWaves * 64) void prep_kernel(RaggedArgs A, char* ws) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    typedef Record<KIND> R;
    __shared__ __align__(16) float tiles[kPrepWaves][2][kC * kGS];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const long task = long(blockIdx.x) * kPrepWaves + w;
    const long slot = task / A.H;
    const int h = int(task - slot * A.H), hk = h / A.share;

    // the sequence and chunk of this slot, if any
    int seq = -1, t0 = 0, clen = 0;
    for (int s0 = 0; s0 < A.n_seqs && seq < 0; s0 += 64) {
        const int s = s0 + lane;
        bool hit = false;
        int tc = 0, cl = 0;
        if (s < A.n_seqs) {
            const SeqSpan sp = seq_span(A, s);
            const long c = slot - first_slot(sp.t0, s);
            hit = sp.live && c >= 0 && c * kC < sp.len;
            tc = sp.t0 + int(c) * kC;
            cl = min(kC, sp.len - int(c) * kC);
        }
        const unsigned long long m = __ballot(hit);
        if (m) {
            const int f = __ffsll(m) - 1;
            seq = s0 + f;
            t0 = __shfl(tc, f, 64);
            clen = __shfl(cl, f, 64);
        }
    }
    if (seq < 0) return;  // no wave waits for another one below

    // k_i . k_j and q_i . k_j: exact products of bf16 values, fp32 sums
    float* gk = tiles[w][0];
    float* gq = tiles[w][1];
    {
        uint4 kf[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const size_t row = (size_t(t0) + min(tile_row(m, lr), clen - 1)) * A.Hk + hk;
            const char* src = static_cast<const char*>(A.k) + (row * kK + 8 * lq) * 2;
#pragma unroll
            for (int s = 0; s < 4; ++s) kf[m][s] = *reinterpret_cast<const uint4*>(src + 64 * s);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const size_t row = (size_t(t0) + min(tile_row(m, lr), clen - 1)) * A.Hk + hk;
            const char* src = static_cast<const char*>(A.q) + (row * kK + 8 * lq) * 2;
            uint4 qf[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) qf[s] = *reinterpret_cast<const uint4*>(src + 64 * s);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                f32x4 dk = {0.f, 0.f, 0.f, 0.f}, dq = dk;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (DELTA) dk = mfma_bf16(kf[m][s], kf[n][s], dk);
                    dq = mfma_bf16(qf[s], kf[n][s], dq);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = (8 * lq + 4 * m + r) * kGS + tile_row(n, lr);
                    if (DELTA) gk[at] = dk[r];
                    gq[at] = dq[r];
                }
            }
        }
    }
    const int j = lane & 31;
    const bool valid = j < clen;
    const size_t tj = size_t(t0) + (valid ? j : 0);
    const float aj = valid ? A.a[tj * A.H + h] : 1.f;
    const float bj = !DELTA ? 1.f : valid ? A.beta[tj * A.H + h] : 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    // column j: the decays' products after token j, one factor at a time (a decay
    // may be 0, so nothing is divided); lanes 0..31 take -A, lanes 32..63 take P
    float* gt = lane < 32 ? gk : gq;
    float d = 0.f, gam = 0.f, run = 1.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        const float ai = __shfl(aj, i, 64);
        const float bi = DELTA ? __shfl(bj, i, 64) : 1.f;
        d = i == j ? 1.f : d * ai;
        run *= ai;
        gam = i == j ? run : gam;
        if (DELTA || lane >= 32) {
            const float g = gt[i * kGS + j] * d;
            gt[i * kGS + j] = lane >= 32 ? (valid ? g : 0.f) : (i > j ? -bi * g : 0.f);
        }
    }
    char* rec = ws + task * R::bytes;
    if (lane < 32) reinterpret_cast<float*>(rec + R::g)[j] = gam;
    else reinterpret_cast<float*>(rec + R::g)[lane] = valid ? d : 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    // column j of (I + A)^-1 by forward substitution, one lane per column
    if (DELTA && lane < 32) {
        float x[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float s0 = i == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const f32x4 n4 = *reinterpret_cast<const f32x4*>(gk + i * kGS + m);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < i) {
                        if (e & 1) s1 = fmaf(n4[e], x[m + e], s1);
                        else s0 = fmaf(n4[e], x[m + e], s0);
                    }
            }
            x[i] = s0 + s1;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kC; ++i) gk[i * kGS + j] = x[i] * bj;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    // both as A operands
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float f[8];
        load8f(gq + tile_row(m, lr) * kGS + 8 * lq, f);
        const Split3 p = split3(f);
#pragma unroll
        for (int e = 0; e < 3; ++e) *reinterpret_cast<uint4*>(rec + R::p + (2 * e + m) * kFrag + lane * 16) = p.t[e];
        if (DELTA) {
            load8f(gk + tile_row(m, lr) * kGS + 8 * lq, f);
            const Split3 t = split3(f);
#pragma unroll
            for (int e = 0; e < 3; ++e)
                *reinterpret_cast<uint4*>(rec + R::t + (2 * e + m) * kFrag + lane * 16) = t.t[e];
        }
    }
}

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks: NW waves of 16 value columns each.
// ---------------------------------------------------------------------------
template <int KIND>
struct ScanStage {  // one chunk's shared operands in LDS, bytes
    static constexpr int k = 0;
    static constexpr int q = kC * kK * 2;
    static constexpr int rec = 2 * kC * kK * 2;
    static constexpr int bytes = rec + Record<KIND>::bytes;
};

// Granule of 16 bytes g of token row r sits at granule g ^ row_swizzle(r): the
// rows of a tile then start in different banks.
__device__ __forceinline__ int row_swizzle(int r) { return (r & 3) | (((r >> 3) & 3) << 2); }

// A wave's lanes each fetch 16 (4) bytes, which land one lane behind the other.
__device__ __forceinline__ void load_to_lds16(const char* src, char* dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void load_to_lds4(const char* src, char* dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)dst, 4, 0, 0);
}

// Six products of two three-term operands, the small ones first.
__device__ __forceinline__ f32x4 mfma_33(const uint4* a, const Split3& b, f32x4 c) {
    c = mfma_bf16(a[2], b.t[0], c);
    c = mfma_bf16(a[0], b.t[2], c);
    c = mfma_bf16(a[1], b.t[1], c);
    c = mfma_bf16(a[1], b.t[0], c);
    c = mfma_bf16(a[0], b.t[1], c);
    return mfma_bf16(a[0], b.t[0], c);
}

// Three products of an exact operand with a three-term one.
__device__ __forceinline__ f32x4 mfma_13(const uint4& a, const Split3& b, f32x4 c) {
    c = mfma_bf16(a, b.t[2], c);
    c = mfma_bf16(a, b.t[1], c);
    return mfma_bf16(a, b.t[0], c);
}

template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void scan_kernel(RaggedArgs A, const char* ws, int V, int slices) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    typedef Record<KIND> R;
    typedef ScanStage<KIND> L;
    extern __shared__ __align__(16) char lds[];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    // heads that share a key head sit on one XCD (blocks go round the eight by index)
    const int per = (A.H + 7) / 8;
    const int xcd = blockIdx.x & 7;
    int rest = blockIdx.x >> 3;
    const int slice = rest % slices;
    rest /= slices;
    const int u = rest % per, seq = rest / per;
    const int h = A.Hk % 8 == 0 ? (xcd + 8 * (u / A.share)) * A.share + u % A.share : xcd + 8 * u;
    if (h >= A.H) return;
    const int hk = h / A.share;
    const SeqSpan sp = seq_span(A, seq);
    if (!sp.live) return;
    const int ct = slice * NW + w;  // column tile
    const bool active = ct * 16 < V;
    const int col = active ? ct * 16 + lr : lr;

    // the state: tile 2 s + o, register r <-> row 32 s + 8 lq + 4 o + r
    f32x4 S[8];
    const int svo = (8 * lq * V + col) * 4;
    if (sp.row0 >= 0) {
        const __amdgpu_buffer_rsrc_t s0 = buffer_rsrc(A.S0 + (size_t(sp.row0) * A.H + h) * (kK * V), kK * V * 4);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[t][r] = buffer_load_f32(s0, svo, (32 * (t >> 1) + 4 * (t & 1) + r) * V * 4);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int n_chunks = (sp.len + kC - 1) / kC;
    const char* rec0 = ws + (first_slot(sp.t0, seq) * A.H + h) * R::bytes;
    const size_t rec_step = size_t(A.H) * R::bytes;
    const char* ksrc = static_cast<const char*>(A.k) + (size_t(sp.t0) * A.Hk + hk) * (kK * 2);
    const char* qsrc = static_cast<const char*>(A.q) + (size_t(sp.t0) * A.Hk + hk) * (kK * 2);

    // chunk c's keys, queries and record to LDS, straight from memory; rows
    // behind the sequence repeat its last token (their columns of T and P are 0)
    auto stage = [&](int c, char* buf) {
        const char* rec = rec0 + c * rec_step;
        constexpr int NREC = R::g / kFrag;
#pragma unroll
        for (int i0 = 0; i0 < 16 + NREC + 1; i0 += NW) {
            const int i = i0 + w;
            if (i < 16) {
                const int r = 4 * (i & 7) + (lane >> 4);
                const int t = min(c * kC + r, sp.len - 1);
                const char* src = i < 8 ? ksrc : qsrc;
                load_to_lds16(src + size_t(t) * (A.Hk * kK * 2) + ((lane & 15) ^ row_swizzle(r)) * 16,
                                buf + i * kFrag);
            } else if (i < 16 + NREC) {
                load_to_lds16(rec + (i - 16) * kFrag + lane * 16, buf + i * kFrag);
            } else if (i == 16 + NREC) {
                load_to_lds4(rec + R::g + lane * 4, buf + L::rec + R::g);
            }
        }
    };
    // this lane's values of chunk c: tokens 8 lq .. 8 lq + 7 (0 behind the sequence)
    const uint32_t vstep = uint32_t(A.H) * V * 2;
    auto load_v = [&](int c, uint16_t* v) {
        const size_t base = ((size_t(sp.t0) + c * kC) * A.H + h) * V;
        const int left = min(kC, sp.len - c * kC);
        const __amdgpu_buffer_rsrc_t rs =
            buffer_rsrc(static_cast<const uint16_t*>(A.v) + base, uint32_t(left - 1) * vstep + V * 2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, int((8 * lq + i) * vstep) + col * 2, 0, 0);
    };

    uint16_t v[8];
    if (n_chunks > 0) {
        stage(0, lds);
        load_v(0, v);
    }
    for (int c = 0; c < n_chunks; ++c) {
        char* buf = lds + (c & 1) * L::bytes;
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's part of the chunk has landed
        __syncthreads();
        uint16_t vn[8];
        if (c + 1 < n_chunks) {
            stage(c + 1, lds + ((c + 1) & 1) * L::bytes);
            load_v(c + 1, vn);
        }
        const float* gam = reinterpret_cast<const float*>(buf + L::rec + R::g);

        // X = K S, Y = Q S
        f32x4 X[2], Y[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) X[m] = Y[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float f[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) f[r] = S[2 * s + r / 4][r & 3];
            const Split3 b = split3(f);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int row = tile_row(m, lr);
                const int at = row * (kK * 2) + ((4 * s + lq) ^ row_swizzle(row)) * 16;
                if (DELTA) X[m] = mfma_13(*reinterpret_cast<const uint4*>(buf + L::k + at), b, X[m]);
                Y[m] = mfma_13(*reinterpret_cast<const uint4*>(buf + L::q + at), b, Y[m]);
            }
        }
        float g[8], sg[8], wt[8];
        load8f(gam + 8 * lq, g);
        load8f(gam + kC + 8 * lq, sg);
        const float gC = gam[kC - 1];
#pragma unroll
        for (int i = 0; i < 8; ++i) wt[i] = __uint_as_float(uint32_t(v[i]) << 16);
        Split3 wb;
        const char* frag = buf + L::rec + lane * 16;
        if (DELTA) {  // w = T (v - gamma X)
#pragma unroll
            for (int i = 0; i < 8; ++i) wt[i] = fmaf(-g[i], X[i / 4][i & 3], wt[i]);
            const Split3 rb = split3(wt);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint4 a[3];
#pragma unroll
                for (int e = 0; e < 3; ++e) a[e] = *reinterpret_cast<const uint4*>(frag + R::t + (2 * e + m) * kFrag);
                const f32x4 d = mfma_33(a, rb, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) wt[4 * m + r] = d[r];
            }
            wb = split3(wt);
        }
        // S <- gamma_C S + K^T (sigma w)
        {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = sg[i] * wt[i];
            const Split3 b = split3(f);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                // rows of K^T by transposed reads: a quarter-wave's lane p points at
                // four channels of token 8 lq + 4 o + p / 4, and lane i receives its
                // row's channel of tokens 8 lq + 4 o .. + 3
                uint32_t a[4];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int row = 8 * lq + 4 * o + (lr >> 2);
                    const char* p = buf + L::k + row * (kK * 2) +
                                    ((4 * (t >> 1) + (lr & 3)) ^ row_swizzle(row)) * 16 + 8 * (t & 1);
                    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s16x4*)(p));
                    const uint2 u2 = __builtin_bit_cast(uint2, x);
                    a[2 * o] = u2.x;
                    a[2 * o + 1] = u2.y;
                }
                S[t] = mfma_13(make_uint4(a[0], a[1], a[2], a[3]), b, S[t] * gC);
            }
        }
        // y = gamma Y + P w
        {
            const size_t base = ((size_t(sp.t0) + c * kC) * A.H + h) * V;
            const int left = min(kC, sp.len - c * kC);
            const uint32_t ystep = uint32_t(A.H) * V * 4;
            const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(A.y + base, uint32_t(left - 1) * ystep + V * 4);
            uint4 vb;
            if (!DELTA)
                vb = make_uint4(v[0] | uint32_t(v[1]) << 16, v[2] | uint32_t(v[3]) << 16, v[4] | uint32_t(v[5]) << 16,
                                v[6] | uint32_t(v[7]) << 16);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                f32x4 acc;
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = g[4 * m + r] * Y[m][r];
                uint4 a[3];
#pragma unroll
                for (int e = 0; e < 3; ++e) a[e] = *reinterpret_cast<const uint4*>(frag + R::p + (2 * e + m) * kFrag);
                if (DELTA) {
                    acc = mfma_33(a, wb, acc);
                } else {
                    acc = mfma_bf16(a[2], vb, acc);
                    acc = mfma_bf16(a[1], vb, acc);
                    acc = mfma_bf16(a[0], vb, acc);
                }
                if (active) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        buffer_store_f32(acc[r], rs, int((8 * lq + 4 * m + r) * ystep) + col * 4, 0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = vn[i];
    }
    if (active) {
        const __amdgpu_buffer_rsrc_t so = buffer_rsrc(A.S + (size_t(sp.row) * A.H + h) * (kK * V), kK * V * 4);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                buffer_store_f32(S[t][r], so, svo, (32 * (t >> 1) + 4 * (t & 1) + r) * V * 4);
    }
}

namespace {

template <int KIND, int NW>
hipError_t launch_scan_t(const RaggedArgs& a, const char* ws, int V, hipStream_t s) {
    const int slices = (V / 16 + NW - 1) / NW;
    const long blocks = long(a.n_seqs) * ((a.H + 7) / 8) * 8 * slices;
    hipLaunchKernelGGL((scan_kernel<KIND, NW>), dim3(uint32_t(blocks)), dim3(NW * 64), 2 * ScanStage<KIND>::bytes, s, a,
                       ws, V, slices);
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_chunked(const RaggedArgs& a, char* ws, int V, hipStream_t s) {
    const long tasks = prefill_slots(a.total, a.n_seqs) * a.H;
    hipLaunchKernelGGL((prep_kernel<KIND>), dim3(uint32_t((tasks + kPrepWaves - 1) / kPrepWaves)),
                       dim3(kPrepWaves * 64), 0, s, a, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    switch (V) {
        case 64: return launch_scan_t<KIND, 4>(a, ws, V, s);
        case 80: return launch_scan_t<KIND, 5>(a, ws, V, s);
        case 96: return launch_scan_t<KIND, 6>(a, ws, V, s);
        case 112: return launch_scan_t<KIND, 7>(a, ws, V, s);
        case 128: return launch_scan_t<KIND, 8>(a, ws, V, s);
    }
    return hipErrorInvalidValue;
}

// Whether a call takes the chunked kernels, else the recurrent one.
bool chunked(const sketchssm_shape& sh, int max_len) {
    return sh.qkv == SKSSM_BF16 && sh.kind != SKSSM_KDA && max_len > 16;
}

}  // namespace

}  // namespace skssm

using namespace skssm;

extern "C" size_t sketchssm_prefill_workspace(const sketchssm_shape* shape, int32_t n_seqs, int32_t total_tokens,
                                              int32_t max_len) {
    if (check_shape(shape) != SKSSM_OK || n_seqs <= 0 || total_tokens < 0 || max_len < 0) return 0;
    if (!chunked(*shape, max_len)) return 0;
    const size_t rec = shape->kind == SKSSM_MAMBA2 ? Record<SKSSM_MAMBA2>::bytes : Record<SKSSM_GDN>::bytes;
    return size_t(prefill_slots(total_tokens, n_seqs)) * shape->H * rec;
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
    if (!chunked(*shape, max_len)) {
        e = launch_recur(*shape, A, s);
    } else {
        // blocks of both launches stay below 2^31
        if (double(prefill_slots(total_tokens, n_seqs)) * shape->H >= 2147483648.0) return SKSSM_ESHAPE;
        if (double(n_seqs) * (shape->H + 7) * 8 >= 2147483648.0) return SKSSM_ESHAPE;
        char* ws = static_cast<char*>(workspace);
        e = shape->kind == SKSSM_MAMBA2 ? launch_chunked<SKSSM_MAMBA2>(A, ws, shape->V, s)
                                        : launch_chunked<SKSSM_GDN>(A, ws, shape->V, s);
    }
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
