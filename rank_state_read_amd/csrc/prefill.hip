// Prefill of ragged prompts for gfx950: the state update in chunks of C = 64
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
// registers.  Value columns are independent of each other: a block owns 16 of
// them, so that a single sequence fills the chip.  Its four waves share a
// chunk's work by rows -- 16 tokens each for K S, Q S, T and P, 32 key channels
// each for the state -- and hand each other their results through LDS as B
// operands.
//
// Products run on the bf16 matrix instruction (16x16x32, fp32 sums) and keep
// fp32 precision: an fp32 operand x is written as hi + mid + lo, three bf16
// numbers of 8 significant bits each.  q, k, v in bf16 are exact operands, so
// their products with an fp32 operand take three instructions, products of two
// fp32 operands six (the terms below 2^-24 are left out).  The fp32 matrix
// instruction has 1/16 of the bf16 rate.
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
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = 64;              // tokens per chunk
constexpr int kFrag = 64 * 16;      // one operand of a wave, bytes
constexpr int kTri = 6 * 3 * kFrag; // T or P: six (row tile, 32-column) operands of three terms

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// x = t[0] + t[1] + t[2] for 2 N consecutive values, each term rounded to bf16.
template <int N>
__device__ __forceinline__ void split3(const float* f, uint32_t (&u)[3][N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x0 = f[2 * i], x1 = f[2 * i + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x0, x1}), bf16x2));
            u[p][i] = h;
            x0 -= __uint_as_float(h << 16);
            x1 -= __uint_as_float(h & 0xffff0000u);
        }
    }
}

// Operand (row tile m, 32-column step s <= m / 2) of a C x C triangle.
__device__ __forceinline__ int tri_frag(int m, int s) { return (m < 2 ? m : 2 * m - 2) + s; }

// A workspace record: P, then T (delta rule), then gamma and sigma.
template <int KIND>
struct Record {
    static constexpr bool delta = KIND != SKSSM_MAMBA2;
    static constexpr int p = 0;
    static constexpr int t = kTri;
    static constexpr int g = delta ? 2 * kTri : kTri;
    static constexpr int bytes = g + 2 * kC * 4;
};

inline long prefill_slots(long total, int n_seqs) { return total / kC + n_seqs; }

// Chunk c of a sequence has slot off / C + seq + c of the workspace: a sequence
// of len tokens has at most (off + len) / C - off / C + 1 chunks, so sequences
// that do not overlap never share a slot.
__device__ __forceinline__ long first_slot(int t0, int seq) { return long(t0) / kC + seq; }

}  // namespace

// ---------------------------------------------------------------------------
// T and P of every chunk and head: a block of four waves per (slot, head).
// ---------------------------------------------------------------------------
constexpr int kGS = kC + 4;  // row stride of a C x C matrix in LDS, floats

// Product of two 16 x 16 blocks in LDS, added to c.
__device__ __forceinline__ f32x4 block_mul(const float* a, const float* b, f32x4 c, int lr, int lq) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = mfma_16x16x4(a[lr * kGS + 4 * s + lq], b[(4 * s + lq) * kGS + lr], c);
    return c;
}
// The same with the second block in the accumulator layout.
__device__ __forceinline__ f32x4 block_mul(const float* a, f32x4 b, f32x4 c, int lr, int lq) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = mfma_16x16x4(a[lr * kGS + 4 * lq + s], b[s], c);
    return c;
}
__device__ __forceinline__ void block_put(float* d, f32x4 c, int lr, int lq) {
#pragma unroll
    for (int r = 0; r < 4; ++r) d[(4 * lq + r) * kGS + lr] = c[r];
}

template <int KIND>
__global__ __launch_bounds__(256) void prep_kernel(RaggedArgs A, char* ws) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    typedef Record<KIND> R;
    __shared__ __align__(16) float gq[kC * kGS];
    __shared__ __align__(16) float gk[DELTA ? kC * kGS : 4];
    __shared__ __align__(16) float bs[kC];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const long slot = blockIdx.x / A.H;
    const int h = int(blockIdx.x - slot * A.H), hk = h / A.share;

    // the sequence and chunk of this slot, if any (every wave looks on its own)
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
    if (seq < 0) return;  // the whole block

    // k_i . k_j and q_i . k_j, row tile w: exact products of bf16 values, fp32 sums
    {
        auto row = [&](const void* base, int tile, u32x4 (&f)[4]) {
            const size_t r = (size_t(t0) + min(16 * tile + lr, clen - 1)) * A.Hk + hk;
            const char* src = static_cast<const char*>(base) + (r * kK + 8 * lq) * 2;
#pragma unroll
            for (int s = 0; s < 4; ++s) f[s] = *reinterpret_cast<const u32x4*>(src + 64 * s);
        };
        u32x4 kf[4], qf[4];
        if (DELTA) row(A.k, w, kf);
        row(A.q, w, qf);
        for (int n = 0; n <= w; ++n) {
            u32x4 nf[4];
            row(A.k, n, nf);
            f32x4 dk = {0.f, 0.f, 0.f, 0.f}, dq = dk;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (DELTA) dk = mfma_bf16(kf[s], nf[s], dk);
                dq = mfma_bf16(qf[s], nf[s], dq);
            }
            if (DELTA) block_put(gk + 16 * w * kGS + 16 * n, dk, lr, lq);
            block_put(gq + 16 * w * kGS + 16 * n, dq, lr, lq);
        }
    }
    const bool valid = lane < clen;
    const size_t tj = size_t(t0) + (valid ? lane : 0);
    const float aj = valid ? A.a[tj * A.H + h] : 1.f;
    const float bj = !DELTA ? 1.f : valid ? A.beta[tj * A.H + h] : 0.f;
    if (w == 0) bs[lane] = bj;
    __syncthreads();

    // column j = lane: the decays' products after token j, one factor at a time (a
    // decay may be 0, so nothing is divided).  Delta rule: two waves write -A, two
    // P, 32 rows each; Mamba-2: 16 rows of P each.
    char* rec = ws + size_t(blockIdx.x) * R::bytes;
    {
        const bool isA = DELTA && (w & 1) == 0;
        const int rows = DELTA ? 32 : 16, r0 = DELTA ? 32 * (w >> 1) : 16 * w;
        float* gt = isA ? gk : gq;
        float d = 0.f, gam = 0.f, run = 1.f;
        for (int i = 0; i < r0; ++i) {
            const float ai = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(aj), i));
            d = i == lane ? 1.f : d * ai;
            run *= ai;
            gam = i == lane ? run : gam;
        }
#pragma unroll 8
        for (int i = r0; i < r0 + rows; ++i) {
            const float ai = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(aj), i));
            const float bi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(bj), i));
            d = i == lane ? 1.f : d * ai;
            run *= ai;
            gam = i == lane ? run : gam;
            const float g = gt[i * kGS + lane] * d;
            const bool in = isA ? i > lane : i >= lane && valid;
            gt[i * kGS + lane] = in ? (isA ? -bi * g : g) : 0.f;
        }
        if (w == 3) {  // the waves that have walked to the end
            float* g = reinterpret_cast<float*>(rec + R::g);
            g[lane] = gam;
            g[kC + lane] = valid ? d : 0.f;
        }
    }
    __syncthreads();

    if (DELTA) {
        // (I + A)^-1 by blocks of 16: the diagonal blocks by forward substitution,
        // one lane per column, then M_ba = M_bb (-A_ba) M_aa for 16 and 32 rows
        if (lane < 16) {
            float* g = gk + 16 * w * kGS + 16 * w;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const f32x4 n4 = *reinterpret_cast<const f32x4*>(g + i * kGS + m);
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
            for (int i = 0; i < 16; ++i) g[i * kGS + lane] = x[i];
        }
        __syncthreads();
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        auto blk = [&](int i, int j) { return gk + 16 * i * kGS + 16 * j; };
        if (w < 2) {  // blocks (1, 0) and (3, 2)
            const f32x4 r = block_mul(blk(2 * w + 1, 2 * w), blk(2 * w, 2 * w), zero, lr, lq);
            const f32x4 m = block_mul(blk(2 * w + 1, 2 * w + 1), r, zero, lr, lq);
            __builtin_amdgcn_wave_barrier();
            block_put(blk(2 * w + 1, 2 * w), m, lr, lq);
        }
        __syncthreads();
        const int ca = w & 1, rb = 2 + (w >> 1);  // block (rb, ca)
        f32x4 m = zero;
        for (int b = 2; b <= rb; ++b) {
            f32x4 r = zero;
            for (int x = ca; x < 2; ++x) r = block_mul(blk(b, x), blk(x, ca), r, lr, lq);
            m = block_mul(blk(rb, b), r, m, lr, lq);
        }
        __syncthreads();
        block_put(blk(rb, ca), m, lr, lq);
        __syncthreads();
    }

    // row tile w of both as A operands
    for (int s = 0; s <= w / 2; ++s) {
        const int at = (16 * w + lr) * kGS + 32 * s + 8 * lq;
        char* out = rec + tri_frag(w, s) * 3 * kFrag + lane * 16;
        float f[8];
        uint32_t u[3][4];
        load8f(gq + at, f);
        split3<4>(f, u);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            *reinterpret_cast<u32x4*>(out + R::p + e * kFrag) = u32x4{u[e][0], u[e][1], u[e][2], u[e][3]};
        if (DELTA) {
            float b[8];
            load8f(gk + at, f);
            load8f(bs + 32 * s + 8 * lq, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= b[i];
            split3<4>(f, u);
#pragma unroll
            for (int e = 0; e < 3; ++e)
                *reinterpret_cast<u32x4*>(out + R::t + e * kFrag) = u32x4{u[e][0], u[e][1], u[e][2], u[e][3]};
        }
    }
}

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks.
// ---------------------------------------------------------------------------
struct ScanLds {  // bytes
    static constexpr int k = 0;                         // keys of two chunks [2][C][K], swizzled
    static constexpr int s = k + 2 * kC * kK * 2;       // the state's B operands: [buffer][4 steps][3 terms]
    static constexpr int sbuf = 12 * kFrag;
    // delta rule: v - gamma K S, w and sigma w, each [2 steps][3 terms]
    static constexpr int r = s + sbuf;
    static constexpr int w = r + 6 * kFrag;
    static constexpr int u = w + 6 * kFrag;
    static constexpr int bytes_delta = u + 6 * kFrag;
    // Mamba-2: two buffers of the state, of v [2 steps] and of sigma v
    static constexpr int v2 = s + 2 * sbuf;
    static constexpr int u2 = v2 + 2 * 2 * kFrag;
    static constexpr int bytes_mamba = u2 + 2 * 6 * kFrag;
};

// Granule of 16 bytes g of token row r sits at granule g ^ row_swizzle(r): the 16
// rows of a tile start in different banks, and so do the four rows and four
// granules of a transposed read.
__device__ __forceinline__ int row_swizzle(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

template <int KIND>
__global__ __launch_bounds__(256) void scan_kernel(RaggedArgs A, const char* ws, int V) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    typedef Record<KIND> R;
    typedef ScanLds L;
    extern __shared__ __align__(16) char lds[];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // the same in every lane
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    // heads that share a key head sit on one XCD (blocks go round the eight by index)
    const int per = (A.H + 7) / 8, slices = V / 16;
    const int xcd = blockIdx.x & 7;
    int rest = blockIdx.x >> 3;
    const int slice = rest % slices;
    rest /= slices;
    const int un = rest % per, seq = rest / per;
    const int h = A.Hk % 8 == 0 ? (xcd + 8 * (un / A.share)) * A.share + un % A.share : xcd + 8 * un;
    if (h >= A.H) return;
    const int hk = h / A.share;
    const SeqSpan sp = seq_span(A, seq);
    if (!sp.live) return;
    const int col = slice * 16 + lr;

    // the state, channels 32 w .. 32 w + 31: tile o, register r <-> channel
    // 32 w + 8 lq + 4 o + r, so a lane holds 8 consecutive channels, one B operand
    f32x4 S[2];
    const int svo = ((32 * w + 8 * lq) * V + col) * 4;
    if (sp.row0 >= 0) {
        const __amdgpu_buffer_rsrc_t s0 = buffer_rsrc(A.S0 + (size_t(sp.row0) * A.H + h) * (kK * V), kK * V * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) S[i / 4][i & 3] = buffer_load_f32(s0, svo, i * V * 4);
    } else {
        S[0] = S[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int n_chunks = (sp.len + kC - 1) / kC;

    const char* rec0 = ws + (first_slot(sp.t0, seq) * A.H + h) * R::bytes;
    const size_t rec_step = size_t(A.H) * R::bytes;
    const char* ksrc = static_cast<const char*>(A.k) + (size_t(sp.t0) * A.Hk + hk) * (kK * 2);
    const char* qsrc = static_cast<const char*>(A.q) + (size_t(sp.t0) * A.Hk + hk) * (kK * 2);
    const uint32_t qk_step = uint32_t(A.Hk) * kK * 2;

    // Loads of chunk c.  Rows behind the sequence repeat its last token: their
    // columns of T and P and their sigma are 0.
    u32x4 kreg[4], qf[4], tf[2][3], pf[2][3];
    f32x4 gam, sig;
    float gC;
    uint32_t v[4];
    auto load_k = [&](int c) {  // rows 16 j + 4 w + lane / 16 of the key tile
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 16 * j + 4 * w + lq;
            const size_t t = min(c * kC + r, sp.len - 1);
            kreg[j] = *reinterpret_cast<const u32x4*>(ksrc + t * qk_step + (lr ^ row_swizzle(r)) * 16);
        }
    };
    auto put_k = [&](int c) {
        char* dst = lds + L::k + (c & 1) * (kC * kK * 2) + (4 * w + lq) * (kK * 2) + lr * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4*>(dst + 16 * j * (kK * 2)) = kreg[j];
    };
    auto load_q = [&](int c) {
        const size_t t = min(c * kC + 16 * w + lr, sp.len - 1);
#pragma unroll
        for (int s = 0; s < 4; ++s) qf[s] = *reinterpret_cast<const u32x4*>(qsrc + t * qk_step + 16 * lq + 64 * s);
    };
    auto load_tri = [&](int c, int what, u32x4 (&f)[2][3]) {
        const char* src = rec0 + c * rec_step + what + lane * 16;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int e = 0; e < 3; ++e)  // waves 0 and 1 have one step only: it stands in for the second
                f[s][e] = *reinterpret_cast<const u32x4*>(src + (tri_frag(w, min(s, w / 2)) * 3 + e) * kFrag);
    };
    auto load_gam = [&](int c) {
        const float* g = reinterpret_cast<const float*>(rec0 + c * rec_step + R::g);
        gam = *reinterpret_cast<const f32x4*>(g + 16 * w + 4 * lq);
        sig = *reinterpret_cast<const f32x4*>(g + kC + 16 * w + 4 * lq);
        gC = g[kC - 1];
    };
    const uint32_t vstep = uint32_t(A.H) * V * 2, ystep = 2 * vstep;
    auto load_v = [&](int c) {  // tokens 16 w + 4 lq + r (0 behind the sequence)
        const size_t base = ((size_t(sp.t0) + c * kC) * A.H + h) * V;
        const int left = min(kC, sp.len - c * kC);
        const __amdgpu_buffer_rsrc_t rs =
            buffer_rsrc(static_cast<const uint16_t*>(A.v) + base, uint32_t(left - 1) * vstep + V * 2);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v[r] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, int((16 * w + 4 * lq + r) * vstep) + col * 2, 0, 0));
    };
    auto store_y = [&](int c, f32x4 y) {
        const size_t base = ((size_t(sp.t0) + c * kC) * A.H + h) * V;
        const int left = min(kC, sp.len - c * kC);
        const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(A.y + base, uint32_t(left - 1) * ystep + V * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) buffer_store_f32(y[r], rs, int((16 * w + 4 * lq + r) * ystep) + col * 4, 0);
    };

    // Four values of tokens 16 w + 4 lq .. + 3 into B operands [2 steps][stride
    // terms]: half a lane's 16 bytes
    const int half = ((2 * (w & 1) + (lq >> 1)) * 16 + lr) * 16 + 8 * (lq & 1);
    auto put_tokens = [&](char* dst, f32x4 x) {
        const float f[4] = {x[0], x[1], x[2], x[3]};
        uint32_t u[3][2];
        split3<2>(f, u);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            *reinterpret_cast<u32x2*>(dst + ((w >> 1) * 3 + e) * kFrag + half) = u32x2{u[e][0], u[e][1]};
    };
    auto put_state = [&](char* dst) {
        float f[8];
        uint32_t u[3][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = S[i / 4][i & 3];
        split3<4>(f, u);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            *reinterpret_cast<u32x4*>(dst + (w * 3 + e) * kFrag + lane * 16) = u32x4{u[e][0], u[e][1], u[e][2], u[e][3]};
    };
    // one 16 x 64 by 64 x 16 product of two three-term operands, small terms first
    auto tri_mul = [&](const u32x4 (&a)[2][3], const char* b, f32x4 c) {
        constexpr int ia[6] = {2, 0, 1, 1, 0, 0}, ib[6] = {0, 2, 1, 0, 1, 0};
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
        u32x4 x[3];
#pragma unroll
        for (int e = 0; e < 3; ++e) x[e] = *reinterpret_cast<const u32x4*>(b + e * kFrag + lane * 16);
        if (w >= 2) {
            u32x4 z[3];
#pragma unroll
            for (int e = 0; e < 3; ++e) z[e] = *reinterpret_cast<const u32x4*>(b + (3 + e) * kFrag + lane * 16);
#pragma unroll
            for (int e = 0; e < 6; ++e) {
                c = mfma_bf16(a[0][ia[e]], x[ib[e]], c);
                d = mfma_bf16(a[1][ia[e]], z[ib[e]], d);
            }
            return c + d;
        }
#pragma unroll
        for (int e = 0; e < 6; ++e) c = mfma_bf16(a[0][ia[e]], x[ib[e]], c);
        return c;
    };
    // S <- gamma_C S + K^T u, u as B operands [2 steps][3 terms]
    auto update = [&](int c, const char* u) {
        const char* kt = lds + L::k + (c & 1) * (kC * kK * 2);
        u32x4 b[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int e = 0; e < 3; ++e) b[s][e] = *reinterpret_cast<const u32x4*>(u + (3 * s + e) * kFrag + lane * 16);
        u32x4 a[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // transposed read: a quarter-wave's lane p points at four channels of
                    // token 32 s + 8 lq + 4 x + p / 4, and lane i receives its row's
                    // channel (tile o) of tokens 32 s + 8 lq + 4 x .. + 3
                    const int row = 32 * s + 8 * lq + 4 * x + (lr >> 2);
                    const char* p = kt + row * (kK * 2) + ((4 * w + (lr & 3)) ^ row_swizzle(row)) * 16 + 8 * o;
                    const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
                    const u32x2 q2 = __builtin_bit_cast(u32x2, q);
                    a[s][o][2 * x] = q2[0];
                    a[s][o][2 * x + 1] = q2[1];
                }
        S[0] *= gC;
        S[1] *= gC;
#pragma unroll
        for (int e = 2; e >= 0; --e)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int o = 0; o < 2; ++o) S[o] = mfma_bf16(a[s][o], b[s][e], S[o]);
    };
    // K S and Q S of this wave's tokens
    auto state_mul = [&](int c, const char* sb, f32x4& X, f32x4& Y) {
        const char* kt = lds + L::k + (c & 1) * (kC * kK * 2);
        const int row = 16 * w + lr;
        u32x4 b[4][3], ka[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int e = 0; e < 3; ++e) b[s][e] = *reinterpret_cast<const u32x4*>(sb + (3 * s + e) * kFrag + lane * 16);
            if (DELTA)
                ka[s] = *reinterpret_cast<const u32x4*>(kt + row * (kK * 2) + ((4 * s + lq) ^ row_swizzle(row)) * 16);
        }
#pragma unroll
        for (int e = 2; e >= 0; --e)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (DELTA) X = mfma_bf16(ka[s], b[s][e], X);
                Y = mfma_bf16(qf[s], b[s][e], Y);
            }
    };

    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if (n_chunks > 0) {
        const int last = n_chunks - 1;
        load_k(0);
        load_q(0);
        load_gam(0);
        load_v(0);
        if constexpr (DELTA) {
            load_tri(0, R::t, tf);
            put_state(lds + L::s);
            put_k(0);
            f32x4 yp = zero;  // y of the chunk before, as far as it is formed
            for (int c = 0; c < n_chunks; ++c) {
                __syncthreads();  // keys and state of chunk c
                const int cn = min(c + 1, last);  // the last chunk loads itself again
                load_k(cn);
                __builtin_amdgcn_sched_barrier(0);
                f32x4 X = zero, Y = zero;
                state_mul(c, lds + L::s, X, Y);
                load_q(cn);
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = fmaf(-gam[r], X[r], __uint_as_float(v[r] << 16));
                    Y[r] *= gam[r];
                }
                put_tokens(lds + L::r, x);
                if (c) store_y(c - 1, tri_mul(pf, lds + L::w, yp));
                load_tri(c, R::p, pf);
                yp = Y;
                __syncthreads();  // v - gamma K S
                x = tri_mul(tf, lds + L::r, zero);
                load_tri(cn, R::t, tf);
                put_tokens(lds + L::u, x * sig);
                put_tokens(lds + L::w, x);
                __syncthreads();  // w
                update(c, lds + L::u);
                load_gam(cn);
                load_v(cn);
                put_state(lds + L::s);
                put_k(c + 1);
            }
            store_y(last, tri_mul(pf, lds + L::w, yp));
        } else {
            auto put_v = [&](int c) {  // v and sigma v of chunk c
                char* dst = lds + L::v2 + (c & 1) * 2 * kFrag + (w >> 1) * kFrag + half;
                *reinterpret_cast<u32x2*>(dst) = u32x2{v[0] | v[1] << 16, v[2] | v[3] << 16};
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = sig[r] * __uint_as_float(v[r] << 16);
                put_tokens(lds + L::u2 + (c & 1) * 6 * kFrag, x);
            };
            load_tri(0, R::p, pf);
            put_state(lds + L::s);
            put_k(0);
            put_v(0);
            f32x4 g = gam;
            float gc = gC;
            for (int c = 0; c < n_chunks; ++c) {
                __syncthreads();  // keys, values and state of chunk c; the other buffers are free
                const int cn = min(c + 1, last);
                load_k(cn);
                load_v(cn);
                load_gam(cn);
                __builtin_amdgcn_sched_barrier(0);
                f32x4 X = zero, Y = zero;
                state_mul(c, lds + L::s + (c & 1) * L::sbuf, X, Y);
                load_q(cn);
                const float gnext = gC;
                gC = gc;
                update(c, lds + L::u2 + (c & 1) * 6 * kFrag);
                gC = gc = gnext;
                put_state(lds + L::s + ((c + 1) & 1) * L::sbuf);
                Y *= g;
                g = gam;
                const char* vb = lds + L::v2 + (c & 1) * 2 * kFrag + lane * 16;
                const u32x4 b0 = *reinterpret_cast<const u32x4*>(vb);
#pragma unroll
                for (int e = 2; e >= 0; --e) Y = mfma_bf16(pf[0][e], b0, Y);
                if (w >= 2) {
                    const u32x4 b1 = *reinterpret_cast<const u32x4*>(vb + kFrag);
#pragma unroll
                    for (int e = 2; e >= 0; --e) Y = mfma_bf16(pf[1][e], b1, Y);
                }
                load_tri(cn, R::p, pf);
                store_y(c, Y);
                put_k(c + 1);
                put_v(c + 1);
            }
        }
    }
    const __amdgpu_buffer_rsrc_t so = buffer_rsrc(A.S + (size_t(sp.row) * A.H + h) * (kK * V), kK * V * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) buffer_store_f32(S[i / 4][i & 3], so, svo, i * V * 4);
}

namespace {

template <int KIND>
hipError_t launch_chunked(const RaggedArgs& a, char* ws, int V, hipStream_t s) {
    constexpr int lds = KIND == SKSSM_MAMBA2 ? ScanLds::bytes_mamba : ScanLds::bytes_delta;
    hipLaunchKernelGGL((prep_kernel<KIND>), dim3(uint32_t(prefill_slots(a.total, a.n_seqs) * a.H)), dim3(256), 0, s, a,
                       ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (lds > 64 * 1024) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(scan_kernel<KIND>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const long blocks = long(a.n_seqs) * ((a.H + 7) / 8) * 8 * (V / 16);
    hipLaunchKernelGGL((scan_kernel<KIND>), dim3(uint32_t(blocks)), dim3(256), lds, s, a, ws, V);
    return hipGetLastError();
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
        if (double(n_seqs) * (shape->H + 7) * (shape->V / 16) >= 2147483648.0) return SKSSM_ESHAPE;
        char* ws = static_cast<char*>(workspace);
        e = shape->kind == SKSSM_MAMBA2 ? launch_chunked<SKSSM_MAMBA2>(A, ws, shape->V, s)
                                        : launch_chunked<SKSSM_GDN>(A, ws, shape->V, s);
    }
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
