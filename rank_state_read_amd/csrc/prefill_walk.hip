// The chunked form for gfx950 (prefill_common.h): chunks of C = 32 tokens.
//
// Two launches.  T and P depend on a chunk's own tokens alone, so the first
// forms them for all chunks of all heads at once and leaves them in the
// workspace; the second walks a sequence's chunks in order with the state in
// registers.  A Mamba-2 layer with bf16 keys has many heads to a key head and
// little work per value, so its P, one per head, would cost more to move than to
// form: the first launch leaves q_i . k_j per key head and the decays' products,
// and the walk forms P from them.
//
// us of the two launches, bf16: GDN, 32 heads of 128, 16001 tokens of 9 sequences, 64
// and 292; Mamba-2, 128 heads of 80, 16003 tokens of 7, 41 and 446; KDA, 32 heads of
// 128, 8190 tokens of 4, 162 and 508.  For GDN the first one moves 260 MB (131 of keys and
// queries, 129 of records), 4.1 TB/s, two thirds of a plain stream's 6.2, while its waves
// wait for data 31% and for their turn 53% of the time: the chain of a chunk's products
// and substitution.  With a key head per head it is 400 MB in 72 us, 5.5 TB/s, nearly the
// stream's.  For KDA fp32 products come on top.  The walk runs its bf16 products at 690,
// 635 and 355 TFLOP/s (a large library product: 1208 to 1343, box to box) with the matrix
// units busy 45%, 31% and 27% of the time.  What bounds it is the
// vector work beside them, which cuts the state and w into terms (350 vector
// instructions to 96 products per wave and chunk of GDN), and for few or uneven
// sequences the chain of a chunk's steps, as the longest sequence's chunks follow each
// other (4.2 us each for KDA, 2.2 for GDN).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "prefill_common.h"

namespace skssm {

namespace {

constexpr int kC = 32;               // tokens per chunk
constexpr int kTri = 3 * 2 * kFrag;  // T or P as A operands: three terms, two row tiles
constexpr int kPlane = kC * kK * 2;  // one bf16 term of a chunk's keys or queries

// A workspace record of a chunk and head: P, T, gamma and sigma, in pieces of 1 KB, 16
// bytes per lane.  P and T are lower triangular, so lanes with 8 columns behind the
// diagonal's hold zeros: those are neither written nor read, 10 of 16 lanes move.  (All
// of them: gdn batch 361 us against 350.)
__device__ __forceinline__ bool record_lane(int lane) { return lane >> 4 <= (lane & 15) >> 2; }

struct Record {
    static constexpr int p = 0;
    static constexpr int t = kTri;
    static constexpr int g = 2 * kTri;
    static constexpr int bytes = g + kFrag;  // whole pieces of 1 KB
};

// Mamba-2 with bf16 keys: gamma and sigma, the decays a [C], and with token groups
// of four F[b][i] = a_{4b+4} .. a_i (1 for i = 4b + 3, 0 before); q_i . k_j per key
// head in four tasks (row tile m, half o of the columns).
struct DecayRecord {
    static constexpr int g = 0;
    static constexpr int a = 2 * kC * 4;
    static constexpr int f = a + kC * 4;
    static constexpr int bytes = f + 8 * kC * 4;
    static constexpr int qk = 4 * kFrag;
};

// Mamba-2 with bf16 keys and queries: P is formed in the walk.
template <int KIND, typename QT>
constexpr bool kFormP = KIND == SKSSM_MAMBA2 && std::is_same<QT, Bf16Tag>::value;

constexpr int kGS = kC + 4;  // row stride of a C x C matrix in LDS, floats

// Product of two 16 x 16 blocks in LDS.
__device__ __forceinline__ f32x4 block_mul(const float* a, const float* b, int lr, int lq) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) c = mfma_16x16x4(a[lr * kGS + 4 * s + lq], b[(4 * s + lq) * kGS + lr], c);
    return c;
}
// The same with the second block in the accumulator layout.
__device__ __forceinline__ f32x4 block_mul(const float* a, f32x4 b, int lr, int lq) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) c = mfma_16x16x4(a[lr * kGS + 4 * lq + s], b[s], c);
    return c;
}

__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t rs, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

// ---------------------------------------------------------------------------
// T and P of every chunk and head: one wave per (slot, head).
// ---------------------------------------------------------------------------

// Row tile m of a matrix as A operand in three terms: f is row tile_row(m, lane % 16),
// columns 8 (lane / 16) .. + 7.
__device__ __forceinline__ void put_operand(char* dst, int m, const float* f, int lane) {
    uint32_t u[3][4];
    split3_rounded<4>(f, u);
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (record_lane(lane))
            *reinterpret_cast<u32x4*>(dst + (2 * e + m) * kFrag + lane * 16) = u32x4{u[e][0], u[e][1], u[e][2], u[e][3]};
}

// The same of a wave's matrix in LDS, its columns scaled.
__device__ __forceinline__ void put_operands(char* dst, const float* m, const float* scale, int lane) {
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        float f[8];
        load8f(m + tile_row(o, lane & 15) * kGS + 8 * (lane >> 4), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= scale ? scale[i] : 1.f;
        put_operand(dst, o, f, lane);
    }
}

// T = (I + A)^-1 diag(beta) of a record from g = -A (strictly lower) in LDS; lane
// j < 32 and j + 32 hold token j's beta (0 behind the sequence).
__device__ __forceinline__ void put_t(char* rec, float* g, float bj, int lane) {
    const int lr = lane & 15, lq = lane >> 4;
    float b[8];
    // (I + A)^-1: the diagonal blocks of 16 by forward substitution, one lane per
    // column, then M_10 = M_11 (-A_10) M_00
    if (lane < 32) {
        float* d = g + (lane & 16) * (kGS + 1);
        const int l = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == l ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const f32x4 n4 = *reinterpret_cast<const f32x4*>(d + i * kGS + m);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < i) {
                        if (e & 1) s1 = fmaf(n4[e], x[m + e], s1);
                        else s0 = fmaf(n4[e], x[m + e], s0);
                    }
            }
            x[i] = s0 + s1;
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i * kGS + l] = x[i];
    }
    wave_sync();
    const f32x4 r10 = block_mul(g + 16 * kGS, g, lr, lq);
    const f32x4 m10 = block_mul(g + 16 * kGS + 16, r10, lr, lq);
    wave_sync();
#pragma unroll
    for (int r = 0; r < 4; ++r) g[(16 + 4 * lq + r) * kGS + lr] = m10[r];
    wave_sync();
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __shfl(bj, 8 * lq + i, 64);
    put_operands(rec + Record::t, g, b, lane);
}

// A chunk's decays a_i, one per lane of each half wave: gamma (the product up to token
// i), sigma (after it) and put(g, F[g][i]) for the 8 groups g of four tokens, F[g][i] =
// a_{4g+4} .. a_i, 1 for i = 4g + 3 and 0 before.  Decays may be 0: nothing is divided.
template <typename Put>
__device__ __forceinline__ void chunk_decays(float av, int lane, float& gamma, float& sigma, Put put) {
    const int q = lane & 3, b = (lane & 31) >> 2;
    // within the group: products up to token i, and after it
    const float p1 = dpp_mov<0x90>(av);  // quad_perm [0,0,1,2]
    float up = q >= 1 ? av * p1 : av;
    const float p2 = dpp_mov<0x40>(up);  // quad_perm [0,0,0,1]
    up = q >= 2 ? up * p2 : up;
    const float n1 = dpp_mov<0xF9>(av);  // quad_perm [1,2,3,3]
    const float s1 = q <= 2 ? n1 : 1.f;
    const float n2 = dpp_mov<0xF9>(s1);
    float down = q <= 1 ? s1 * n2 : s1;
    const float n3 = dpp_mov<0xFF>(av);  // quad_perm [3,3,3,3]
    down = q == 0 ? down * n3 : down;
    float r = up, sg = down;
#pragma unroll
    for (int g = 7; g >= 0; --g) {
        const float bg = __shfl(up, (lane & 32) + 4 * g + 3, 64);
        put(g, g > b ? 0.f : g == b ? (q == 3 ? 1.f : 0.f) : r);
        r = g < b ? r * bg : r;
        sg = g > b ? sg * bg : sg;
    }
    gamma = r;
    sigma = sg;
}

// One decay per token.  A wave's four tasks (row tile m, half o of the columns) give
// k_j . k_i and k_j . q_i with lane = row i = tile_row(m, lr) and columns j = 8 lq + 4 o
// + r (bf16: exact products on the bf16 instruction; fp32: the fp32 instruction), the
// layout of P as an operand, and the decays between follow from F as in the walk.
// Only A goes through LDS, for its inverse.  (With both there, their rows multiplied by
// the decays one token after the other, 16001 tokens of 32 heads take 71 us instead of
// 64, and 77 tokens 8.7 instead of 6.8.)
template <bool DELTA, typename QT>
__global__ __launch_bounds__(256) void prep_scalar_kernel(RaggedArgs A, char* ws) {
    constexpr bool BF = std::is_same<QT, Bf16Tag>::value;
    typedef Record R;
    __shared__ __align__(16) float tiles[4][DELTA ? kC * kGS : 4];
    __shared__ __align__(16) float decays[4][9 * kC];  // F, a
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const long task = long(blockIdx.x) * 4 + w;
    const long slot = task / A.H;
    const int h = int(task - slot * A.H), hk = h / A.share;
    int t0 = 0;
    const int clen = slot_chunk<kC>(A, slot, lane, h == 0, t0);
    if (clen == 0) return;  // no wave waits for another one below

    float* g = tiles[w];
    float* f = decays[w];
    const int j = lane & 31;
    const bool valid = j < clen;
    const size_t tj = size_t(t0) + (valid ? j : 0);
    const float aj = valid ? A.a[tj * A.H + h] : 1.f;
    const float bj = !DELTA ? 1.f : valid ? A.beta[tj * A.H + h] : 0.f;
    // operands of a row tile: 64 bytes of each of 16 rows a step, for one bf16 product
    // of 32 channels or four fp32 products of 4 (lane's channels 16 s + 4 lq + e; with
    // a lane's channels in one run, 32 lq .., a step touches 64 lines instead of 16 and
    // 3001 tokens of 32 heads took 41 us instead of 30)
    constexpr int NV = BF ? 4 : 8;
    const Cursor<kC> ck(A.k, t0, A.Hk, hk, kK * Vec8<QT>::kElemBytes), cq(A.q, t0, A.Hk, hk, kK * Vec8<QT>::kElemBytes);
    const __amdgpu_buffer_rsrc_t rk = ck.rsrc(clen), rq = cq.rsrc(clen);
    auto row = [&](__amdgpu_buffer_rsrc_t rs, int m, u32x4 (&x)[NV]) {
        const int at = tile_row(m, lr) * int(ck.stride) + 16 * lq;
#pragma unroll
        for (int s = 0; s < NV; ++s) x[s] = load16(rs, at + 64 * s);
    };
    auto mul = [&](const u32x4 (&x)[NV], const u32x4 (&y)[NV]) {
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NV; ++s) {
            if (BF) {
                d = mfma_bf16(x[s], y[s], d);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) d = mfma_16x16x4(__uint_as_float(x[s][e]), __uint_as_float(y[s][e]), d);
            }
        }
        return d;
    };
    u32x4 kf[2][NV], qf[NV];
    row(rk, 0, kf[0]);
    row(rk, 1, kf[1]);
    row(rq, 0, qf);
    char* rec = ws + task * R::bytes;
    {
        float gam, sig;
        chunk_decays(aj, lane, gam, sig, [&](int b, float x) {
            if (lane < 32) f[b * kC + j] = x;
        });
        if (lane < 32) f[8 * kC + j] = aj;
        reinterpret_cast<float*>(rec + R::g)[lane] = lane < 32 ? gam : (valid ? sig : 0.f);
    }
    wave_sync();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int i = tile_row(m, lr);
        const float bi = __shfl(bj, i, 64);
        float z[8];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int b = 2 * lq + o;
            const f32x4 a4 = *reinterpret_cast<const f32x4*>(f + 8 * kC + 4 * b);
            const f32x4 dq = mul(kf[o], qf);
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            if (DELTA) d = mul(kf[o], kf[m]);
            float x = f[b * kC + i];
#pragma unroll
            for (int r = 3; r >= 0; --r) {
                if (r < 3) x = i - 4 * b == r ? 1.f : x * a4[r + 1];
                z[4 * o + r] = dq[r] * x;
                d[r] *= i - 4 * b == r ? 0.f : -bi * x;
            }
            if (DELTA) *reinterpret_cast<f32x4*>(g + i * kGS + 4 * b) = d;
        }
        if (m == 0) row(rq, 1, qf);
        put_operand(rec + R::p, m, z, lane);
    }
    if (DELTA) {
        wave_sync();
        put_t(rec, g, bj, lane);
    }
}

// Mamba-2 with bf16 keys: one wave per (slot, key head) for q_i . k_j, formed
// transposed so that a lane holds four columns of a row, and one per slot and two
// heads, lane i = token i, for the decays' products.
__global__ __launch_bounds__(256) void prep_mamba2_kernel(RaggedArgs A, char* ws, long slots) {
    typedef DecayRecord R;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int units = A.Hk + (A.H + 1) / 2;
    const long task = long(blockIdx.x) * 4 + w;
    const long slot = task / units;
    const int u = int(task - slot * units);
    int t0 = 0;
    const int clen = slot_chunk<kC>(A, slot, lane, u == 0, t0);
    if (clen == 0) return;  // no wave waits for another one below
    if (u < A.Hk) {
        const Cursor<kC> ck(A.k, t0, A.Hk, u, kK * 2), cq(A.q, t0, A.Hk, u, kK * 2);
        const __amdgpu_buffer_rsrc_t rk = ck.rsrc(clen), rq = cq.rsrc(clen);
        u32x4 kf[2][4], qf[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int at = tile_row(m, lr) * int(ck.stride) + 64 * s + 16 * lq;
                kf[m][s] = load16(rk, at);
                qf[m][s] = load16(rq, at);
            }
        char* out = ws + slots * A.H * R::bytes + (slot * A.Hk + u) * R::qk + lane * 16;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 4; ++s) d = mfma_bf16(kf[o][s], qf[m][s], d);
                *reinterpret_cast<f32x4*>(out + (2 * m + o) * kFrag) = d;
            }
        return;
    }
    const int i = lane & 31, h = 2 * (u - A.Hk) + (lane >> 5);
    const bool in = i < clen && h < A.H;
    const float av = in ? A.a[(size_t(t0) + i) * A.H + h] : 1.f;
    char* rec = ws + (slot * A.H + h) * R::bytes;
    float* f = reinterpret_cast<float*>(rec + R::f) + i;
    float r, sg;
    chunk_decays(av, lane, r, sg, [&](int g, float x) {
        if (h < A.H) f[g * kC] = x;
    });
    if (h < A.H) {
        reinterpret_cast<float*>(rec + R::a)[i] = av;
        reinterpret_cast<float*>(rec + R::g)[i] = r;
        reinterpret_cast<float*>(rec + R::g)[kC + i] = in ? sg : 0.f;
    }
}

// KDA: a decay per key channel, which does not leave the sums over channels and
// must not be divided by.  For tokens j < i let b be the highest bit in which they
// differ: all tokens with bit b set (U) against all with it clear (L), 16 each,
//   A_ij ~ sum_c (k_i a_{m+1} .. a_i) (k_j a_{j+1} .. a_m),  m the last token of L
// in the 2^{b+1}-block of i and j: one 16 x 16 product over the channels per bit,
// used where i and j share their higher bits.  The partial products of decays
// over 2^b-blocks follow from those over half blocks.  Two waves share a chunk and
// head, 64 channels each, one to a lane: with all 128 in one wave the decays' products
// alone took half its registers, and float32 keys had to be read again for every bit
// (64 sequences, 16384 tokens, 32 heads, the whole call: 841 us against 1030).  The
// scaled rows reach the fp32 matrix instruction through LDS, the sums stay in
// registers until the rows' space is free for them.
constexpr int kPS = kK / 2 + 4;  // row stride of the scaled rows, floats

template <typename QT>
__global__ __launch_bounds__(128) void prep_kda_kernel(RaggedArgs A, char* ws) {
    constexpr bool BF = std::is_same<QT, Bf16Tag>::value;
    typedef Record R;
    __shared__ __align__(16) float rows[2][48 * kPS];
    static_assert(sizeof(rows) >= 2 * kC * kGS * 4, "holds A and P in the end");
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const long task = blockIdx.x;
    const long slot = task / A.H;
    const int h = int(task - slot * A.H), hk = h / A.share;
    int t0 = 0;
    const int clen = slot_chunk<kC>(A, slot, lane, h == 0 && w == 0, t0);
    if (clen == 0) return;  // both waves

    // this lane's channel of every token; pre and suf: the decays' products over a
    // token's 2^b-block up to it and after it
    uint32_t kq[kC], q32[BF ? 1 : kC];  // bf16: key and query in one register
    float pre[kC], suf[kC];
    {
        const int c = 64 * w + lane;
        const size_t kq0 = (size_t(t0) * A.Hk + hk) * kK + c, kqs = size_t(A.Hk) * kK;
        const float* a0 = A.a + (size_t(t0) * A.H + h) * kK + c;
#pragma unroll
        for (int t = 0; t < kC; ++t) {
            const bool in = t < clen;
            const size_t at = in ? t : 0;
            typedef typename std::conditional<BF, uint16_t, uint32_t>::type bits_t;
            const uint32_t k1 = static_cast<const bits_t*>(A.k)[kq0 + at * kqs];
            const uint32_t q1 = static_cast<const bits_t*>(A.q)[kq0 + at * kqs];
            const float a1 = a0[at * A.H * kK];
            kq[t] = in ? BF ? k1 << 16 | q1 : k1 : 0u;
            if (!BF) q32[t] = in ? q1 : 0u;
            pre[t] = in ? a1 : 1.f;
            suf[t] = 1.f;
        }
    }
    auto key = [&](int t) { return __uint_as_float(BF ? kq[t] & 0xffff0000u : kq[t]); };
    auto query = [&](int t) { return __uint_as_float(BF ? kq[t] << 16 : q32[t]); };
    // 16 x 16 products of rows x and y of the scaled rows
    float* su = rows[w];
    float* sq = su + 16 * kPS;
    float* sl = su + 32 * kPS;
    auto mul = [&](const float* x, const float* y) {
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const f32x4 xa = *reinterpret_cast<const f32x4*>(x + lr * kPS + 16 * lq + 4 * s);
            const f32x4 ya = *reinterpret_cast<const f32x4*>(y + lr * kPS + 16 * lq + 4 * s);
#pragma unroll
            for (int e = 0; e < 4; ++e) d = mfma_16x16x4(xa[e], ya[e], d);
        }
        return d;
    };
    // the diagonal of P, q_i . k_i: row sums of the products
    f32x4 diag[2] = {};
#pragma unroll
    for (int t = 0; t < kC; ++t) su[t * kPS + lane] = query(t) * key(t);
    wave_sync();
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const f32x4 xa = *reinterpret_cast<const f32x4*>(su + (16 * m + lr) * kPS + 16 * lq + 4 * s);
#pragma unroll
            for (int e = 0; e < 4; ++e) diag[m] = mfma_16x16x4(xa[e], 1.f, diag[m]);
        }
    wave_sync();
    f32x4 d[5], dq[5];
#pragma unroll
    for (int b = 0; b < 5; ++b) {
        // pre, suf are over 2^b-blocks here
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const int lo = ((t >> b) << (b + 1)) | (t & ((1 << b) - 1)), up = lo | (1 << b);
            su[t * kPS + lane] = key(up) * pre[up];
            sq[t * kPS + lane] = query(up) * pre[up];
            sl[t * kPS + lane] = key(lo) * suf[lo];
        }
        wave_sync();
        d[b] = mul(su, sl);
        dq[b] = mul(sq, sl);
        wave_sync();
#pragma unroll
        for (int t = 0; t < kC; ++t)
            if (!((t >> b) & 1)) suf[t] *= pre[t | ((2 << b) - 1)];
#pragma unroll
        for (int t = 0; t < kC; ++t)
            if ((t >> b) & 1) pre[t] *= pre[(t & ~((2 << b) - 1)) | ((1 << b) - 1)];
    }
    // A and P, wave 1's part added to wave 0's
    const int j = lane & 31;
    const float bj = j < clen ? A.beta[(size_t(t0) + j) * A.H + h] : 0.f;
    float* g = rows[0];
    float* gq = g + kC * kGS;
    __syncthreads();
    if (w == 0)
        for (int i = lane; i < kC * kGS; i += 64) g[i] = gq[i] = 0.f;
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
        __syncthreads();
        if (w != turn) continue;
        wave_sync();
#pragma unroll
        for (int b = 0; b < 5; ++b) {
            const int lj = ((lr >> b) << (b + 1)) | (lr & ((1 << b) - 1));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 4 * lq + r;
                const int ui = ((t >> b) << (b + 1)) | (t & ((1 << b) - 1)) | (1 << b);
                const float bi = __shfl(bj, ui, 64);
                if ((t >> b) == (lr >> b)) {
                    g[ui * kGS + lj] += -bi * d[b][r];
                    gq[ui * kGS + lj] += dq[b][r];
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * lq + r == lr) gq[(16 * m + lr) * (kGS + 1)] += diag[m][r];
    }
    __syncthreads();
    char* rec = ws + task * R::bytes;
    if (w == 0) put_t(rec, g, bj, lane);
    else put_operands(rec + R::p, gq, nullptr, lane);
}

}  // namespace

// ---------------------------------------------------------------------------
// Segments.  With few sequences and heads a walk leaves most of the chip idle: its
// chunks follow each other.  A state passes through a segment of tokens as
// S -> M S + N, so a long sequence is cut into segments of `len` tokens and three
// launches take the walk's place: one forms M and N of every segment but the last
// (the walk without outputs, on the identity without values and on the zero
// state), one the state at each segment's end in turn, and one walks all segments
// at once from there.  Mamba-2's M is one number.
// ---------------------------------------------------------------------------
struct Segments {
    int len;     // tokens, a multiple of C; 0: none
    int most;    // segments of the longest sequence
    char* ends;  // per segment and head N [K, V], which becomes the state at its end, and M [K, K]
    // (first: the sequence's first chunk, in slots; those of sequences do not overlap)
    __device__ __forceinline__ float* n_of(uint32_t first, int seq, int seg, int H, int h, int V) const {
        return reinterpret_cast<float*>(ends) +
               ((long(first / uint32_t(len / kC)) + seq + seg) * H + h) * long(kK * V + kK * kK);
    }
};

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks: NW waves of 16 value columns each,
// V / (16 NW) blocks per sequence and head.
//
// A chunk's operands pass through LDS: T and P as the first launch left them; keys
// and queries as bf16 planes of one term (bf16 inputs, whose decays stay outside
// the products) or of three -- float32 keys and queries, and for KDA gamma K,
// gamma Q and sigma K, which are formed here from the inputs.
//   one term:    one barrier a chunk; the next chunk is on its way from memory
//                through registers to the other buffer meanwhile;
//   three terms: one buffer of planes and two barriers, between which the waves
//                form the next chunk's planes from inputs already in registers.
// ---------------------------------------------------------------------------
template <int KIND, typename QT, int NW, int HB>
struct WalkLds {  // bytes
    static constexpr bool bf = std::is_same<QT, Bf16Tag>::value, kda = KIND == SKSSM_KDA;
    static constexpr int terms = bf && !kda ? 1 : 3;
    static constexpr int v = NW * kFrag * (bf ? 1 : 2);        // a chunk's values of a head [C][16 NW]
    static constexpr int q = terms * kPlane;                   // queries' planes behind the keys'
    static constexpr int kd = 2 * terms * kPlane;              // KDA: sigma K
    static constexpr int kqbuf = (kda ? 3 : 2) * terms * kPlane;
    static constexpr int kq = 0;
    static constexpr int vals = kq + (terms == 1 ? 2 : 1) * kqbuf;
    static constexpr int rec = vals + 2 * HB * v;                  // P, (T,) gamma and sigma of two chunks
    static constexpr int p = 0, t = kTri;
    static constexpr int g = (kFormP<KIND, QT> ? 1 : 2) * kTri;
    static constexpr int recbuf = kFormP<KIND, QT> ? g + 2 * kC * 4 : Record::bytes;
    static constexpr int gp = rec + 2 * HB * recbuf;               // KDA: decays' products of token groups [8][K],
    static constexpr int gc = gp + (kda ? 8 * kK * 4 : 0);     // of the chunk [K]
    static constexpr int bytes = gc + (kda ? kK * 4 : 0);
};

// HB heads of a key head to a block, NW waves each.  ENDS: M and N of segments, no
// outputs; the columns of M follow those of N.
template <int KIND, typename QT, int NW, int HB, bool ENDS>
__global__ __launch_bounds__(HB * NW * 64)
__attribute__((amdgpu_waves_per_eu(kFormP<KIND, QT> ? 3 : 2)))
void walk_kernel(RaggedArgs A, const char* ws, long slots, int V, Segments SG) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2, KDA = KIND == SKSSM_KDA;
    constexpr bool BF = std::is_same<QT, Bf16Tag>::value;
    typedef WalkLds<KIND, QT, NW, HB> L;
    constexpr int NT = HB * NW;
    constexpr bool FORMP = kFormP<KIND, QT>, OUT = !ENDS;
    typedef Record R;
    constexpr int TERMS = L::terms;
    extern __shared__ __align__(16) char lds[];
    const int bw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // the same in every lane
    const int w = bw % NW, hb = bw / NW;                              // column tile and head in the block
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int per = (A.H / HB + 7) / 8;
    const int vslices = V / (16 * NW), slices = vslices + (ENDS && DELTA ? (kK / 16 + NW - 1) / NW : 0);
    const int xcd = blockIdx.x & 7;
    int rest = blockIdx.x >> 3;
    const int slice = rest % slices;
    rest /= slices;
    const int h = head_of<HB>(A, xcd, rest % per) + hb;
    if (h >= A.H) return;  // of all the block's heads, or none
    rest /= per;
    const int seg = SG.len ? rest % SG.most : 0;
    if (SG.len) rest /= SG.most;
    const int hk = h / A.share, seq = seq_of_rank(A, rest, lane);
    SeqSpan sp = seq_span_uniform(A, seq);
    if (!sp.live) return;
    uint32_t first;
    if (!first_slot<kC>(A, seq, sp.len, first)) return;
    // the segment's part of the sequence
    const int seq_t0 = sp.t0;
    bool at_end = true;
    int n = 1;
    if (SG.len) {
        n = max(1, (sp.len + SG.len - 1) / SG.len);
        at_end = seg == n - 1;
        if (ENDS ? seg >= n - 1 : seg >= n) return;
        sp.t0 += seg * SG.len;
        sp.len = min(SG.len, sp.len - seg * SG.len);
    }
    const bool is_m = ENDS && slice >= vslices;  // columns of M
    if (is_m && seg == 0) return;                // the first segment starts from the sequence's own state
    const int mcol = 16 * ((slice - vslices) * NW + w) + lr;
    const int col = 16 * (slice * NW + w) + lr;

    // the state: tile 2 s + o, register r <-> channel 32 s + 8 lq + 4 o + r
    f32x4 S[8];
    const int svo = (8 * lq * V + col) * 4;
    // (the last segment's state may take S0's place while the first one starts: it starts from a copy)
    if (seg > 0 ? !ENDS : sp.row0 >= 0) {
        const float* from = !ENDS && n > 1 ? SG.n_of(first, seq, seg > 0 ? seg - 1 : n - 1, A.H, h, V)
                                           : A.S0 + (size_t(sp.row0) * A.H + h) * (kK * V);
        const __amdgpu_buffer_rsrc_t s0 = buffer_rsrc(from, kK * V * 4);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[t][r] = buffer_load_f32(s0, svo, (32 * (t >> 1) + 4 * (t & 1) + r) * V * 4);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[t][r] = is_m && 32 * (t >> 1) + 8 * lq + 4 * (t & 1) + r == mcol ? 1.f : 0.f;
    }
    if (ENDS && seg == 0) {
        const __amdgpu_buffer_rsrc_t s0 = buffer_rsrc(SG.n_of(first, seq, n - 1, A.H, h, V), kK * V * 4);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                buffer_store_f32(S[t][r], s0, svo, (32 * (t >> 1) + 4 * (t & 1) + r) * V * 4);
    }

    // ---- where a chunk's data come from ----
    constexpr int E = Vec8<QT>::kElemBytes;
    const uint32_t krow = kK * E, vrow = uint32_t(V) * E;
    char* const my_vals = lds + L::vals + hb * 2 * L::v;
    char* const my_rec = lds + L::rec + hb * 2 * L::recbuf;
    Cursor<kC> ck(A.k, sp.t0, A.Hk, hk, krow), cq(A.q, sp.t0, A.Hk, hk, krow);
    Cursor<kC> cv(A.v, sp.t0, A.H, h, vrow), cy(A.y, sp.t0, A.H, h, uint32_t(V) * 4);
    Cursor<kC> ca(A.a, sp.t0, A.H, h, kK * 4);  // KDA
    constexpr int RB = FORMP ? DecayRecord::bytes : R::bytes;
    const long slot0 = long(first) + (sp.t0 - seq_t0) / kC;
    uint64_t crec = reinterpret_cast<uint64_t>(ws) + (slot0 * A.H + h) * RB;

    // Pieces of 1 KB, on their way from memory to LDS through a wave's registers:
    // those of a head's record, piece w + j NW by its wave w; of its value columns; and
    // (one term) 16 of keys and queries, four rows each, granules swizzled.
    constexpr int KQP = OUT ? 16 : 8;                 // without outputs no queries
    constexpr int RAT = OUT ? 0 : R::t;               // and no P
    constexpr int NKQ = TERMS == 1 ? (KQP + NT - 1) / NT : 0, NVP = BF ? 1 : 2;
    constexpr int NR = (R::bytes - RAT) / kFrag, NRW = FORMP ? 1 : (NR + NW - 1) / NW;
    constexpr int NP = NKQ + NRW + NVP;
    u32x4 st[NP];
    int kqoff[NKQ ? NKQ : 1], voff[NVP];
#pragma unroll
    for (int j = 0; j < NKQ; ++j) {
        const int r = 4 * ((bw + j * NT) & 7) + lq;
        kqoff[j] = int(r * ck.stride) + (lr ^ row_swizzle(r)) * 16;
    }
#pragma unroll
    for (int j = 0; j < NVP; ++j) {
        const int at = (w + j * NW) * kFrag + lane * 16;
        voff[j] = (at / (16 * E * NW)) * int(cv.stride) + at % (16 * E * NW) + slice * NW * 16 * E;
    }
    __amdgpu_buffer_rsrc_t rsk, rsq, rsv, rsr;
    const int reclane = record_lane(lane) ? lane * 16 : 1 << 30;  // out of range: reads as 0
    auto aim = [&](int rows) {  // the next chunk, `rows` tokens from its first on
        if (TERMS == 1) {
            const uint32_t n = ck.bytes(rows);
            rsk = ck.rsrc_of(n);
            rsq = cq.rsrc_of(n);
            ck.next();
            cq.next();
        }
        rsv = cv.rsrc(is_m ? 0 : rows);  // M takes no values
        cv.next();
        rsr = buffer_rsrc(reinterpret_cast<const void*>(crec), rows > 0 ? RB : 0);
        crec += uint64_t(A.H) * RB;
    };
    auto fetch = [&](int j) {
        if (j < NKQ) st[j] = load16(bw + j * NT < 8 ? rsk : rsq, kqoff[j]);
        else if (j >= NKQ + NRW) st[j] = load16(rsv, voff[j - NKQ - NRW]);
        else if (FORMP) st[j] = load16(rsr, DecayRecord::g + (lane & 15) * 16);
        else st[j] = load16(rsr, RAT + (w + (j - NKQ) * NW) * kFrag + reclane);
    };
    auto put = [&](int j, char* kq, char* v, char* rec) {
        const int o = lane * 16;
        if (j < NKQ) {
            if ((j + 1) * NT <= KQP || bw + j * NT < KQP)
                *reinterpret_cast<u32x4*>(kq + (bw + j * NT) * kFrag + o) = st[j];
        } else if (j >= NKQ + NRW) {
            *reinterpret_cast<u32x4*>(v + (w + (j - NKQ - NRW) * NW) * kFrag + o) = st[j];
        } else if (FORMP) {
            if (w == 0 && lane < 16) *reinterpret_cast<u32x4*>(rec + L::g + o) = st[j];
        } else {
            const int i = w + (j - NKQ) * NW;
            if ((j - NKQ + 1) * NW <= NR || i < NR) *reinterpret_cast<u32x4*>(rec + RAT + i * kFrag + o) = st[j];
        }
    };

    // ---- Mamba-2 with bf16 keys: P of a chunk ----
    // Waves 0 .. 3 take a task each: 16 x 16 values, lane = row tile_row(m, lr) and
    // columns 4 b .. 4 b + 3 with b = 2 lq + o; the decays between follow from F.
    uint64_t cqk = reinterpret_cast<uint64_t>(ws) + uint64_t(slots) * A.H * DecayRecord::bytes +
                   (slot0 * A.Hk + hk) * DecayRecord::qk;
    f32x4 qk = {0.f, 0.f, 0.f, 0.f}, a4 = qk;
    float f0 = 0.f;
    const int pm = (w >> 1) & 1, po = w & 1, prow = tile_row(pm, lr), pb = 2 * lq + po;
    auto load_p = [&](int rows) {  // from rsr's record: call it after aim()
        const __amdgpu_buffer_rsrc_t rq = buffer_rsrc(reinterpret_cast<const void*>(cqk), rows > 0 ? DecayRecord::qk : 0);
        qk = __builtin_bit_cast(f32x4, load16(rq, (w & 3) * kFrag + lane * 16));
        a4 = __builtin_bit_cast(f32x4, load16(rsr, DecayRecord::a + 16 * pb));
        f0 = buffer_load_f32(rsr, DecayRecord::f + (pb * kC + prow) * 4, 0);
        cqk += uint64_t(A.Hk) * DecayRecord::qk;
    };
    auto put_p = [&](char* dst) {
        float z[4], x = f0;
        z[3] = qk[3] * x;
#pragma unroll
        for (int r = 2; r >= 0; --r) {
            x = prow - 4 * pb == r ? 1.f : x * a4[r + 1];
            z[r] = qk[r] * x;
        }
        uint32_t u[3][2];
        split3<2>(z, u);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            *reinterpret_cast<u32x2*>(dst + (2 * e + pm) * kFrag + lane * 16 + 8 * po) = u32x2{u[e][0], u[e][1]};
    };

    // ---- three terms: planes from the inputs ----
    // Lane = two channels, wave w = token groups w, w + NW, .. of four tokens.
    constexpr int NG = (8 + NW - 1) / NW;
    typedef typename std::conditional<BF, uint32_t, f32x2>::type pair_t;
    pair_t kin[TERMS == 3 ? NG : 1][4], qin[TERMS == 3 ? NG : 1][4];
    f32x2 ain[KDA ? NG : 1][4];
    auto load_pair = [&](__amdgpu_buffer_rsrc_t rs, int off) {
        if constexpr (BF) return uint32_t(__builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
        else return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
    };
    auto unpack = [&](pair_t x) {
        if constexpr (BF) return f32x2{__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)};
        else return x;
    };
    auto load_inputs = [&](int rows) {
        const __amdgpu_buffer_rsrc_t rk = ck.rsrc(rows), rq = cq.rsrc(rows), ra = ca.rsrc(rows);
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * (w + n * NW) + i;  // beyond the chunk where NW does not divide 8: not used
                kin[n][i] = load_pair(rk, t * int(ck.stride) + lane * 2 * E);
                if (OUT) qin[n][i] = load_pair(rq, t * int(cq.stride) + lane * 2 * E);
                if (KDA)
                    ain[n][i] = __builtin_bit_cast(
                        f32x2, __builtin_amdgcn_raw_buffer_load_b64(ra, t * int(ca.stride) + lane * 8, 0, 0));
            }
        ck.next();
        cq.next();
        ca.next();
    };
    auto put_groups = [&](int rows) {  // KDA: each token group's decays' product
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)  // behind the sequence nothing decays
                if (4 * (w + n * NW) + i >= rows) ain[n][i] = f32x2{1.f, 1.f};
            if ((n + 1) * NW <= 8 || w + n * NW < 8)
                *reinterpret_cast<f32x2*>(lds + L::gp + ((w + n * NW) * kK + 2 * lane) * 4) =
                    (ain[n][0] * ain[n][1]) * (ain[n][2] * ain[n][3]);
        }
    };
    auto put_planes = [&]() {
        f32x2 gprod[KDA ? 8 : 1];
        if (KDA) {
#pragma unroll
            for (int g = 0; g < 8; ++g) gprod[g] = *reinterpret_cast<const f32x2*>(lds + L::gp + (g * kK + 2 * lane) * 4);
            if (w == 0) {
                f32x2 x = gprod[0];
#pragma unroll
                for (int g = 1; g < 8; ++g) x *= gprod[g];
                *reinterpret_cast<f32x2*>(lds + L::gc + 2 * lane * 4) = x;
            }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int grp = w + n * NW;
            if ((n + 1) * NW > 8 && grp >= 8) break;
            f32x2 pre[4], suf[4];
            if (KDA) {
                f32x2 p = {1.f, 1.f}, q = p;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if (g < grp) p *= gprod[g];
                    if (7 - g > grp) q *= gprod[7 - g];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p *= ain[n][i];
                    pre[i] = p;
                    suf[3 - i] = q;
                    q *= ain[n][3 - i];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * grp + i;
                char* at = lds + L::kq + r * (kK * 2) + (((lane >> 2) ^ row_swizzle(r)) * 16) + (lane & 3) * 4;
                auto three = [&](char* dst, f32x2 x) {
                    const float f[2] = {x[0], x[1]};
                    uint32_t u[3][1];
                    split3_rounded<1>(f, u);
#pragma unroll
                    for (int e = 0; e < 3; ++e) *reinterpret_cast<uint32_t*>(dst + e * kPlane) = u[e][0];
                };
                const f32x2 kx = unpack(kin[n][i]);
                three(at, KDA ? kx * pre[i] : kx);
                if (OUT) {
                    const f32x2 qx = unpack(qin[n][i]);
                    three(at + L::q, KDA ? qx * pre[i] : qx);
                }
                if (KDA) three(at + L::kd, kx * suf[i]);
            }
        }
    };

    // this lane's places in a plane: row operands, step s at xor 64 s; transposed
    // reads (a quarter-wave's lane p points at four channels of token
    // 8 lq + 4 x + p / 4, and lane i receives its row's channel of tokens
    // 8 lq + 4 x .. + 3), step s at xor 64 s, tile o at + 8 o; bf16 values likewise
    int ra[2], ta[2], va[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int row = tile_row(m, lr);
        ra[m] = row * (kK * 2) + ((lq ^ row_swizzle(row)) * 16);
        const int tk = 8 * lq + 4 * m + (lr >> 2);
        ta[m] = tk * (kK * 2) + (((lr & 3) ^ row_swizzle(tk)) * 16);
        va[m] = tk * (32 * NW) + 32 * w + 8 * (lr & 3);
    }
    auto split_state = [&](int s) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = S[2 * s + i / 4][i & 3];
        return split8(f);
    };

    // The order of a step, with one term: what it reads first, then its products with
    // the vector instructions between them.  (Left to the compiler: gdn batch 361 -> 379
    // us; with three terms the compiler's own order is the faster one, kda batch 681 ->
    // 672 us.)
    auto pin = [&]() {
        if constexpr (TERMS == 1) __builtin_amdgcn_sched_barrier(0);
    };
    auto mix = [&](auto products, auto between) {
        if constexpr (TERMS == 1) {
#pragma unroll
            for (int i = 0; i < products.value; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, between.value, 0);
            }
        }
    };
    float through = 1.f;  // Mamba-2's M
    int left = sp.len;  // tokens from chunk c on
    if (left > 0) {
        aim(left);
#pragma unroll
        for (int j = 0; j < NP; ++j) fetch(j);
        if (FORMP && OUT) {
            load_p(left);
            if (w < 4) put_p(my_rec + L::p);
        }
        if (TERMS == 3) {
            load_inputs(left);
            if (KDA) {
                put_groups(left);
                __syncthreads();
            }
            put_planes();
            load_inputs(left - kC);
        }
#pragma unroll
        for (int j = 0; j < NP; ++j) put(j, lds + L::kq, my_vals, my_rec);
        aim(left - kC);
#pragma unroll
        for (int j = 0; j < NP; ++j) fetch(j);
        if (FORMP && OUT) load_p(left - kC);
        Split sb = split_state(0);
        for (int c = 0; left > 0; ++c) {
            __syncthreads();  // everything of chunk c is there, and nobody reads chunk c - 1 any more
            const int cur = c & 1;
            const char* keys = lds + L::kq + (TERMS == 1 ? cur : 0) * L::kqbuf;
            const char* rec = my_rec + cur * L::recbuf;
            const float* gam = reinterpret_cast<const float*>(rec + L::g);
            const char* pf = rec + L::p + lane * 16;
            const char* tf = rec + L::t + lane * 16;
            const char* vals = my_vals + cur * L::v;
            aim(left - 2 * kC);

            // X = K S, Y = Q S: while a step's products run, the next step's state is
            // split, the operands of the one after are read, and a quarter of the next
            // chunk goes to LDS and of the one behind it leaves memory
            f32x4 X[2] = {}, Y[2] = {};
            constexpr int AB = TERMS == 1 ? 2 : 1;  // three terms: an operand is read where it is used
            u32x4 ka[AB][2][TERMS], qa[AB][2][TERMS], a[2][3];
            auto read_rows = [&](int s) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < TERMS; ++e) {
                        const char* p = keys + (ra[m] ^ (64 * s)) + e * kPlane;
                        if (DELTA) ka[s % AB][m][e] = *reinterpret_cast<const u32x4*>(p);
                        if (OUT) qa[s % AB][m][e] = *reinterpret_cast<const u32x4*>(p + L::q);
                    }
            };
            auto read_tri = [&](const char* f) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 3; ++e) a[m][e] = *reinterpret_cast<const u32x4*>(f + (2 * e + m) * kFrag);
            };
            read_rows(0);
            pin();
            float g[8], sg[8], wt[8], gC = 0.f;
            u32x4 vb = {0, 0, 0, 0};  // values, tokens 8 lq .. 8 lq + 7
            auto unpack_values = [&]() {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wt[2 * i] = __uint_as_float(vb[i] << 16);
                    wt[2 * i + 1] = __uint_as_float(vb[i] & 0xffff0000u);
                }
            };
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (TERMS == 1 && s < 3) read_rows(s + 1);
                if (s == 3) {
                    if (DELTA) read_tri(tf);
                    if (!KDA) {
                        load8f(gam + 8 * lq, g);
                        if (!FORMP) load8f(gam + kC + 8 * lq, sg);
                        gC = gam[kC - 1];
                    }
                }
                if (s == 2) {
                    if constexpr (BF) {
                        const u32x2 lo = tr_read(vals + va[0]), hi = tr_read(vals + va[1]);
                        vb = u32x4{lo[0], lo[1], hi[0], hi[1]};
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            wt[i] = *reinterpret_cast<const float*>(vals + ((8 * lq + i) * 16 * NW + 16 * w + lr) * 4);
                    }
                }
#pragma unroll
                for (int j = NP * s / 4; j < NP * (s + 1) / 4; ++j) {
                    put(j, lds + L::kq + (cur ^ 1) * L::kqbuf, my_vals + (cur ^ 1) * L::v, my_rec + (cur ^ 1) * L::recbuf);
                    fetch(j);
                }
                Split nb;
                if (s < 3 && (DELTA || OUT)) nb = split_state(s + 1);
                if constexpr (TERMS == 1) {
#pragma unroll
                    for (int e = 2; e >= 0; --e)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            if (DELTA) X[m] = mfma_bf16(ka[s % AB][m][0], sb.t[e], X[m]);
                            if (OUT) Y[m] = mfma_bf16(qa[s % AB][m][0], sb.t[e], Y[m]);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 6; ++e)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            if (DELTA) X[m] = mfma_bf16(ka[s % AB][m][kTermA[e]], sb.t[kTermB[e]], X[m]);
                            if (OUT) Y[m] = mfma_bf16(qa[s % AB][m][kTermA[e]], sb.t[kTermB[e]], Y[m]);
                        }
                    if (s < 3) read_rows(s + 1);
                }
                if (s < 3) {
                    if (DELTA || OUT) sb = nb;
                } else if constexpr (BF && !FORMP) {
                    unpack_values();
                }
                if (TERMS == 1) __builtin_amdgcn_sched_group_barrier(0x100, 11, 0);
                if (DELTA && OUT) mix(std::integral_constant<int, 12>(), std::integral_constant<int, 4>());
                else mix(std::integral_constant<int, 6>(), std::integral_constant<int, 8>());
                pin();
            }
            Split wb, rb;
            if (DELTA) {  // w = T (v - gamma X)
#pragma unroll
                for (int i = 0; i < 8; ++i) wt[i] = KDA ? wt[i] - X[i / 4][i & 3] : fmaf(-g[i], X[i / 4][i & 3], wt[i]);
                rb = split8(wt);
            }
            // rows of (sigma K)^T of step s
            u32x4 kt[2][2][TERMS];
            auto read_kt = [&](int s) {
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int e = 0; e < TERMS; ++e)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const u32x2 q2 = tr_read(keys + (KDA ? L::kd : 0) + e * kPlane + (ta[x] ^ (64 * s)) + 8 * o);
                            kt[s & 1][o][e][2 * x] = q2[0];
                            kt[s & 1][o][e][2 * x + 1] = q2[1];
                        }
            };
            read_kt(0);
            f32x4 d[2] = {};
            if (DELTA) {
#pragma unroll
                for (int e = 0; e < 6; ++e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) d[m] = mfma_bf16(a[m][kTermA[e]], rb.t[kTermB[e]], d[m]);
            }
            if (KDA) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    S[i] *= *reinterpret_cast<const f32x4*>(lds + L::gc + (32 * (i >> 1) + 8 * lq + 4 * (i & 1)) * 4);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    S[i] *= gC;
                    if (OUT) Y[i / 4][i & 3] *= g[i];
                }
                if (ENDS && !DELTA) through *= gC;
            }
            if (DELTA) {
#pragma unroll
                for (int i = 0; i < 8; ++i) wt[i] = d[i / 4][i & 3];
                mix(std::integral_constant<int, 12>(), std::integral_constant<int, 4>());
            }
            pin();
            // S <- gamma_C S + (sigma K)^T w
            if constexpr (FORMP) {
                load8f(gam + kC + 8 * lq, sg);
                unpack_values();
            }
            {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = KDA ? wt[i] : sg[i] * wt[i];
                rb = split8(f);
            }
            pin();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s < 3) read_kt(s + 1);
                if (OUT && s == (FORMP ? 3 : 2)) read_tri(pf);
                if (OUT && !KDA && !FORMP) {
                    uint32_t u[3][1];
                    split3<1>(wt + 2 * s, u);
#pragma unroll
                    for (int e = 0; e < 3; ++e) wb.t[e][s] = u[e][0];
                }
                if constexpr (TERMS == 1) {
#pragma unroll
                    for (int e = 2; e >= 0; --e)
#pragma unroll
                        for (int o = 0; o < 2; ++o) S[2 * s + o] = mfma_bf16(kt[s & 1][o][0], rb.t[e], S[2 * s + o]);
                } else {
#pragma unroll
                    for (int e = 0; e < 6; ++e)
#pragma unroll
                        for (int o = 0; o < 2; ++o)
                            S[2 * s + o] = mfma_bf16(kt[s & 1][o][kTermA[e]], rb.t[kTermB[e]], S[2 * s + o]);
                }
                if (TERMS == 1) __builtin_amdgcn_sched_group_barrier(0x100, 18, 0);
                mix(std::integral_constant<int, 6>(), std::integral_constant<int, 8>());
                pin();
            }
            if (KDA) wb = rb;
            // y = gamma Y + P w, beside the next chunk's first split
            if (DELTA || OUT) sb = split_state(0);
            if constexpr (ENDS) {
            } else if constexpr (FORMP) {  // w is v itself, an exact operand
#pragma unroll
                for (int e = 2; e >= 0; --e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) Y[m] = mfma_bf16(a[m][e], vb, Y[m]);
            } else {
#pragma unroll
                for (int e = 0; e < 6; ++e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) Y[m] = mfma_bf16(a[m][kTermA[e]], wb.t[kTermB[e]], Y[m]);
            }
            if (FORMP) mix(std::integral_constant<int, 6>(), std::integral_constant<int, 8>());
            else mix(std::integral_constant<int, 12>(), std::integral_constant<int, 4>());
            pin();
            if (OUT) {
                const __amdgpu_buffer_rsrc_t rs = cy.rsrc(left);
                const int at = 8 * lq * int(cy.stride) + col * 4;
#pragma unroll
                for (int i = 0; i < 8; ++i) buffer_store_f32(Y[i / 4][i & 3], rs, at + i * int(cy.stride), 0);
                cy.next();
            }
            if (FORMP && OUT) {  // P of the next chunk
                if (w < 4) put_p(my_rec + (cur ^ 1) * L::recbuf + L::p);
                load_p(left - 2 * kC);
            }
            if (TERMS == 3) {
                if (KDA) put_groups(left - kC);
                __syncthreads();  // every wave is done with the planes; the groups' products are there
                put_planes();
                load_inputs(left - 2 * kC);
            }
            left -= kC;
        }
    }
    // the last state
    if (ENDS ? is_m && mcol >= kK : !at_end) return;
    const int cols = is_m ? kK : V;
    float* to = !ENDS ? A.S + (size_t(sp.row) * A.H + h) * (kK * V)
                      : SG.n_of(first, seq, seg, A.H, h, V) + (is_m ? kK * V : 0);
    if (ENDS && !DELTA && slice == 0 && w == 0 && lane == 0) to[kK * V] = through;
    const __amdgpu_buffer_rsrc_t so = buffer_rsrc(to, kK * cols * 4);
    const int wo = (8 * lq * cols + (is_m ? mcol : col)) * 4;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) buffer_store_f32(S[t][r], so, wo, (32 * (t >> 1) + 4 * (t & 1) + r) * cols * 4);
}

// The state at the end of each segment in turn: S_g = N_g + M_g S_{g-1}.  A block has
// 16 value columns of one head, the state in LDS; wave w forms rows 32 w ..
// 32 w + 31 with the fp32 matrix instruction.  Bound by the latency of a segment's
// loads (3 segments, 32 heads of 128: 17 us; Mamba-2, 128 heads of 80: 13 us).
template <bool DELTA>
__global__ __launch_bounds__(256) void join_kernel(RaggedArgs A, int V, Segments SG) {
    constexpr int SS = 16 + 1;
    __shared__ float st[kK * SS];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int slices = V / 16;
    int rest = blockIdx.x;
    const int slice = rest % slices;
    rest /= slices;
    const int h = rest % A.H, seq = rest / A.H;
    const SeqSpan sp = seq_span_uniform(A, seq);
    if (!sp.live) return;
    uint32_t first;
    if (!first_slot<kC>(A, seq, sp.len, first)) return;
    const int n = (sp.len + SG.len - 1) / SG.len;
    const int col = 16 * slice + lr, row = 32 * w + 4 * lq;  // rows row + 16 o + r
    f32x4 c[2];
    for (int g = 0; g < n - 1; ++g) {
        float* at = SG.n_of(first, seq, g, A.H, h, V);
        if (!DELTA) {
            const float m = at[kK * V];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float* p = at + (row + 16 * (i / 4) + (i & 3)) * V + col;
                c[i / 4][i & 3] = g ? fmaf(m, c[i / 4][i & 3], *p) : *p;
                if (g) *p = c[i / 4][i & 3];
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i / 4][i & 3] = at[(row + 16 * (i / 4) + (i & 3)) * V + col];
        if (g) {
            const float* m = at + kK * V + (32 * w + lr) * kK + 32 * lq;  // lane's channels 32 lq + s
            f32x4 ma[2][8];
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int s = 0; s < 8; ++s) ma[o][s] = *reinterpret_cast<const f32x4*>(m + 16 * o * kK + 4 * s);
#pragma unroll
            for (int s = 0; s < 32; ++s) {
                const float b = st[(32 * lq + s) * SS + lr];
#pragma unroll
                for (int o = 0; o < 2; ++o) c[o] = mfma_16x16x4(ma[o][s / 4][s & 3], b, c[o]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) at[(row + 16 * (i / 4) + (i & 3)) * V + col] = c[i / 4][i & 3];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) st[(row + 16 * (i / 4) + (i & 3)) * SS + lr] = c[i / 4][i & 3];
        __syncthreads();
    }
}

namespace {

struct Cut {
    int waves, heads;  // waves of a head and heads of a block
    Segments sg;
};

template <int KIND, typename QT, int NW, int HB, bool ENDS>
hipError_t launch_walk_t(const RaggedArgs& a, const char* ws, int V, const Segments& sg, hipStream_t s) {
    const long slots = prefill_slots<kC>(a.total, a.n_seqs);
    constexpr int lds = WalkLds<KIND, QT, NW, HB>::bytes;
    static_assert(lds <= 160 * 1024, "LDS of a CU");
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(walk_kernel<KIND, QT, NW, HB, ENDS>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const int slices = V / (16 * NW) + (ENDS && KIND != SKSSM_MAMBA2 ? (kK / 16 + NW - 1) / NW : 0);
    const long blocks = long(a.n_seqs) * (sg.len ? sg.most : 1) * ((a.H / HB + 7) / 8) * 8 * slices;
    hipLaunchKernelGGL((walk_kernel<KIND, QT, NW, HB, ENDS>), dim3(uint32_t(blocks)), dim3(HB * NW * 64), lds, s, a, ws, slots, V,
                       sg);
    return hipGetLastError();
}

template <int KIND, typename QT, int NW, int HB>
hipError_t launch_walk_b(const RaggedArgs& a, const char* ws, int V, const Segments& sg, hipStream_t s) {
    if constexpr (NW < 8) {  // blocks of 8 waves walk no segments
        if (sg.len) {
            hipError_t e = launch_walk_t<KIND, QT, NW, HB, true>(a, ws, V, sg, s);
            if (e != hipSuccess) return e;
            const long blocks = long(a.n_seqs) * a.H * (V / 16);  // a few hundred thousand at most: cut_of
            hipLaunchKernelGGL((join_kernel<KIND != SKSSM_MAMBA2>), dim3(uint32_t(blocks)), dim3(256), 0, s, a, V, sg);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return launch_walk_t<KIND, QT, NW, HB, false>(a, ws, V, sg, s);
}

template <int KIND, typename QT, int NW>
hipError_t launch_walk_n(const RaggedArgs& a, const char* ws, int V, const Cut& cut, hipStream_t s) {
    if constexpr (kFormP<KIND, QT> && (NW == 5 || NW == 6))
        if (cut.heads == 2) return launch_walk_b<KIND, QT, NW, 2>(a, ws, V, cut.sg, s);
    return launch_walk_b<KIND, QT, NW, 1>(a, ws, V, cut.sg, s);
}

template <int KIND, typename QT>
hipError_t launch_walk_v(const RaggedArgs& a, const char* ws, int V, const Cut& cut, hipStream_t s) {
    switch (V) {
        case 64: return launch_walk_n<KIND, QT, 4>(a, ws, V, cut, s);
        case 80: return launch_walk_n<KIND, QT, 5>(a, ws, V, cut, s);
        case 96: return launch_walk_n<KIND, QT, 6>(a, ws, V, cut, s);
        case 112: return launch_walk_n<KIND, QT, 7>(a, ws, V, cut, s);
        case 128:
            if constexpr (KIND == SKSSM_KDA || std::is_same<QT, F32Tag>::value)
                if (cut.waves == 8) return launch_walk_n<KIND, QT, 8>(a, ws, V, cut, s);
            return launch_walk_n<KIND, QT, 4>(a, ws, V, cut, s);
    }
    return hipErrorInvalidValue;
}

template <typename QT>
hipError_t launch_prep(int kind, const RaggedArgs& a, char* ws, hipStream_t s) {
    const long tasks = prefill_slots<kC>(a.total, a.n_seqs) * a.H;
    const dim3 by4(uint32_t((tasks + 3) / 4));
    const long units = prefill_slots<kC>(a.total, a.n_seqs) * (a.Hk + (a.H + 1) / 2);
    if (kFormP<SKSSM_MAMBA2, QT> && kind == SKSSM_MAMBA2)
        hipLaunchKernelGGL(prep_mamba2_kernel, dim3(uint32_t((units + 3) / 4)), dim3(256), 0, s, a, ws,
                           prefill_slots<kC>(a.total, a.n_seqs));
    else if (kind == SKSSM_KDA) hipLaunchKernelGGL((prep_kda_kernel<QT>), dim3(uint32_t(tasks)), dim3(128), 0, s, a, ws);
    else if (kind == SKSSM_GDN) hipLaunchKernelGGL((prep_scalar_kernel<true, QT>), by4, dim3(256), 0, s, a, ws);
    else hipLaunchKernelGGL((prep_scalar_kernel<false, QT>), by4, dim3(256), 0, s, a, ws);
    return hipGetLastError();
}

}  // namespace

namespace {

size_t record_bytes(const sketchssm_shape& sh, long n_seqs, long total) {
    const size_t slots = prefill_slots<kC>(total, n_seqs);
    size_t n = slots * sh.H * Record::bytes;
    if (sh.kind == SKSSM_MAMBA2 && sh.qkv == SKSSM_BF16)
        n = slots * (size_t(sh.H) * DecayRecord::bytes + size_t(kq_heads_of(sh)) * DecayRecord::qk);
    return (n + 255) / 256 * 256;
}

// The workspace: the chunks' records, each sequence's first slot, the segments' ends.
size_t list_bytes(long n_seqs) { return (size_t(n_seqs) * sizeof(uint32_t) + 255) / 256 * 256; }

// How the walk is cut into blocks.  With few sequences the longest decides: blocks
// are counted as though all were as long as it.
//
// Two heads of a key head share a block, its keys and its queries, in Mamba-2 layers
// with bf16 keys whose head has 5 or 6 waves: a CU takes one such block of one head,
// as a SIMD takes 3 of these waves and a block's fifth and sixth go where the next
// block's would; of two heads it takes 10 or 12 waves.  us apart and together, 16384
// tokens of 64 sequences: 128 heads of 80 895, 607; 64 heads of 96 461, 350; but 64
// heads of 64, where a CU takes blocks of 4 waves anyway, 255, 281.  With less than
// a pair for three CUs of four, blocks of one head: 512 tokens of one sequence, 128
// heads of 80, 41, 52.
//
// 128 columns are two blocks of 4 waves.  With three terms a CU takes one block, and
// both form the same planes: one block of 8 waves has less to do, though a chunk of
// it lasts longer, so it is taken where such blocks fill the CUs.  us with 4 and with
// 8 waves, 32 heads: KDA, 16384 tokens of 64 sequences 1052, 755, 2000 tokens of 4 143,
// 158; GDN with float32 keys 727, 547 and 103, 121.
//
// Long sequences are cut into segments so that there is a block for each of the 256
// CUs, in segments of 256 tokens or more, where that is worth the second pass.  One
// sequence, us without and with: GDN, 32 heads of 128, 4 segments: 4096 tokens 256,
// 172 and 1024 tokens 73, 70; 64 heads, 2 segments: 4096 tokens 283, 269 and 1024
// tokens 78, 82; more segments than CUs need (64 heads, 4): 284, 297.  Mamba-2, 16
// heads of 64, 4096 tokens, 16 segments: 229, 75.  Where the second pass is cheaper
// beside the walk, half as many tokens will do: Mamba-2, which has no M, 128 heads of
// 80, 1024 tokens 93, 70; KDA, 64 heads, 2 segments of 1024 tokens 186, 181; float32 GDN,
// 32 heads of 96, 2 of 1293 224, 213.  Among many short ones most blocks of both passes
// have no segment; a sequence of 8192 tokens behind others of 8, GDN, 8 heads: 64
// others (16640 blocks) 489, 199, 256 others (65792) 498, 638; 32 heads: 64 others (8320)
// 535, 497, 256 others (32896) 610, 941.
Cut cut_of(const sketchssm_shape& sh, long n_seqs, long total, long max_len) {
    const int nw = sh.V == 128 ? 4 : sh.V / 16;
    Cut cut = {nw, 1, {0, 1, nullptr}};
    const long len = std::min(max_len, total);
    if (len <= 0) return cut;
    long per_seq = long(sh.H) * (sh.V / (16 * nw));
    const long longest = (total + len - 1) / len, most = len / 256;
    if (sh.kind == SKSSM_MAMBA2 && sh.qkv == SKSSM_BF16 && (nw == 5 || nw == 6) && sh.H / kq_heads_of(sh) % 2 == 0 &&
        longest * per_seq / 2 * std::max(most, 1l) >= 192) {
        cut.heads = 2;
        per_seq /= 2;
    }
    if (sh.V == 128 && (sh.kind == SKSSM_KDA || sh.qkv == SKSSM_F32) && longest * sh.H >= 256) cut.waves = 8;
    const long count = std::min(256 / (longest * per_seq), most);
    if (count < 2 || count * len < (sh.kind == SKSSM_GDN && sh.qkv == SKSSM_BF16 ? 4096 : 2048)) return cut;
    if (n_seqs * per_seq * count > 20000) return cut;  // most blocks would have no segment
    cut.sg.len = int((len + count - 1) / count + kC - 1) / kC * kC;
    cut.sg.most = int((len + cut.sg.len - 1) / cut.sg.len);
    return cut;
}

// Whether every launch of a call is within bounds, asked before the first one.  (The
// segments' launches are of 20000 blocks and the same again for M at most.)
bool fits(const sketchssm_shape& sh, const Cut& cut, long n_seqs, long total) {
    const int per_xcd = (sh.H / cut.heads + 7) / 8;  // of the walk's blocks, of `heads` heads each
    const int waves = sh.kind == SKSSM_KDA ? 2 * sh.H
                      : sh.kind == SKSSM_MAMBA2 && sh.qkv == SKSSM_BF16 ? kq_heads_of(sh) + (sh.H + 1) / 2
                                                                        : sh.H;  // of a chunk's preparation
    return launch_fits(double(prefill_slots<kC>(total, n_seqs)) * waves + 4, 64) &&
           launch_fits(double(n_seqs) * cut.sg.most * per_xcd * 8 * cut.heads, sh.V / 16 * 64);
}

size_t segment_bytes(const sketchssm_shape& sh, const Segments& sg, long n_seqs, long total) {
    if (!sg.len) return 0;
    return (size_t(prefill_slots<kC>(total, n_seqs)) / (sg.len / kC) + n_seqs) * sh.H * (kK * sh.V + kK * kK) * 4;
}

}  // namespace

size_t walk_workspace(const sketchssm_shape& sh, long n_seqs, long total, long max_len) {
    const Cut cut = cut_of(sh, n_seqs, total, max_len);
    if (!fits(sh, cut, n_seqs, total)) return 0;
    return record_bytes(sh, n_seqs, total) + list_bytes(n_seqs) + segment_bytes(sh, cut.sg, n_seqs, total);
}

hipError_t launch_walk(const sketchssm_shape& sh, const RaggedArgs& args, char* ws, hipStream_t s) {
    const bool bf = sh.qkv == SKSSM_BF16;
    RaggedArgs a = args;
    Cut cut = cut_of(sh, a.n_seqs, a.total, a.max_len);
    if (!fits(sh, cut, a.n_seqs, a.total)) return hipErrorInvalidConfiguration;
    char* const list = ws + record_bytes(sh, a.n_seqs, a.total);
    a.firsts = reinterpret_cast<uint32_t*>(list);
    const hipError_t e = bf ? launch_prep<Bf16Tag>(sh.kind, a, ws, s) : launch_prep<F32Tag>(sh.kind, a, ws, s);
    if (e != hipSuccess) return e;
    cut.sg.ends = list + list_bytes(a.n_seqs);
    switch (sh.kind) {
        case SKSSM_MAMBA2:
            return bf ? launch_walk_v<SKSSM_MAMBA2, Bf16Tag>(a, ws, sh.V, cut, s)
                      : launch_walk_v<SKSSM_MAMBA2, F32Tag>(a, ws, sh.V, cut, s);
        case SKSSM_GDN:
            return bf ? launch_walk_v<SKSSM_GDN, Bf16Tag>(a, ws, sh.V, cut, s)
                      : launch_walk_v<SKSSM_GDN, F32Tag>(a, ws, sh.V, cut, s);
        case SKSSM_KDA:
            return bf ? launch_walk_v<SKSSM_KDA, Bf16Tag>(a, ws, sh.V, cut, s)
                      : launch_walk_v<SKSSM_KDA, F32Tag>(a, ws, sh.V, cut, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace skssm
