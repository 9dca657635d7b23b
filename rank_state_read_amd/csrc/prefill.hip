// Prefill of ragged prompts for gfx950 (see prefill_common.h for the chunked form).
//
// Two launches for the delta rule: T depends on a chunk's own tokens alone, so
// the first forms it for all chunks of all heads at once and leaves it in the
// workspace; the second walks a sequence's chunks in order with the state in
// registers.  Mamba-2 needs the walk only.
#include <hip/hip_runtime.h>

#include <cstdlib>
#include <type_traits>

#include "prefill_common.h"

namespace skssm {

// ---------------------------------------------------------------------------
// T of every chunk and head: one wave per (slot, head).
// ---------------------------------------------------------------------------
namespace {

constexpr int kPrepWaves = 4;
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

__device__ __forceinline__ float lane_value(float x, int i) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), i));
}

// The sequence and chunk of a workspace slot: first token and tokens, none: 0.
__device__ __forceinline__ int slot_chunk(const RaggedArgs& A, long slot, int lane, int& t0) {
    for (int s0 = 0; s0 < A.n_seqs; s0 += 64) {
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
            t0 = __shfl(tc, f, 64);
            return __shfl(cl, f, 64);
        }
    }
    return 0;
}

}  // namespace

__global__ __launch_bounds__(kPrepWaves * 64) void prep_gdn_kernel(RaggedArgs A, char* ws) {
    typedef Record<SKSSM_GDN> R;
    __shared__ __align__(16) float tiles[kPrepWaves][2][kC * kGS];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const long task = long(blockIdx.x) * kPrepWaves + w;
    const long slot = task / A.H;
    const int h = int(task - slot * A.H), hk = h / A.share;
    int t0 = 0;
    const int clen = slot_chunk(A, slot, lane, t0);
    if (clen == 0) return;  // no wave waits for another one below

    // k_i . k_j and q_i . k_j: exact products of bf16 values, fp32 sums
    float* g = tiles[w][0];
    float* gq = tiles[w][1];
    const int j = lane & 31;
    const bool valid = j < clen;
    const size_t tj = size_t(t0) + (valid ? j : 0);
    const float aj = valid ? A.a[tj * A.H + h] : 1.f;
    const float bj = valid ? A.beta[tj * A.H + h] : 0.f;
    {
        u32x4 kf[2][4];
        auto row = [&](const void* base, int m, u32x4 (&f)[4]) {
            const size_t r = (size_t(t0) + min(16 * m + lr, clen - 1)) * A.Hk + hk;
            const char* src = static_cast<const char*>(base) + (r * kK + 8 * lq) * 2;
#pragma unroll
            for (int s = 0; s < 4; ++s) f[s] = *reinterpret_cast<const u32x4*>(src + 64 * s);
        };
        row(A.k, 0, kf[0]);
        row(A.k, 1, kf[1]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            u32x4 qf[4];
            row(A.q, m, qf);
#pragma unroll
            for (int n = 0; n <= m; ++n) {
                f32x4 d = {0.f, 0.f, 0.f, 0.f}, dq = d;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    d = mfma_bf16(kf[m][s], kf[n][s], d);
                    dq = mfma_bf16(qf[s], kf[n][s], dq);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = (16 * m + 4 * lq + r) * kGS + 16 * n + lr;
                    g[at] = d[r];
                    gq[at] = dq[r];
                }
            }
        }
    }
    wave_sync();

    // column j: the decays' products after token j one factor at a time (a decay may
    // be 0, so nothing is divided); lanes 0 .. 31 take -A, lanes 32 .. 63 take P
    char* rec = ws + task * R::bytes;
    {
        float* gt = lane < 32 ? g : gq;
        float d = 0.f, run = 1.f, gam = 0.f;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            const float ai = lane_value(aj, i), bi = lane_value(bj, i);
            d = i == j ? 1.f : d * ai;
            run *= ai;
            gam = i == j ? run : gam;
            const float x = d * gt[i * kGS + j];
            gt[i * kGS + j] = lane < 32 ? (i > j ? -bi * x : 0.f) : (i >= j && valid ? x : 0.f);
        }
        reinterpret_cast<float*>(rec + R::g)[lane] = lane < 32 ? gam : (valid ? d : 0.f);
    }
    wave_sync();
    // (I + A)^-1: the diagonal blocks of 16 by forward substitution, one lane per
    // column, then M_10 = M_11 (-A_10) M_00
    if (lane < 32) {
        float* b = g + (lane & 16) * (kGS + 1);
        const int l = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == l ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const f32x4 n4 = *reinterpret_cast<const f32x4*>(b + i * kGS + m);
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
        for (int i = 0; i < 16; ++i) b[i * kGS + l] = x[i];
    }
    wave_sync();
    const f32x4 r10 = block_mul(g + 16 * kGS, g, lr, lq);
    const f32x4 m10 = block_mul(g + 16 * kGS + 16, r10, lr, lq);
    wave_sync();
#pragma unroll
    for (int r = 0; r < 4; ++r) g[(16 + 4 * lq + r) * kGS + lr] = m10[r];
    wave_sync();

    // P and T = (I + A)^-1 diag(beta) as A operands
    float b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __shfl(bj, 8 * lq + i, 64);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float f[8];
        const int at = tile_row(m, lr) * kGS + 8 * lq;
        load8f(g + at, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= b[i];
        const Split t = split8(f);
        load8f(gq + at, f);
        const Split p = split8(f);
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            *reinterpret_cast<u32x4*>(rec + R::t + (2 * e + m) * kFrag + lane * 16) = t.t[e];
            *reinterpret_cast<u32x4*>(rec + R::p + (2 * e + m) * kFrag + lane * 16) = p.t[e];
        }
    }
}

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks, bf16 keys and queries, one decay per token:
// NW waves of 16 value columns, V / (16 NW) blocks per sequence and head.
//
// One barrier per chunk.  While chunk c is computed, the next chunk's keys,
// queries, values and record come from memory to registers, and then to the
// other LDS buffer.  Mamba-2 has no record: P of chunk c + 1 is formed from its
// keys and queries, so those are fetched two chunks ahead.
// ---------------------------------------------------------------------------
template <int KIND, int NW>
struct WalkLds {  // bytes
    static constexpr bool delta = KIND != SKSSM_MAMBA2;
    static constexpr int v = NW * kFrag;                       // a chunk's values [C][16 NW] in bf16
    static constexpr int kqbuf = 2 * kPlane;                   // keys, queries
    static constexpr int kq = 0;
    static constexpr int nkq = delta ? 2 : 3;
    static constexpr int vals = kq + nkq * kqbuf;              // two chunks
    static constexpr int rec = vals + 2 * v;                   // delta rule: records of two chunks
    static constexpr int p = rec;                              // Mamba-2: P of two chunks,
    static constexpr int f = p + 2 * kTri;                     // decays' products of two chunks [8][C], then a [C],
    static constexpr int fbuf = 9 * kC * 4;
    static constexpr int g = f + 2 * fbuf;                     // gamma, sigma of three chunks
    static constexpr int gbuf = 2 * kC * 4;
    static constexpr int bytes = delta ? rec + 2 * Record<SKSSM_GDN>::bytes : g + 3 * gbuf;
};

// A buffer resource whose first address moves on by a step per chunk; it covers
// `rows` rows of `row` bytes at a stride, so that tokens behind the sequence read
// as 0 and are not written.
struct Cursor {
    uint64_t at;
    uint32_t stride, row;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int rows) const {
        return buffer_rsrc(reinterpret_cast<const void*>(at), rows > 0 ? uint32_t(min(rows, kC) - 1) * stride + row : 0u);
    }
    __device__ __forceinline__ void next() { at += uint64_t(kC) * stride; }
};

template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2)))
void walk_kernel(RaggedArgs A, const char* ws, int V) {
    constexpr bool DELTA = KIND != SKSSM_MAMBA2;
    typedef WalkLds<KIND, NW> L;
    typedef Record<SKSSM_GDN> R;
    extern __shared__ __align__(16) char lds[];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // the same in every lane
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int per = (A.H + 7) / 8;
    const int slices = V / (16 * NW);
    const int xcd = blockIdx.x & 7;
    int rest = blockIdx.x >> 3;
    const int slice = rest % slices;
    rest /= slices;
    const int seq = rest / per, h = head_of(A, xcd, rest % per);
    if (h >= A.H) return;
    const int hk = h / A.share;
    const SeqSpan sp = seq_span(A, seq);
    if (!sp.live) return;
    const int col = 16 * (slice * NW + w) + lr;

    // the state: tile 2 s + o, register r <-> channel 32 s + 8 lq + 4 o + r
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

    // ---- where a chunk's data come from ----
    auto first = [&](const void* base, int heads, int head, int row) {
        return reinterpret_cast<uint64_t>(base) + (uint64_t(sp.t0) * heads + head) * uint64_t(row);
    };
    const uint32_t krow = kK * 2, vrow = uint32_t(V) * 2;
    Cursor ck{first(A.k, A.Hk, hk, krow), A.Hk * krow, krow};
    Cursor cq{first(A.q, A.Hk, hk, krow), A.Hk * krow, krow};
    Cursor cv{first(A.v, A.H, h, vrow), A.H * vrow, vrow};
    Cursor cy{first(A.y, A.H, h, 2 * vrow), A.H * 2 * vrow, 2 * vrow};
    uint64_t crec = reinterpret_cast<uint64_t>(ws) + (first_slot(sp.t0, seq) * A.H + h) * R::bytes;

    // keys and queries: 16 pieces of 1 KB (four rows), piece w + j NW by wave w;
    // granules swizzled
    constexpr int NKQ = (16 + NW - 1) / NW;
    u32x4 kq[NKQ];
    int kqoff[NKQ];
#pragma unroll
    for (int j = 0; j < NKQ; ++j) {
        const int r = 4 * ((w + j * NW) & 7) + lq;
        kqoff[j] = int(r * ck.stride) + (lr ^ row_swizzle(r)) * 16;
    }
    auto load_kq = [&](int rows) {
        const __amdgpu_buffer_rsrc_t rk = ck.rsrc(rows), rq = cq.rsrc(rows);
#pragma unroll
        for (int j = 0; j < NKQ; ++j)
            kq[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w + j * NW < 8 ? rk : rq, kqoff[j], 0, 0));
        ck.next();
        cq.next();
    };
    auto put_kq = [&](char* dst) {
#pragma unroll
        for (int j = 0; j < NKQ; ++j)
            if ((j + 1) * NW <= 16 || w + j * NW < 16)
                *reinterpret_cast<u32x4*>(dst + (w + j * NW) * kFrag + lane * 16) = kq[j];
    };
    // values: the block's columns, one piece per wave
    u32x4 vp;
    const int vat = w * kFrag + lane * 16;
    const int voff = (vat / (32 * NW)) * int(cv.stride) + vat % (32 * NW) + slice * NW * 32;
    auto load_v = [&](int rows) {
        vp = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(cv.rsrc(rows), voff, 0, 0));
        cv.next();
    };
    auto put_v = [&](char* dst) { *reinterpret_cast<u32x4*>(dst + vat) = vp; };
    // a record, piece w + j NW by wave w
    constexpr int NR = R::bytes / kFrag, NRW = DELTA ? (NR + NW - 1) / NW : 1;
    u32x4 rp[NRW];
    auto load_rec = [&](int rows) {
        const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(reinterpret_cast<const void*>(crec), rows > 0 ? R::bytes : 0);
#pragma unroll
        for (int j = 0; j < NRW; ++j)
            rp[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (w + j * NW) * kFrag + lane * 16, 0, 0));
        crec += uint64_t(A.H) * R::bytes;
    };
    auto put_rec = [&](char* dst) {
#pragma unroll
        for (int j = 0; j < NRW; ++j)
            if ((j + 1) * NW <= NR || w + j * NW < NR)
                *reinterpret_cast<u32x4*>(dst + (w + j * NW) * kFrag + lane * 16) = rp[j];
    };

    // ---- Mamba-2: decays' products and P ----
    float av = 1.f;
    bool in = false;
    auto load_a = [&](int c) {  // the decay of token lane % 32
        const int t = c * kC + (lane & 31);
        in = t < sp.len;
        av = in ? A.a[(size_t(sp.t0) + t) * A.H + h] : 1.f;
    };
    // By one wave, lane i = token i: with groups of four tokens,
    // F[b][i] = a_{4b+4} .. a_i (0 for i < 4b + 3), the decays themselves, gamma and
    // sigma.  The two half-waves write the same.
    auto put_decays = [&](char* dst, char* gs) {
        const int i = lane & 31, q = i & 3, b = i >> 2;
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
        float* f = reinterpret_cast<float*>(dst) + i;
        const float own = q == 3 ? 1.f : 0.f;
#pragma unroll
        for (int g = 7; g >= 0; --g) {
            const float bg = lane_value(up, 4 * g + 3);
            f[g * kC] = g > b ? 0.f : g == b ? own : r;
            r = g < b ? r * bg : r;
            sg = g > b ? sg * bg : sg;
        }
        f[8 * kC] = av;
        reinterpret_cast<float*>(gs)[i] = r;
        reinterpret_cast<float*>(gs)[kC + i] = in ? sg : 0.f;
    };
    // P of a chunk: four tasks (row tile m, half o of the columns), each 16 x 16
    // values of Q K^T, formed transposed so that a lane holds four columns of a row
    auto put_p = [&](int task, const char* keys, const char* dec, char* dst) {
        const int m = task >> 1, o = task & 1;
        const int ri = tile_row(m, lr), rj = tile_row(o, lr);
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const u32x4 ka = *reinterpret_cast<const u32x4*>(keys + rj * (kK * 2) + ((4 * s + lq) ^ row_swizzle(rj)) * 16);
            const u32x4 qb = *reinterpret_cast<const u32x4*>(keys + kPlane + ri * (kK * 2) +
                                                             ((4 * s + lq) ^ row_swizzle(ri)) * 16);
            d = mfma_bf16(ka, qb, d);
        }
        const float* f = reinterpret_cast<const float*>(dec);
        const int b = 2 * lq + o, dist = ri - 4 * b;  // columns 4 b .. 4 b + 3
        float x = f[b * kC + ri];
        const f32x4 a4 = *reinterpret_cast<const f32x4*>(f + 8 * kC + 4 * b);
        float z[4];
        z[3] = d[3] * x;
#pragma unroll
        for (int r = 2; r >= 0; --r) {
            x = dist == r ? 1.f : x * a4[r + 1];
            z[r] = d[r] * x;
        }
        uint32_t u[3][2];
        split3<2>(z, u);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            *reinterpret_cast<u32x2*>(dst + (2 * e + m) * kFrag + lane * 16 + 8 * o) = u32x2{u[e][0], u[e][1]};
    };

    // this lane's places in a buffer of keys: row operands, step s at xor 64 s;
    // transposed reads (a quarter-wave's lane p points at four channels of token
    // 8 lq + 4 x + p / 4, and lane i receives its row's channel of tokens
    // 8 lq + 4 x .. + 3), step s at xor 64 s, tile o at + 8 o; values likewise
    int ra[2], ta[2], va[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int row = tile_row(m, lr);
        ra[m] = row * (kK * 2) + ((lq ^ row_swizzle(row)) * 16);
        const int tk = 8 * lq + 4 * m + (lr >> 2);
        ta[m] = tk * (kK * 2) + (((lr & 3) ^ row_swizzle(tk)) * 16);
        va[m] = tk * (32 * NW) + 32 * w + 8 * (lr & 3);
    }
    auto tr_read = [&](const char* p) {
        return __builtin_bit_cast(u32x2,
                                  __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p)));
    };
    auto split_state = [&](int s) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = S[2 * s + i / 4][i & 3];
        return split8(f);
    };

    int left = sp.len;  // tokens from chunk c on
    if (left > 0) {
        load_kq(left);
        load_v(left);
        if (DELTA) load_rec(left);
        put_kq(lds + L::kq);
        put_v(lds + L::vals);
        if (DELTA) {
            put_rec(lds + L::rec);
        } else {
            load_kq(left - kC);
            if (w == NW - 1) {
                load_a(0);
                put_decays(lds + L::f, lds + L::g);
                load_a(1);
                put_decays(lds + L::f + L::fbuf, lds + L::g + L::gbuf);
                load_a(2);
            }
            put_kq(lds + L::kq + L::kqbuf);
            __syncthreads();
            if (w < 4) put_p(w, lds + L::kq, lds + L::f, lds + L::p);
        }
        int b0 = 0, b1 = 1, b2 = 2;  // Mamba-2: buffers of chunks c, c + 1, c + 2
        Split sb = split_state(0);
        for (int c = 0; left > 0; ++c) {
            __syncthreads();  // everything of chunk c is there, and nobody reads chunk c - 1 any more
            const int cur = c & 1;
            const char* keys = lds + L::kq + (DELTA ? cur : b0) * L::kqbuf;
            const char* rec = lds + L::rec + cur * R::bytes;
            const float* gam = reinterpret_cast<const float*>(DELTA ? rec + R::g : lds + L::g + b0 * L::gbuf);
            const char* pf = (DELTA ? rec + R::p : lds + L::p + cur * kTri) + lane * 16;
            const char* tf = rec + R::t + lane * 16;
            const char* vals = lds + L::vals + cur * L::v;
            load_kq(left - (DELTA ? 1 : 2) * kC);
            load_v(left - kC);
            if (DELTA) load_rec(left - kC);
            __builtin_amdgcn_sched_barrier(0);  // the loads go out before the chunk is computed

            // X = K S, Y = Q S: while a step's products run, the next step's state is
            // split and the operands of the one after are read
            f32x4 X[2] = {}, Y[2] = {};
            u32x4 ka[2][2], qa[2][2], a[2][3];
            auto read_rows = [&](int s) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const char* p = keys + (ra[m] ^ (64 * s));
                    if (DELTA) ka[s & 1][m] = *reinterpret_cast<const u32x4*>(p);
                    qa[s & 1][m] = *reinterpret_cast<const u32x4*>(p + kPlane);
                }
            };
            auto read_tri = [&](const char* f) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 3; ++e) a[m][e] = *reinterpret_cast<const u32x4*>(f + (2 * e + m) * kFrag);
            };
            read_rows(0);
            __builtin_amdgcn_sched_barrier(0);
            float g[8], sg[8], wt[8], gC = 0.f;
            u32x4 vb = {0, 0, 0, 0};  // values, tokens 8 lq .. 8 lq + 7: an exact B operand
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s < 3) {
                    read_rows(s + 1);
                } else {
                    if (DELTA) read_tri(tf);
                    load8f(gam + 8 * lq, g);
                    load8f(gam + kC + 8 * lq, sg);
                    gC = gam[kC - 1];
                }
                if (s == 2) {
                    const u32x2 lo = tr_read(vals + va[0]), hi = tr_read(vals + va[1]);
                    vb = u32x4{lo[0], lo[1], hi[0], hi[1]};
                }
                Split nb;
                if (s < 3) nb = split_state(s + 1);
#pragma unroll
                for (int e = 2; e >= 0; --e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (DELTA) X[m] = mfma_bf16(ka[s & 1][m], sb.t[e], X[m]);
                        Y[m] = mfma_bf16(qa[s & 1][m], sb.t[e], Y[m]);
                    }
                if (s < 3) {
                    sb = nb;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        wt[2 * i] = __uint_as_float(vb[i] << 16);
                        wt[2 * i + 1] = __uint_as_float(vb[i] & 0xffff0000u);
                    }
                }
                __builtin_amdgcn_sched_group_barrier(0x100, 11, 0);
#pragma unroll
                for (int i = 0; i < (DELTA ? 12 : 6); ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, DELTA ? 4 : 8, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            Split wb, rb;
            if (DELTA) {  // w = T (v - gamma X)
#pragma unroll
                for (int i = 0; i < 8; ++i) wt[i] = fmaf(-g[i], X[i / 4][i & 3], wt[i]);
                rb = split8(wt);
            }
            // rows of K^T of step s
            u32x4 kt[2][2];
            auto read_kt = [&](int s) {
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const u32x2 q2 = tr_read(keys + (ta[x] ^ (64 * s)) + 8 * o);
                        kt[s & 1][o][2 * x] = q2[0];
                        kt[s & 1][o][2 * x + 1] = q2[1];
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
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                S[i] *= gC;
                Y[i / 4][i & 3] *= g[i];
            }
            if (DELTA) {
#pragma unroll
                for (int i = 0; i < 8; ++i) wt[i] = d[i / 4][i & 3];
            }
            // S <- gamma_C S + K^T (sigma w)
            {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = sg[i] * wt[i];
                rb = split8(f);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s < 3) read_kt(s + 1);
                if (s == 2) read_tri(pf);
                if (DELTA && s == 0) wb = split8(wt);
#pragma unroll
                for (int e = 2; e >= 0; --e)
#pragma unroll
                    for (int o = 0; o < 2; ++o) S[2 * s + o] = mfma_bf16(kt[s & 1][o], rb.t[e], S[2 * s + o]);
                __builtin_amdgcn_sched_group_barrier(0x100, 10, 0);
#pragma unroll
                for (int i = 0; i < 6; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // y = gamma Y + P w, beside the next chunk's first split
            sb = split_state(0);
            if (DELTA) {
#pragma unroll
                for (int e = 0; e < 6; ++e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) Y[m] = mfma_bf16(a[m][kTermA[e]], wb.t[kTermB[e]], Y[m]);
            } else {
#pragma unroll
                for (int e = 2; e >= 0; --e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) Y[m] = mfma_bf16(a[m][e], vb, Y[m]);
            }
#pragma unroll
            for (int i = 0; i < (DELTA ? 12 : 6); ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, DELTA ? 4 : 8, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            {
                const __amdgpu_buffer_rsrc_t rs = cy.rsrc(left);
                const int at = 8 * lq * int(cy.stride) + col * 4;
#pragma unroll
                for (int i = 0; i < 8; ++i) buffer_store_f32(Y[i / 4][i & 3], rs, at + i * int(cy.stride), 0);
                cy.next();
            }
            // the chunks to come
            put_v(lds + L::vals + (cur ^ 1) * L::v);
            if (DELTA) {
                put_kq(lds + L::kq + (cur ^ 1) * L::kqbuf);
                put_rec(lds + L::rec + (cur ^ 1) * R::bytes);
            } else {
                if (w < 4)
                    put_p(w, lds + L::kq + b1 * L::kqbuf, lds + L::f + (cur ^ 1) * L::fbuf, lds + L::p + (cur ^ 1) * kTri);
                put_kq(lds + L::kq + b2 * L::kqbuf);
                if (w == NW - 1) {
                    put_decays(lds + L::f + cur * L::fbuf, lds + L::g + b2 * L::gbuf);
                    load_a(c + 3);
                }
                const int t = b0;
                b0 = b1;
                b1 = b2;
                b2 = t;
            }
            left -= kC;
        }
    }
    const __amdgpu_buffer_rsrc_t so = buffer_rsrc(A.S + (size_t(sp.row) * A.H + h) * (kK * V), kK * V * 4);
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) buffer_store_f32(S[t][r], so, svo, (32 * (t >> 1) + 4 * (t & 1) + r) * V * 4);
}

namespace {

template <int KIND, int NW>
hipError_t launch_walk_t(const RaggedArgs& a, const char* ws, int V, hipStream_t s) {
    constexpr int lds = WalkLds<KIND, NW>::bytes;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(walk_kernel<KIND, NW>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const long blocks = long(a.n_seqs) * ((a.H + 7) / 8) * 8 * (V / (16 * NW));
    hipLaunchKernelGGL((walk_kernel<KIND, NW>), dim3(uint32_t(blocks)), dim3(NW * 64), lds, s, a, ws, V);
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_walk(const RaggedArgs& a, const char* ws, int V, hipStream_t s) {
    switch (V) {
        case 64: return launch_walk_t<KIND, 4>(a, ws, V, s);
        case 80: return launch_walk_t<KIND, 5>(a, ws, V, s);
        case 96: return launch_walk_t<KIND, 6>(a, ws, V, s);
        case 112: return launch_walk_t<KIND, 7>(a, ws, V, s);
        case 128: return getenv("NW8") ? launch_walk_t<KIND, 8>(a, ws, V, s) : launch_walk_t<KIND, 4>(a, ws, V, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_gdn(const RaggedArgs& a, char* ws, int V, hipStream_t s) {
    const long tasks = prefill_slots(a.total, a.n_seqs) * a.H;
    hipLaunchKernelGGL(prep_gdn_kernel, dim3(uint32_t((tasks + kPrepWaves - 1) / kPrepWaves)), dim3(kPrepWaves * 64), 0,
                       s, a, ws);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_walk<SKSSM_GDN>(a, ws, V, s) : e;
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
    if (!chunked(*shape, max_len) || shape->kind == SKSSM_MAMBA2) return 0;
    return size_t(prefill_slots(total_tokens, n_seqs)) * shape->H * Record<SKSSM_GDN>::bytes;
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
        if (double(n_seqs) * (shape->H + 7) >= 2147483648.0) return SKSSM_ESHAPE;
        char* ws = static_cast<char*>(workspace);
        e = shape->kind == SKSSM_MAMBA2 ? launch_walk<SKSSM_MAMBA2>(A, ws, shape->V, s) : launch_gdn(A, ws, shape->V, s);
    }
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
