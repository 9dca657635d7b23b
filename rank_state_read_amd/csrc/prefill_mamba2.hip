// Prefill of Mamba-2 layers (bf16 keys, queries and values) for gfx950.
#include <hip/hip_runtime.h>

#include "prefill_common.h"

namespace skssm {

namespace {

constexpr int kC = 32;
constexpr int kTri = 3 * 2 * kFrag;
constexpr int kPlane = kC * kK * 2;

struct NoRecord {
    static constexpr int p = 0, t = 0, g = 0, bytes = 1024;
};
__device__ __forceinline__ float lane_value(float x, int i) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), i));
}

}  // namespace

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks, bf16 keys and queries, one decay per token:
// NW waves of 16 value columns, V / (16 NW) blocks per sequence and head.
//
// One barrier per chunk.  While chunk c is computed, the next chunk's keys,
// queries, values and record come from memory to registers, and then to the
// other LDS buffer.  Mamba-2 has no record: P of chunk c + 1 is formed from its
// keys and queries, so those are fetched two chunks ahead.
// ---------------------------------------------------------------------------
template <int NW>
struct Mamba2Lds {  // bytes
    static constexpr int v = NW * kFrag;                       // a chunk's values [C][16 NW] in bf16
    static constexpr int kqbuf = 2 * kPlane;                   // keys, queries
    static constexpr int kq = 0;
    static constexpr int nkq = 3;
    static constexpr int vals = kq + nkq * kqbuf;              // two chunks
    static constexpr int rec = vals + 2 * v;                   // delta rule: records of two chunks
    static constexpr int p = rec;                              // Mamba-2: P of two chunks,
    static constexpr int f = p + 2 * kTri;                     // decays' products of two chunks [8][C], then a [C],
    static constexpr int fbuf = 9 * kC * 4;
    static constexpr int g = f + 2 * fbuf;                     // gamma, sigma of three chunks
    static constexpr int gbuf = 2 * kC * 4;
    static constexpr int bytes = g + 3 * gbuf;
};

template <int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2)))
void walk_mamba2_kernel(RaggedArgs A, int V) {
    constexpr bool DELTA = false;
    typedef Mamba2Lds<NW> L;
    typedef NoRecord R;
    const char* ws = nullptr;
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
    const uint32_t krow = kK * 2, vrow = uint32_t(V) * 2;
    Cursor<kC> ck(A.k, sp.t0, A.Hk, hk, krow), cq(A.q, sp.t0, A.Hk, hk, krow);
    Cursor<kC> cv(A.v, sp.t0, A.H, h, vrow), cy(A.y, sp.t0, A.H, h, 2 * vrow);
    uint64_t crec = reinterpret_cast<uint64_t>(ws) + (first_slot<kC>(sp.t0, seq) * A.H + h) * R::bytes;

    // Pieces of 1 KB, on their way from memory to LDS through a wave's registers:
    // 16 of keys and queries (four rows each, granules swizzled) and those of the
    // record, piece w + j NW by wave w, and one of the block's value columns.
    constexpr int NKQ = (16 + NW - 1) / NW, NR = R::bytes / kFrag, NRW = DELTA ? (NR + NW - 1) / NW : 0;
    constexpr int NP = NKQ + 1 + NRW;
    u32x4 st[NP];
    int kqoff[NKQ];
#pragma unroll
    for (int j = 0; j < NKQ; ++j) {
        const int r = 4 * ((w + j * NW) & 7) + lq;
        kqoff[j] = int(r * ck.stride) + (lr ^ row_swizzle(r)) * 16;
    }
    const int vat = w * kFrag + lane * 16;
    const int voff = (vat / (32 * NW)) * int(cv.stride) + vat % (32 * NW) + slice * NW * 32;
    __amdgpu_buffer_rsrc_t rsk, rsq, rsv, rsr;
    auto aim_kq = [&](int rows) {  // the next chunk's keys and queries, `rows` tokens from its first on
        rsk = ck.rsrc(rows);
        rsq = cq.rsrc(rows);
        ck.next();
        cq.next();
    };
    auto aim_v = [&](int rows) {
        rsv = cv.rsrc(rows);
        cv.next();
        if (DELTA) {
            rsr = buffer_rsrc(reinterpret_cast<const void*>(crec), rows > 0 ? R::bytes : 0);
            crec += uint64_t(A.H) * R::bytes;
        }
    };
    auto fetch = [&](int j) {
        if (j < NKQ)
            st[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w + j * NW < 8 ? rsk : rsq, kqoff[j], 0, 0));
        else if (j == NKQ)
            st[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsv, voff, 0, 0));
        else
            st[j] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsr, (w + (j - NKQ - 1) * NW) * kFrag + lane * 16, 0, 0));
    };
    auto put = [&](int j, char* kq, char* v, char* rec) {
        const int o = lane * 16;
        if (j < NKQ) {
            if ((j + 1) * NW <= 16 || w + j * NW < 16) *reinterpret_cast<u32x4*>(kq + (w + j * NW) * kFrag + o) = st[j];
        } else if (j == NKQ) {
            *reinterpret_cast<u32x4*>(v + vat) = st[j];
        } else {
            const int i = w + (j - NKQ - 1) * NW;
            if ((j - NKQ) * NW <= NR || i < NR) *reinterpret_cast<u32x4*>(rec + i * kFrag + o) = st[j];
        }
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
    auto split_state = [&](int s) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = S[2 * s + i / 4][i & 3];
        return split8(f);
    };

    int left = sp.len;  // tokens from chunk c on
    if (left > 0) {
        aim_kq(left);
        aim_v(left);
#pragma unroll
        for (int j = 0; j < NP; ++j) fetch(j);
#pragma unroll
        for (int j = 0; j < NP; ++j) put(j, lds + L::kq, lds + L::vals, lds + L::rec);
        aim_kq(left - kC);
        aim_v(left - kC);
#pragma unroll
        for (int j = 0; j < NP; ++j) fetch(j);
        if (!DELTA) {
            if (w == NW - 1) {
                load_a(0);
                put_decays(lds + L::f, lds + L::g);
                load_a(1);
                put_decays(lds + L::f + L::fbuf, lds + L::g + L::gbuf);
                load_a(2);
            }
            aim_kq(left - 2 * kC);
#pragma unroll
            for (int j = 0; j < NKQ; ++j) put(j, lds + L::kq + L::kqbuf, nullptr, nullptr);
#pragma unroll
            for (int j = 0; j < NKQ; ++j) fetch(j);
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
            aim_kq(left - (DELTA ? 2 : 3) * kC);
            aim_v(left - 2 * kC);

            // X = K S, Y = Q S: while a step's products run, the next step's state is
            // split, the operands of the one after are read, and a quarter of the next
            // chunk goes to LDS and of the one behind it leaves memory
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
#pragma unroll
                for (int j = NP * s / 4; j < NP * (s + 1) / 4; ++j) {
                    put(j, lds + L::kq + (DELTA ? cur ^ 1 : b2) * L::kqbuf, lds + L::vals + (cur ^ 1) * L::v,
                        lds + L::rec + (cur ^ 1) * R::bytes);
                    fetch(j);
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
#pragma unroll
                for (int i = 0; i < 12; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
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
                if (DELTA) {
                    uint32_t u[3][1];
                    split3<1>(wt + 2 * s, u);
#pragma unroll
                    for (int e = 0; e < 3; ++e) wb.t[e][s] = u[e][0];
                }
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
            if (!DELTA) {  // P of the next chunk, decays of the one behind it
                if (w < 4)
                    put_p(w, lds + L::kq + b1 * L::kqbuf, lds + L::f + (cur ^ 1) * L::fbuf, lds + L::p + (cur ^ 1) * kTri);
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

template <int NW>
hipError_t launch_mamba2_t(const RaggedArgs& a, int V, hipStream_t s) {
    constexpr int lds = Mamba2Lds<NW>::bytes;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(walk_mamba2_kernel<NW>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const long blocks = long(a.n_seqs) * ((a.H + 7) / 8) * 8 * (V / (16 * NW));
    if (blocks >= (1l << 31)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((walk_mamba2_kernel<NW>), dim3(uint32_t(blocks)), dim3(NW * 64), lds, s, a, V);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mamba2(const RaggedArgs& a, int V, hipStream_t s) {
    switch (V) {
        case 64: return launch_mamba2_t<4>(a, V, s);
        case 80: return launch_mamba2_t<5>(a, V, s);
        case 96: return launch_mamba2_t<6>(a, V, s);
        case 112: return launch_mamba2_t<7>(a, V, s);
        case 128: return launch_mamba2_t<8>(a, V, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace skssm
