// What the prefill kernels share: chunks of C = 32 tokens, operands of the bf16
// matrix instruction with fp32 precision, and the walk's work on one chunk.
//
// Per sequence and head, within a chunk that starts at state S, with gamma_i the
// decays' product up to token i, gamma_ij that after j up to i and sigma_j that
// after j to the chunk's end (per key channel for KDA):
//   A_ij = beta_i sum_c gamma_ij k_i k_j  (j < i),   P_ij = sum_c gamma_ij q_i k_j  (j <= i)
//   T    = (I + A)^-1 diag(beta)                      (Mamba-2: w = v instead)
//   w    = T (v - (gamma K) S),   y = (gamma Q) S + P w,   S <- gamma_C S + (sigma K)^T w
//
// Products run on the bf16 matrix instruction (16x16x32, fp32 sums) and keep
// fp32 precision: an fp32 operand x is written as hi + mid + lo, three bf16
// numbers of 8 significant bits each, without a rest.  q, k, v in bf16 are exact
// operands, so their products with an fp32 operand take three instructions, products
// of two fp32 operands six: hi hi, hi mid, mid hi, mid mid, hi lo, lo hi.  The rest is
// left out, two products of mid and lo of up to 2^-22 of hi hi each and lo lo.  The A
// operand's terms (T, P, the planes of keys and queries) are rounded, so that mid and lo
// have either sign and what is left out has a mean of 0; the B operand's (the state, w),
// formed on the chain of a walk's steps, are cut off, and so is a P beside bf16 values,
// where nothing is left out.  Relative to the product, over normal
// values: mean 0, mean square (1.8e-8)^2, at most 1.5e-7 (both cut off: mean -4.1e-8,
// mean square (6.0e-8)^2, at most 4.0e-7; a rounding to fp32: (2.5e-8)^2, 6.0e-8).  The
// fp32 matrix instruction has 1/16 of the bf16 rate.
//
// Value columns are independent of each other.  In the walk over a sequence's
// chunks one wave owns 16 of them for all 128 key channels, so that nothing it
// computes has to reach another wave: the accumulator layout (lane l, register r
// <-> row 4 (l/16) + r, column l % 16) becomes the next product's B operand
// (lane l <-> 8 consecutive rows from 8 (l/16), column l % 16) without leaving
// the lane.  Rows 4 q + r of the two tiles of a 32-row group stand for group rows
// 8 q + r and 8 q + 4 + r, which the A operand's rows follow.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "ragged.h"
#include "sketchssm_internal.h"

namespace skssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kFrag = 64 * 16;  // one operand of a wave, bytes

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// x = term 0 + term 1 + term 2 exactly, for 2 N consecutive values: eight of an fp32
// number's 24 bits each, cut off.  (Rounded terms, as below, cost a conversion and a
// shift where these cost a permutation and a mask; with those here too: mamba2 batch
// 484 us against 467, gdn long 614 against 584.  The remainders could be bf16 dot
// products with (-1, 0) and (0, -1), one instruction instead of two, but those share the
// matrix unit: three beside a matrix instruction take 40 cycles, three subtractions 21.)
template <int N>
__device__ __forceinline__ void split3(const float* f, uint32_t (&u)[3][N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x0 = f[2 * i], x1 = f[2 * i + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
            u[p][i] = __builtin_amdgcn_perm(b1, b0, 0x07060302);  // the upper halves
            x0 -= __uint_as_float(b0 & 0xffff0000u);
            x1 -= __uint_as_float(b1 & 0xffff0000u);
        }
    }
}

// The same with rounded terms, exact as well: what two of them leave has at most 7 bits.
// (A finite value beyond bf16's largest, 3.39e38, becomes inf.)
template <int N>
__device__ __forceinline__ void split3_rounded(const float* f, uint32_t (&u)[3][N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x0 = f[2 * i], x1 = f[2 * i + 1];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t h = pack_bf16(x0, x1);
            u[p][i] = h;
            x0 -= __uint_as_float(h << 16);
            x1 -= __uint_as_float(h & 0xffff0000u);
        }
        u[2][i] = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302);
    }
}

// Eight values as a B operand of three terms.
struct Split {
    u32x4 t[3];
};
__device__ __forceinline__ Split split8(const float* f) {
    uint32_t u[3][4];
    split3<4>(f, u);
    Split s;
#pragma unroll
    for (int p = 0; p < 3; ++p) s.t[p] = u32x4{u[p][0], u[p][1], u[p][2], u[p][3]};
    return s;
}

// Row i of row tile m of a 32-row group (see above).
__device__ __forceinline__ int tile_row(int m, int i) { return 8 * (i >> 2) + 4 * m + (i & 3); }

// Granule of 16 bytes g of a plane's token row r sits at granule g ^ row_swizzle(r):
// the 16 rows of a tile start in different banks, and the 16 pieces that a
// quarter-wave's transposed read collects lie in all of them.
__device__ __forceinline__ int row_swizzle(int r) { return (r & 3) | (((r >> 3) & 3) << 2); }

// The products of three-term operands that matter, small ones first.
__device__ constexpr int kTermA[6] = {2, 0, 1, 1, 0, 0};
__device__ constexpr int kTermB[6] = {0, 2, 1, 0, 1, 0};

// A sequence's chunks have consecutive slots of the workspace, behind those of the live
// sequences before it in the list.  Sequences that do not overlap have at most
// total / C + n_seqs chunks together, whatever their order.  (Slots counted from a
// sequence's first token, t0 / C + seq, need no sums but hold only where the offsets
// never decrease.)  Lists with sequences that overlap may ask for more: those that no
// slot is left for take part no further.  Sums are modulo 2^32, which such lists alone
// can reach.
template <int C>
__host__ __device__ inline long prefill_slots(long total, long n_seqs) {
    return total / C + n_seqs;
}
template <int C>
__device__ __forceinline__ uint32_t chunks_of(uint32_t tokens) {
    return (tokens + C - 1) / C;
}
template <int C>
__device__ __forceinline__ bool has_room(const RaggedArgs& A, uint32_t first, uint32_t n) {
    const uint32_t slots = uint32_t(prefill_slots<C>(A.total, A.n_seqs));
    return first <= slots && n <= slots - first;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_mov_u32(uint32_t x) {  // 0 where there is no source
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, ROWS, 0xF, false));
}
// Sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
    x += dpp_mov_u32<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8
    x += dpp_mov_u32<0x112, 0xF>(x);
    x += dpp_mov_u32<0x114, 0xF>(x);
    x += dpp_mov_u32<0x118, 0xF>(x);
    x += dpp_mov_u32<0x142, 0xA>(x);  // row_bcast 15 into rows 1 and 3
    x += dpp_mov_u32<0x143, 0xC>(x);  // row_bcast 31 into rows 2 and 3
    return x;
}

// The sequence and chunk of a workspace slot: first token and tokens, none: 0.  One wave
// of each slot notes its sequence's first slot for the launches behind (`note`).
template <int C>
__device__ __forceinline__ int slot_chunk(const RaggedArgs& A, long slot, int lane, bool note, int& t0) {
    uint32_t before = 0;
    for (int s0 = 0; s0 < A.n_seqs; s0 += 64) {
        const int s = s0 + lane;
        const SeqSpan sp = seq_span(A, min(s, A.n_seqs - 1));
        const uint32_t n = s < A.n_seqs && sp.live ? chunks_of<C>(sp.len) : 0;
        const uint32_t upto = before + wave_scan(n), first = upto - n, c = uint32_t(slot) - first;
        const bool hit = c < n && has_room<C>(A, first, n);
        const unsigned long long m = __ballot(hit);
        if (m) {
            if (note && hit && c == 0) A.firsts[s] = first;
            const int f = __ffsll(m) - 1, at = hit ? int(c) * C : 0;
            t0 = __builtin_amdgcn_readlane(sp.t0 + at, f);
            return __builtin_amdgcn_readlane(min(C, sp.len - at), f);
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return 0;
}

// The first slot of live sequence `seq` of `tokens` tokens.  (An empty one has none, and
// one that found no room whatever the workspace held: out of range, or undefined as
// the results of lists with overlaps are.)
template <int C>
__device__ __forceinline__ bool first_slot(const RaggedArgs& A, int seq, int tokens, uint32_t& first) {
    first = 0;
    if (tokens == 0) return true;
    if (seq > 0) first = __builtin_amdgcn_readfirstlane(A.firsts[seq]);
    return has_room<C>(A, first, chunks_of<C>(tokens));
}

// The sequence that the r-th group of blocks takes: the longest first, so that the
// last blocks to start are short ones.  In full order up to 64 sequences, one per
// lane; with more only the long ones go first (us of a GDN layer, 32 heads of 128,
// 99 sequences of 100 tokens and behind them one of 6000: 529 against 630 in the order
// they come in; 100 of 160 tokens: 425, 428).
__device__ __forceinline__ int seq_of_rank(const RaggedArgs& A, int r, int lane) {
    if (A.n_seqs > 64) return seq_long_first(A, r, lane);
    const long n = lane < A.n_seqs ? long(A.offsets[lane + 1]) - A.offsets[lane] : -1;
    const int len = int(min(max(n, lane < A.n_seqs ? 0l : -1l), long(A.total)));  // the lists may hold anything
    int rank = 0;
    for (int j = 0; j < A.n_seqs; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane) ? 1 : 0;
    }
    return __ffsll(__ballot(lane < A.n_seqs && rank == r)) - 1;
}

// The rows of one head over a sequence's chunks: a buffer resource whose first
// address moves on by C tokens a time and which ends with the sequence, so that
// what lies behind it reads as 0 and is not written.
template <int C>
struct Cursor {
    uint64_t at;
    uint32_t stride, row;
    __device__ __forceinline__ Cursor(const void* base, int t0, int heads, int head, uint32_t row_bytes)
        : at(reinterpret_cast<uint64_t>(base) + (uint64_t(t0) * heads + head) * row_bytes),
          stride(heads * row_bytes),
          row(row_bytes) {}
    // bytes of a chunk with `rows` tokens from its first to the end of the sequence
    __device__ __forceinline__ uint32_t bytes(int rows) const {
        // (the compiler takes vector registers for this, which a resource must not have)
        return __builtin_amdgcn_readfirstlane(rows >= C ? (C - 1) * stride + row
                                              : rows > 0 ? (rows - 1) * stride + row
                                                         : 0u);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(uint32_t n) const {
        return buffer_rsrc(reinterpret_cast<const void*>(at), n);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int rows) const { return rsrc_of(bytes(rows)); }
    __device__ __forceinline__ void next() { at += uint64_t(C) * stride; }
};

// Transposed LDS read: lane p of a quarter-wave points at four consecutive bf16
// values; lane i receives value i % 4 of lanes i / 4, 4 + i / 4, 8 + i / 4, 12 + i / 4.
__device__ __forceinline__ u32x2 tr_read(const char* p) {
    return __builtin_bit_cast(u32x2,
                              __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p)));
}

// The heads' order over the blocks: those that share a key head sit on one XCD
// (blocks go round the eight by index).  First head of unit u of XCD x, a unit being
// HB heads of one key head, or >= H.
template <int HB>
__device__ __forceinline__ int head_of(const RaggedArgs& A, int x, int u) {
    const int share = A.share / HB;
    return HB * (A.Hk % 8 == 0 ? (x + 8 * (u / share)) * share + u % share : x + 8 * u);
}

// The chunked form's launches (prefill_walk.hip).
size_t walk_workspace(const sketchssm_shape& sh, long n_seqs, long total, long max_len);
hipError_t launch_walk(const sketchssm_shape& sh, const RaggedArgs& a, char* ws, hipStream_t s);

}  // namespace skssm
