// States cached in 8 bits on gfx950.  Per key row of V state values one scale s:
//   i8    s = the least bf16 number >= 2^-100 with 127 s >= max|x|, code = x / s to
//         the nearest whole number
//   e4m3  s = the least power of two >= 2^-100 with 448 s >= max|x|, code = the e4m3
//         number nearest to x / s
// both with ties to even and without any rounding before that one, so that a code
// does not depend on how it is computed.  A row that holds an infinity or a NaN gets
// the scale NaN and reads back as NaN.
//
// 48 states of 128 heads of 128 x 80 (316 MB each way): loaded in 54 us in both formats (5.8 TB/s, most of it
// writes), which is memory's time; stored in 68 us in whole numbers and 64 in e4m3 (4.7 and 4.9 TB/s, most of it
// reads).  A store in whole numbers has 786 vector instructions a wave, which keep the vector units busy all along,
// the one in e4m3 327: what the others cost beside its loads is the 4 us between them.  96 states of 32 heads of
// 128 x 128 in e4m3 loaded in 37 (5.5 TB/s).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "sketchssm_internal.h"

namespace skssm {

namespace {

constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100

struct CacheArgs {
    const float* S;
    float* out;  // state rows written by a load
    void* codes;
    uint16_t* scales;
    const int32_t* rows;
    const int32_t* slots;
    int B, n_slots, n;
    int H;
};

__device__ __forceinline__ uint32_t row_max16(uint32_t x) {
    auto other = [&](auto ctrl) {
        return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    x = max(x, other(std::integral_constant<int, 0xB1>()));
    x = max(x, other(std::integral_constant<int, 0x4E>()));
    x = max(x, other(std::integral_constant<int, 0x141>()));
    x = max(x, other(std::integral_constant<int, 0x140>()));
    return x;
}

// The scale of a row whose largest magnitude is `top` (finite): its bf16 bits in the
// upper half.  127 s and 448 s are exact in fp32.
template <int FMT>
__device__ __forceinline__ uint32_t scale_bits(float top) {
    if constexpr (FMT == SKSSM_CACHE_I8) {
        // truncated to bf16, at most one step below the answer
        const uint32_t b = __float_as_uint(fmaxf(top / 127.f, kMinScale)) & 0xffff0000u;
        return 127.f * __uint_as_float(b) >= top ? b : b + 0x10000u;
    } else {
        const uint32_t b = __float_as_uint(fmaxf(top / 448.f, kMinScale)) & 0x7f800000u;
        return 448.f * __uint_as_float(b) >= top ? b : b + 0x800000u;
    }
}

// x / s to the nearest whole number, ties to even.  The product with the rounded 1 / s is off by
// less than one; what it leaves of x is exact in fp32 and puts the neighbours right.
__device__ __forceinline__ int code_i8(float x, float s, float inv) {
    float n = rintf(x * inv);
    const float left = fmaf(-n, s, x);
    const float half = 0.5f * s;
    const bool odd = (int(n) & 1) != 0;
    if (left > half || (left == half && odd)) n += 1.f;
    if (left < -half || (left == -half && odd)) n -= 1.f;
    return int(n);
}

}  // namespace

// A team of 16 lanes takes kRows key rows: lane l has values 4 l .. 4 l + 3 and, where the row
// is longer, 64 + 4 l .. 64 + 4 l + 3, so that a row's load and store cover whole lines (one row a team, 8
// values a lane: 170 us for the 120 of the store and the load above).
constexpr int kRows = 4;

template <int V, int FMT>
__global__ __launch_bounds__(256) void cache_store_kernel(CacheArgs A) {
    const int l = threadIdx.x & 15;
    const uint32_t first = (blockIdx.x * 16 + (threadIdx.x >> 4)) * kRows;  // key row of the call
    const uint32_t per = uint32_t(A.H) * kK;
    const uint32_t i = first / per;
    if (i >= uint32_t(A.n)) return;
    const int row = A.rows ? A.rows[i] : int(i), slot = A.slots ? A.slots[i] : int(i);
    if (row < 0 || row >= A.B || slot < 0 || slot >= A.n_slots) return;
    const uint32_t hk = first - i * per;
    const bool more = 64 + 4 * l < V;
    const float* S = A.S + (size_t(row) * per + hk) * V + 4 * l;
    float4 x[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        x[r][0] = ldnt_f4(S + r * V);
        x[r][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (more)
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[r][1] = ldnt_f4(S + r * V + 64);
    const size_t at = size_t(slot) * per + hk;
    uint8_t* codes = static_cast<uint8_t*>(A.codes) + at * V + 4 * l;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float f[8] = {x[r][0].x, x[r][0].y, x[r][0].z, x[r][0].w, x[r][1].x, x[r][1].y, x[r][1].z, x[r][1].w};
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
        top = row_max16(top);
        const bool finite = top < 0x7f800000u;
        const uint32_t sb = finite ? scale_bits<FMT>(__uint_as_float(top)) : 0x7fc00000u;
        if (l == r) A.scales[at + r] = uint16_t(sb >> 16);
        const float s = __uint_as_float(sb), inv = 1.f / s;
        uint32_t c[2] = {0u, 0u};
        if constexpr (FMT == SKSSM_CACHE_I8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e / 4] |= (uint32_t(code_i8(f[e], s, inv)) & 0xffu) << (8 * (e % 4));
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int u = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e] * inv, f[4 * e + 1] * inv, 0, false);
                c[e] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e + 2] * inv, f[4 * e + 3] * inv, u, true));
            }
        }
        *reinterpret_cast<uint32_t*>(codes + r * V) = finite ? c[0] : 0u;
        if (more) *reinterpret_cast<uint32_t*>(codes + r * V + 64) = finite ? c[1] : 0u;
    }
}

template <int FMT>
__device__ __forceinline__ f32x4 values_of(uint32_t c, float s) {
    f32x4 x;
    if constexpr (FMT == SKSSM_CACHE_I8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = float(int8_t(c >> (8 * e)));
    } else {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(c), false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(c), true);
        x = f32x4{lo[0], lo[1], hi[0], hi[1]};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= s;
    return x;
}

template <int V, int FMT>
__global__ __launch_bounds__(256) void cache_load_kernel(CacheArgs A) {
    const int l = threadIdx.x & 15;
    const uint32_t first = (blockIdx.x * 16 + (threadIdx.x >> 4)) * kRows;
    const uint32_t per = uint32_t(A.H) * kK;
    const uint32_t i = first / per;
    if (i >= uint32_t(A.n)) return;
    const int row = A.rows ? A.rows[i] : int(i), slot = A.slots ? A.slots[i] : int(i);
    if (row < 0 || row >= A.B || slot >= A.n_slots) return;
    const uint32_t hk = first - i * per;
    const bool more = 64 + 4 * l < V;
    f32x4 x[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) x[r][0] = x[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (slot >= 0) {
        const size_t at = size_t(slot) * per + hk;
        const uint8_t* codes = static_cast<const uint8_t*>(A.codes) + at * V + 4 * l;
        const uint2 sc = *reinterpret_cast<const uint2*>(A.scales + at);  // four of them
        uint32_t c[kRows][2];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            c[r][0] = *reinterpret_cast<const uint32_t*>(codes + r * V);
            c[r][1] = more ? *reinterpret_cast<const uint32_t*>(codes + r * V + 64) : 0u;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const uint32_t b = r < 2 ? sc.x : sc.y;
            const float s = __uint_as_float(r % 2 ? b & 0xffff0000u : b << 16);
            x[r][0] = values_of<FMT>(c[r][0], s);
            x[r][1] = values_of<FMT>(c[r][1], s);
        }
    }
    float* S = A.out + (size_t(row) * per + hk) * V + 4 * l;
#pragma unroll
    for (int r = 0; r < kRows; ++r) __builtin_nontemporal_store(x[r][0], reinterpret_cast<f32x4*>(S + r * V));
    if (more)
#pragma unroll
        for (int r = 0; r < kRows; ++r) __builtin_nontemporal_store(x[r][1], reinterpret_cast<f32x4*>(S + r * V + 64));
}

namespace {

template <int V>
hipError_t launch_cache_v(bool store, int fmt, const CacheArgs& a, uint32_t blocks, hipStream_t s) {
    if (store) {
        if (fmt == SKSSM_CACHE_I8)
            hipLaunchKernelGGL((cache_store_kernel<V, SKSSM_CACHE_I8>), dim3(blocks), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((cache_store_kernel<V, SKSSM_CACHE_E4M3>), dim3(blocks), dim3(256), 0, s, a);
    } else {
        if (fmt == SKSSM_CACHE_I8)
            hipLaunchKernelGGL((cache_load_kernel<V, SKSSM_CACHE_I8>), dim3(blocks), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((cache_load_kernel<V, SKSSM_CACHE_E4M3>), dim3(blocks), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

sketchssm_status cache_call(bool store, const sketchssm_shape* shape, const CacheArgs& given, int format,
                            void* stream) {
    sketchssm_status st = check_shape(shape);
    if (st != SKSSM_OK) return st;
    CacheArgs A = given;
    if (format != SKSSM_CACHE_I8 && format != SKSSM_CACHE_E4M3) return SKSSM_EINVAL;
    if (A.n < 0 || A.n_slots < 0) return SKSSM_EINVAL;
    if (A.n > 0 && (!(store ? A.S : A.out) || (A.n_slots > 0 && (!A.codes || !A.scales)))) return SKSSM_EINVAL;
    const void* ptrs[] = {A.S, A.out, A.codes, A.scales, A.rows, A.slots};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return SKSSM_EALIGN;
    A.B = shape->B;
    A.H = shape->H;
    // a call's key rows, kRows of them to 16 lanes, are counted in 32 bits
    const double blocks = (double(A.n) * A.H * (kK / kRows) + 15) / 16;
    if (!launch_fits(blocks, 256)) return SKSSM_ESHAPE;
    if (A.n == 0) return SKSSM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipErrorInvalidValue;
    switch (shape->V) {
        case 64: e = launch_cache_v<64>(store, format, A, uint32_t(blocks), s); break;
        case 80: e = launch_cache_v<80>(store, format, A, uint32_t(blocks), s); break;
        case 96: e = launch_cache_v<96>(store, format, A, uint32_t(blocks), s); break;
        case 112: e = launch_cache_v<112>(store, format, A, uint32_t(blocks), s); break;
        case 128: e = launch_cache_v<128>(store, format, A, uint32_t(blocks), s); break;
    }
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}

}  // namespace

}  // namespace skssm

using namespace skssm;

extern "C" sketchssm_status sketchssm_cache_store(const sketchssm_shape* shape, const float* S, const int32_t* rows,
                                                  void* codes, uint16_t* scales, const int32_t* slots,
                                                  int32_t n_slots, int32_t n, int32_t format, void* stream) {
    CacheArgs A = {};
    A.S = S;
    A.rows = rows;
    A.codes = codes;
    A.scales = scales;
    A.slots = slots;
    A.n_slots = n_slots;
    A.n = n;
    return cache_call(true, shape, A, format, stream);
}

extern "C" sketchssm_status sketchssm_cache_load(const sketchssm_shape* shape, const void* codes,
                                                 const uint16_t* scales, const int32_t* slots, int32_t n_slots,
                                                 float* S, const int32_t* rows, int32_t n, int32_t format,
                                                 void* stream) {
    CacheArgs A = {};
    A.out = S;
    A.rows = rows;
    A.codes = const_cast<void*>(codes);
    A.scales = const_cast<uint16_t*>(scales);
    A.slots = slots;
    A.n_slots = n_slots;
    A.n = n;
    return cache_call(false, shape, A, format, stream);
}
