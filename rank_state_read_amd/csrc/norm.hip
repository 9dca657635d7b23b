// The gated norm behind a layer's output on gfx950.  Per token, over groups of
// `heads` consecutive heads (width = heads V values):
//   x   = y + D_h skip                              (skip optional)
//   out = norm(x silu(z)) w | norm(x) w silu(z) | norm(x) w sigmoid(z) | norm(x) w
//   norm(x) = x / sqrt(mean(x^2) + eps)
// The gate before the norm over a group of heads is a Mamba-2 layer's form, a
// norm per head and then the gate that of the delta-rule layers.
//
// One pass: a group's values stay in the registers of one team of lanes between
// the sum of squares and the output, so every input is read once and every
// output written once; the sum and the scaling are fp32, with one rounding at
// the store.  A lane holds 8 consecutive values per step (V is a multiple of 16,
// so 8 values never cross a head).  Teams: one 16-lane DPP row for the widths of
// one head, a wave, a quarter block or a block for wider groups.
//
// Bound by memory: 16001 tokens of 32 heads of 128, gate behind the norm, 91 us, 5.8
// TB/s (a plain stream that writes as much as it reads: 5.9 to 6.2); 256 tokens
// of 128 heads of 80 in groups of 16 heads 7.9 us, mostly latency.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "sketchssm_internal.h"

namespace skssm {

struct NormArgs {
    const float* y;
    const void* skip;
    const float* D;
    const void* z;
    const float* w;
    void* out;
    uint32_t groups;  // tokens * H / heads
    int per_row;      // groups per token: H / heads
    int heads, V, width;
    int w_width;      // weight values: V (every head the same) or H V
    int gate;
    float eps;
};

template <typename QT>
__device__ __forceinline__ void store8(void* base, size_t e, const float* f) {
    if constexpr (std::is_same<QT, Bf16Tag>::value) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        store8f(static_cast<float*>(base) + e, f);
    }
}

// Sum over a team of LANES lanes; every lane gets the same bits.
template <int LANES>
__device__ __forceinline__ float team_sum(float x, float* red) {
    x = row_sum16(x);
    if constexpr (LANES > 16) {
        x += __shfl_xor(x, 16, 64);
        x += __shfl_xor(x, 32, 64);
    }
    if constexpr (LANES > 64) {  // the team is the block
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int i = 1; i < LANES / 64; ++i) x += red[i];
    }
    return x;
}

template <int LANES, int STEPS, typename QT>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void gated_norm_kernel(NormArgs A) {
    constexpr int NT = LANES > 256 ? LANES : 256;
    constexpr int TEAMS = NT / LANES;
    __shared__ float red[16];
    const int lane = threadIdx.x % LANES;
    const uint32_t group = blockIdx.x * TEAMS + threadIdx.x / LANES;
    if (LANES <= 64 && group >= A.groups) return;
    const uint32_t row = group / uint32_t(A.per_row);
    const int g = int(group - row * uint32_t(A.per_row));
    const size_t base = size_t(group) * A.width;

    float x[STEPS][8], gt[STEPS][8];
    float ss = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int c = 8 * (lane + LANES * s);
        if (c < A.width) {
            load8f(A.y + base + c, x[s]);
            if (A.z) Vec8<QT>::unpack(Vec8<QT>::load(A.z, base + c), gt[s]);
            if (A.skip) {
                float f[8];
                Vec8<QT>::unpack(Vec8<QT>::load(A.skip, base + c), f);
                const float d = A.D[g * A.heads + c / A.V];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[s][i] = fmaf(d, f[i], x[s][i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[s][i] = gt[s][i] = 0.f;
        }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (A.gate != SKSSM_GATE_NONE) {
                const float sg = 1.f / (1.f + expf(-gt[s][i]));
                gt[s][i] = A.gate == SKSSM_GATE_SIGMOID ? sg : gt[s][i] * sg;
                if (A.gate == SKSSM_GATE_SILU_FIRST) x[s][i] *= gt[s][i];
            }
            ss = fmaf(x[s][i], x[s][i], ss);
        }
    ss = team_sum<LANES>(ss, red);
    const float inv = 1.f / sqrtf(ss / float(A.width) + A.eps);
    const int w0 = A.w_width == A.V ? 0 : g * A.width;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int c = 8 * (lane + LANES * s);
        if (c < A.width) {
            float f[8];
            load8f(A.w + (A.w_width == A.V ? c % A.V : w0 + c), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] *= x[s][i] * inv;
                if (A.gate == SKSSM_GATE_SILU || A.gate == SKSSM_GATE_SIGMOID) f[i] *= gt[s][i];
            }
            store8<QT>(A.out, base + c, f);
        }
    }
}

template <int LANES, int STEPS, typename QT>
static hipError_t launch_norm_t(const NormArgs& a, hipStream_t s) {
    constexpr int NT = LANES > 256 ? LANES : 256;
    constexpr uint32_t teams = NT / LANES;
    if (!launch_fits((a.groups + teams - 1) / teams, NT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((gated_norm_kernel<LANES, STEPS, QT>), dim3((a.groups + teams - 1) / teams), dim3(NT), 0, s, a);
    return hipGetLastError();
}

// The team and its steps: few idle lanes, and few barriers per value.  us of the team
// chosen and of its neighbours, bf16, 64 tokens and then 2^23 values:
//   width  128: 16 lanes  3.0, 13.8; 64 lanes 3.4, 33.5
//   width  256: 16 x 2    4.0, 15.6; 64 lanes 3.1, 19.4: by the number of groups
//   width  512: 64 lanes  3.1, 14.0; 256 lanes 3.3, 27.0; 16 x 4 6.3, 19.0
//   width  640: 64 x 2    4.3, 19.4; 256 lanes 4.2, 24.7
//   width 2048: 256 lanes 3.1, 14.0; 64 x 4 6.4, 19.3; 1024 lanes 3.8, 28.1
//   width 2560: 256 x 2   4.2, 17.3; 1024 lanes 4.1, 24.3 (4096: 4.2, 16.2 and 3.9, 17.9)
//   width 8192: 1024 lanes 4.2, 14.1; 256 x 4 6.5, 19.0
//   width 10240: 1024 x 2 6.4, 20.0; 1024 x 4 9.0, 36.0
template <typename QT>
static hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.width <= 128) return launch_norm_t<16, 1, QT>(a, s);
    if (a.width <= 256 && a.groups > 8192) return launch_norm_t<16, 2, QT>(a, s);
    if (a.width <= 512) return launch_norm_t<64, 1, QT>(a, s);
    if (a.width <= 1024) return launch_norm_t<64, 2, QT>(a, s);
    if (a.width <= 2048) return launch_norm_t<256, 1, QT>(a, s);
    if (a.width <= 4096) return launch_norm_t<256, 2, QT>(a, s);
    if (a.width <= 8192) return launch_norm_t<1024, 1, QT>(a, s);
    if (a.width <= 16384) return launch_norm_t<1024, 2, QT>(a, s);
    return launch_norm_t<1024, 4, QT>(a, s);
}
static_assert(1024 * 4 * 8 >= kMaxHeads * 128, "the widest group");

}  // namespace skssm

using namespace skssm;

extern "C" sketchssm_status sketchssm_gated_norm(const sketchssm_shape* shape, const float* y, const void* skip,
                                                 const float* D, const void* z, const float* weight,
                                                 int32_t weight_heads, int32_t norm_heads, int32_t gate, float eps,
                                                 int32_t n_tokens, void* out, void* stream) {
    const sketchssm_status st = check_shape(shape);
    if (st != SKSSM_OK) return st;
    if (gate < SKSSM_GATE_NONE || gate > SKSSM_GATE_SIGMOID) return SKSSM_EINVAL;
    if (n_tokens < 0 || !(eps >= 0.f)) return SKSSM_EINVAL;
    if (norm_heads < 1 || norm_heads > shape->H || shape->H % norm_heads != 0) return SKSSM_ESHAPE;
    if (weight_heads != 1 && weight_heads != shape->H) return SKSSM_ESHAPE;
    if (!weight || (skip != nullptr) != (D != nullptr)) return SKSSM_EINVAL;
    if (n_tokens > 0 && (!y || !out || (gate != SKSSM_GATE_NONE) != (z != nullptr))) return SKSSM_EINVAL;
    const void* ptrs[] = {y, skip, D, z, weight, out};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return SKSSM_EALIGN;
    const double groups = double(n_tokens) * (shape->H / norm_heads);
    if (groups >= 2147483648.0) return SKSSM_ESHAPE;
    if (n_tokens == 0) return SKSSM_OK;
    NormArgs A;
    A.y = y;
    A.skip = skip;
    A.D = D;
    A.z = z;
    A.w = weight;
    A.out = out;
    A.groups = uint32_t(groups);
    A.per_row = shape->H / norm_heads;
    A.heads = norm_heads;
    A.V = shape->V;
    A.width = norm_heads * shape->V;
    A.w_width = weight_heads * shape->V;
    A.gate = gate;
    A.eps = eps;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = shape->qkv == SKSSM_BF16 ? launch_norm<Bf16Tag>(A, s) : launch_norm<F32Tag>(A, s);
    if (e == hipErrorInvalidConfiguration) return SKSSM_ESHAPE;  // more threads than a launch takes
    return e == hipSuccess ? SKSSM_OK : SKSSM_ELAUNCH;
}
