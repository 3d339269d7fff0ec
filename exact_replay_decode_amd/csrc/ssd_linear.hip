// ssd_linear.hip -- matrix product with bias, activation and residual in its
// epilogue: the mixer's projections (and any other linear layer of a step).
//   out[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
//
// Every output is one fp32 accumulation chain of matrix-core instructions over
// k ascending from zero: v_mfma_f32_16x16x32_bf16 (32 k a step) or
// v_mfma_f32_16x16x4_f32 (4 k a step), k past K filled with zeros on both
// sides. An MFMA result element depends on its own row, its own column and
// its accumulator only, so every kernel here that walks k in this order
// gives the same bits whatever its tile shape, and a row's bits do not
// depend on the number of rows. (The price is that k is never split over
// waves that would add partial sums.)
//
// The instruction's rows are output columns n and its columns are rows m of x:
// a lane then holds four consecutive n of one row, which it stores together.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssd_device.hpp"
#include "ssd_step.h"
#include "ssd_step.hpp"

namespace ssd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- epilogue ---------------------------------------------------------------

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
    case SSD_ACT_SILU:
        return __fdividef(v, 1.0f + __expf(-v));
    case SSD_ACT_GELU: {
        // 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), u = sqrt(2/pi)(v + 0.044715 v^3)
        const float u2 = 1.5957691216057308f * fmaf(0.044715f * v * v, v, v);
        return __fdividef(v, 1.0f + __expf(-u2));
    }
    case SSD_ACT_RELU2:
        return v <= 0.0f ? 0.0f : v * v;   // (a NaN stays one)
    default:
        return v;
    }
}

// Lane l of a 16 x 16 tile holds row m = l % 16, columns n = 4 (l / 16) + i:
// bias, activation, residual, one rounding, stored. n0, m0: the tile's first
// column (a multiple of 16) and row.
__device__ __forceinline__ void store_tile(const LinearArgs &a, int m0, int n0, const f32x4 &acc) {
    const int lane = threadIdx.x & 63;
    const int m = m0 + (lane & 15), n = n0 + 4 * (lane >> 4);
    if (m >= a.M || n >= a.N)
        return;
    LinearSeg s = a.seg[0];
    if (a.nseg > 1 && n0 >= s.n1)
        s = n0 >= a.seg[1].n1 ? a.seg[2] : a.seg[1];
    const int64_t at = (int64_t)m * (s.n1 - s.n0) + (n - s.n0);
    const int cnt = min(4, a.N - n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= cnt)
            break;
        float v = acc[i];
        if (a.bias)
            v += a.bias[n + i];
        v = activate(v, a.act);
        if (a.residual)
            v += a.io_bf16 ? IoBF16::ld(static_cast<const uint16_t *>(a.residual), at + i)
                           : static_cast<const float *>(a.residual)[at + i];
        if (s.bf16)
            static_cast<uint16_t *>(s.p)[at + i] = bf16_rne(v);
        else
            static_cast<float *>(s.p)[at + i] = v;
    }
}

// ---- one tile per wave ------------------------------------------------------

// A wave computes RT tiles of 16 rows x 16 columns, its operands loaded
// straight from memory.
template <int RT>
__global__ __launch_bounds__(256) void k_linear_bf16(LinearArgs a, int mtiles) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    const int n0 = (int)(t / mtiles) * 16, m0 = (int)(t % mtiles) * 16 * RT;
    if (n0 >= a.N)
        return;
    const int r = lane & 15, k0 = 8 * (lane >> 4);
    const uint16_t *w = static_cast<const uint16_t *>(a.w) +
                        (int64_t)min(n0 + r, a.N - 1) * a.K + k0;
    const uint16_t *x[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        x[i] = static_cast<const uint16_t *>(a.x) +
               (int64_t)min(m0 + 16 * i + r, a.M - 1) * a.K + k0;
    f32x4 acc[RT] = {};
    for (int k = 0; k < a.K; k += 32) {
        const bool in = k + k0 < a.K;
        const u32x4 zero = {0, 0, 0, 0};
        const u32x4 wv = in ? *reinterpret_cast<const u32x4 *>(w + k) : zero;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const u32x4 xv = in ? *reinterpret_cast<const u32x4 *>(x[i] + k) : zero;
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, wv), __builtin_bit_cast(bf16x8, xv), acc[i], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
        store_tile(a, m0 + 16 * i, n0, acc[i]);
}

template <int RT>
__global__ __launch_bounds__(256) void k_linear_f32(LinearArgs a, int mtiles) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    const int n0 = (int)(t / mtiles) * 16, m0 = (int)(t % mtiles) * 16 * RT;
    if (n0 >= a.N)
        return;
    const int r = lane & 15, k0 = lane >> 4;   // K is a multiple of 4: no tail
    const float *w = static_cast<const float *>(a.w) + (int64_t)min(n0 + r, a.N - 1) * a.K + k0;
    const float *x[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        x[i] = static_cast<const float *>(a.x) +
               (int64_t)min(m0 + 16 * i + r, a.M - 1) * a.K + k0;
    f32x4 acc[RT] = {};
    for (int k = 0; k < a.K; k += 4) {
        const float wv = w[k];
#pragma unroll
        for (int i = 0; i < RT; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv, x[i][k], acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
        store_tile(a, m0 + 16 * i, n0, acc[i]);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t stream) {
    const int ntiles = (a.N + 15) / 16;
    const int rt = a.M > 16 ? 4 : 1;
    const int mtiles = (a.M + 16 * rt - 1) / (16 * rt);
    const dim3 grid((unsigned)(((int64_t)ntiles * mtiles + 3) / 4)), block(256);
    if (a.io_bf16) {
        if (rt == 1)
            k_linear_bf16<1><<<grid, block, 0, stream>>>(a, mtiles);
        else
            k_linear_bf16<4><<<grid, block, 0, stream>>>(a, mtiles);
    } else {
        if (rt == 1)
            k_linear_f32<1><<<grid, block, 0, stream>>>(a, mtiles);
        else
            k_linear_f32<4><<<grid, block, 0, stream>>>(a, mtiles);
    }
    return hipGetLastError();
}

}  // namespace ssd
