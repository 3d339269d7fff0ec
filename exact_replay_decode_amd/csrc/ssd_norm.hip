// ssd_norm.hip -- gated RMS norm of the scan's output, the step between the
// scan and the out-projection of the Mamba2 mixer.
//   norm_before_gate = 0:  v = y g(z), out = v r w,       r = rsqrt(mean(v^2) + eps)
//   norm_before_gate = 1:  v = y,      out = (v r w) g(z)
// over groups of gs channels, g(z) = z / (1 + exp(-z)); fp32, rounded once.
//
// One workgroup of W waves per (row, group): every thread owns NV pieces of
// eight channels (piece i of thread t starts at channel 8 (i 64 W + t)), keeps
// them in registers between the sum and the scaling (y and z are read once,
// the output written once), and the sum of squares is taken in a fixed order:
// a thread's values in turn, a DPP tree over the wave, the waves' sums in
// order. The order depends on gs alone, so a row's bits do not depend on the
// number of rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_device.hpp"
#include "ssd_step.hpp"

namespace ssd {
namespace {

// Eight channels, loaded and stored as 16-byte pieces.
template <class IO>
struct Eight;
template <>
struct Eight<IoBF16> {
    __device__ static __forceinline__ void load(const void *p, int64_t at, float (&f)[8]) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ void store(void *p, int64_t at, const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = bf16_rne(f[2 * k]) | ((uint32_t)bf16_rne(f[2 * k + 1]) << 16);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Eight<IoF32> {
    __device__ static __forceinline__ void load(const void *p, int64_t at, float (&f)[8]) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 a = q[0], b = q[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ static __forceinline__ void store(void *p, int64_t at, const float (&f)[8]) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// SiLU with the hardware exp2 and reciprocal (a few ulps, far below the bf16
// rounding), as in the conv before the scan.
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

template <class IO, int W, int NV>
__global__ __launch_bounds__(64 * W) void k_gated_norm(NormArgs a) {
    const int groups = a.C / a.gs;
    const int64_t row = blockIdx.x / groups;
    const int c0 = (int)(blockIdx.x % groups) * a.gs;
    const int64_t base = row * a.C + c0;
    float v[NV][8], g[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * 64 * W + (int)threadIdx.x);
        if (c < a.gs) {
            Eight<IO>::load(a.y, base + c, v[i]);
            if (a.z)
                Eight<IO>::load(a.z, base + c, g[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * 64 * W + (int)threadIdx.x);
        if (c < a.gs) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[i][j] = a.z ? silu(g[i][j]) : 1.0f;
                if (!a.before)
                    v[i][j] *= g[i][j];
                sum = fmaf(v[i][j], v[i][j], sum);
            }
        }
    }
    sum = wave_scan_inclusive(sum);   // the wave's sum in lane 63
    if constexpr (W > 1) {
        __shared__ float part[W];
        if ((threadIdx.x & 63) == 63)
            part[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = part[0];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += part[w];
    } else {
        sum = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum), 63));
    }
    const float r = rsqrtf(sum / (float)a.gs + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * 64 * W + (int)threadIdx.x);
        if (c < a.gs) {
            float w[8], o[8];
            Eight<IoF32>::load(a.w, c0 + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = v[i][j] * r * w[j];
                if (a.before)
                    o[j] *= g[i][j];
            }
            Eight<IO>::store(a.out, base + c, o);
        }
    }
}

template <class IO>
hipError_t norm_impl(const NormArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.T * (a.C / a.gs)));
    if (a.gs <= 512)
        k_gated_norm<IO, 1, 1><<<grid, dim3(64), 0, stream>>>(a);
    else if (a.gs <= 1024)
        k_gated_norm<IO, 2, 1><<<grid, dim3(128), 0, stream>>>(a);
    else if (a.gs <= 2048)
        k_gated_norm<IO, 4, 1><<<grid, dim3(256), 0, stream>>>(a);
    else if (a.gs <= 4096)
        k_gated_norm<IO, 4, 2><<<grid, dim3(256), 0, stream>>>(a);
    else if (a.gs <= 8192)
        k_gated_norm<IO, 4, 4><<<grid, dim3(256), 0, stream>>>(a);
    else if (a.gs <= 16384)
        k_gated_norm<IO, 16, 2><<<grid, dim3(1024), 0, stream>>>(a);
    else
        k_gated_norm<IO, 16, 4><<<grid, dim3(1024), 0, stream>>>(a);   // gs <= 32768
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_norm(const NormArgs &a, hipStream_t stream) {
    return a.io_bf16 ? norm_impl<IoBF16>(a, stream) : norm_impl<IoF32>(a, stream);
}

}  // namespace ssd
