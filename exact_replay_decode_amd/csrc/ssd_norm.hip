// ssd_norm.hip -- gated RMS norm of the scan's output, the step between the
// scan and the out-projection of the Mamba2 mixer.
//   norm_before_gate = 0:  v = y g(z), out = v r w,       r = rsqrt(mean(v^2) + eps)
//   norm_before_gate = 1:  v = y,      out = (v r w) g(z)
// over groups of gs channels, g(z) = z / (1 + exp(-z)); fp32, rounded once.
//
// A (row, group) is worked on by L lanes of a wave (groups up to 512 channels) or
// by a workgroup. Every lane owns NV pieces of eight channels (piece i of lane l starts at channel
// 8 (i lanes + l)), keeps them in registers between the sum and the scaling (y and
// z are read once, the output written once), and the sum of squares is taken in a
// fixed order: a lane's values in turn, a tree over the lanes, the waves' sums in
// order. The order depends on gs alone, so a row's bits do not depend on the
// number of rows.
// It is a stream: 16384 rows of 64 heads in 8 groups (403 MB) take 70-75 us, 5.4-5.8
// TB/s (a copy of 1 GiB moves 5.0).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_step.hpp"
#include "ssd_step_device.hpp"

namespace ssd {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// NT: past the caches (a large output would only push others out of them).
template <bool NT, class V>
__device__ __forceinline__ void put(V *p, const V &v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

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
    template <bool NT>
    __device__ static __forceinline__ void store(void *p, int64_t at, const float (&f)[8]) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = bf16_rne(f[2 * k]) | ((uint32_t)bf16_rne(f[2 * k + 1]) << 16);
        put<NT>(reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at), w);
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
    template <bool NT>
    __device__ static __forceinline__ void store(void *p, int64_t at, const float (&f)[8]) {
        f32x4 *q = reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at);
        put<NT>(q, (f32x4){f[0], f[1], f[2], f[3]});
        put<NT>(q + 1, (f32x4){f[4], f[5], f[6], f[7]});
    }
};

template <class IO>
__device__ __forceinline__ float silu(float z) {
    return z * (sizeof(typename IO::T) == 2 ? sigmoid_bf16(z) : sigmoid_f32(z));
}

// The lane's pieces of one group, lanes apart: the gated values and their sum of
// squares, then the scaled output.
template <class IO, int NV, bool NT>
struct Pieces {
    float v[NV][8], g[NV][8];
    __device__ __forceinline__ float load(const NormArgs &a, int64_t base, int lane, int lanes) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * lanes + lane);
            if (c < a.gs) {
                Eight<IO>::load(a.y, base + c, v[i]);
                if (a.z)
                    Eight<IO>::load(a.z, base + c, g[i]);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * lanes + lane);
            if (c < a.gs) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    g[i][j] = a.z ? silu<IO>(g[i][j]) : 1.0f;
                    if (!a.before)
                        v[i][j] *= g[i][j];
                    sum = fmaf(v[i][j], v[i][j], sum);
                }
            }
        }
        return sum;
    }
    __device__ __forceinline__ void store(const NormArgs &a, int64_t base, int c0, int lane,
                                          int lanes, float sum) {
        const float r = rsqrtf(sum / (float)a.gs + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * lanes + lane);
            if (c < a.gs) {
                float w[8], o[8];
                Eight<IoF32>::load(a.w, c0 + c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j] = v[i][j] * r * w[j];
                    if (a.before)
                        o[j] *= g[i][j];
                }
                Eight<IO>::template store<NT>(a.out, base + c, o);
            }
        }
    }
};

// L lanes a group, 64 / L groups a wave, four waves a workgroup.
template <class IO, int L, bool NT>
__global__ __launch_bounds__(256) void k_norm_lanes(NormArgs a) {
    const int groups = a.C / a.gs, lane = threadIdx.x % L;
    const int64_t u = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    if (u >= a.T * groups)
        return;
    const int c0 = (int)(u % groups) * a.gs;
    const int64_t base = u / groups * a.C + c0;
    Pieces<IO, 1, NT> p;
    float sum = p.load(a, base, lane, L);
    if constexpr (L == 64) {
        sum = wave_scan_inclusive(sum);   // the wave's sum in lane 63
        sum = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum), 63));
    } else {
#pragma unroll
        for (int o = 1; o < L; o <<= 1)
            sum += __shfl_xor(sum, o, L);
    }
    p.store(a, base, c0, lane, L, sum);
}

// A workgroup of W waves a group.
template <class IO, int W, int NV, bool NT>
__global__ __launch_bounds__(64 * W) void k_norm_waves(NormArgs a) {
    __shared__ float part[W];
    const int groups = a.C / a.gs;
    const int c0 = (int)(blockIdx.x % groups) * a.gs;
    const int64_t base = blockIdx.x / groups * (int64_t)a.C + c0;
    Pieces<IO, NV, NT> p;
    float sum = wave_scan_inclusive(p.load(a, base, threadIdx.x, 64 * W));
    if ((threadIdx.x & 63) == 63)
        part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w)
        sum += part[w];
    p.store(a, base, c0, threadIdx.x, 64 * W, sum);
}

// The output goes past the caches when y, z and it come near the 256 MB of the
// last one (403 MB: 83 -> 73 us, 201 MB: 40.5 -> 38.4; 25 MB the other way round:
// 7.2 -> 7.6).
bool past_caches(const NormArgs &a) {
    return 3 * a.T * a.C * (a.io_bf16 ? 2 : 4) > (int64_t)128 << 20;
}

template <class IO, int L>
hipError_t by_lanes(const NormArgs &a, hipStream_t stream) {
    const int64_t units = a.T * (a.C / a.gs);
    const dim3 grid((unsigned)((units + 256 / L - 1) / (256 / L)));
    if (past_caches(a))
        k_norm_lanes<IO, L, true><<<grid, dim3(256), 0, stream>>>(a);
    else
        k_norm_lanes<IO, L, false><<<grid, dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

template <class IO, int W, int NV>
hipError_t by_waves(const NormArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.T * (a.C / a.gs)));
    if (past_caches(a))
        k_norm_waves<IO, W, NV, true><<<grid, dim3(64 * W), 0, stream>>>(a);
    else
        k_norm_waves<IO, W, NV, false><<<grid, dim3(64 * W), 0, stream>>>(a);
    return hipGetLastError();
}

// Groups of up to 512 channels share waves (16384 rows of 64 groups of 64: 473 us
// with a wave each, 74 us eight to a wave). Above, one piece a lane and more waves
// beat more pieces in one wave (8192 rows of 2048 fp32: 29.8 against 33.9 us; 2048
// rows of 2048 bf16: 7.2 against 7.8) until the waves are four.
template <class IO>
hipError_t norm_impl(const NormArgs &a, hipStream_t stream) {
    const int gs = a.gs;
    if (gs <= 16) return by_lanes<IO, 2>(a, stream);
    if (gs <= 32) return by_lanes<IO, 4>(a, stream);
    if (gs <= 64) return by_lanes<IO, 8>(a, stream);
    if (gs <= 128) return by_lanes<IO, 16>(a, stream);
    if (gs <= 256) return by_lanes<IO, 32>(a, stream);
    if (gs <= 512) return by_lanes<IO, 64>(a, stream);
    if (gs <= 1024) return by_waves<IO, 2, 1>(a, stream);
    if (gs <= 2048) return by_waves<IO, 4, 1>(a, stream);
    if (gs <= 4096) return by_waves<IO, 4, 2>(a, stream);
    if (gs <= 8192) return by_waves<IO, 4, 4>(a, stream);
    if (gs <= 16384) return by_waves<IO, 16, 2>(a, stream);
    return by_waves<IO, 16, 4>(a, stream);   // gs <= 32768
}

}  // namespace

hipError_t launch_gated_norm(const NormArgs &a, hipStream_t stream) {
    return a.io_bf16 ? norm_impl<IoBF16>(a, stream) : norm_impl<IoF32>(a, stream);
}

}  // namespace ssd
