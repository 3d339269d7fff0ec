// ssd_step_device.hpp -- device helpers that the operators around the scan share.
#pragma once

#include "ssd_device.hpp"

namespace ssd {

// 1 / (1 + e^-u), 1 / inf = 0. For a bf16 result: v_exp_f32 of the rounded u log2 e,
// which is off by |u| 2^-24 of e, and v_rcp_f32; together at most (|u| + 6) 2^-24,
// below 2^-17 wherever e is finite, against the rounding's 2^-9.
__device__ __forceinline__ float sigmoid_bf16(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-u));
}
// For an fp32 result: what t = u log2 e loses by its rounding (known exactly, by fmaf)
// and by log2 e as stored comes back as a factor 1 + r ln 2, and the whole is within
// 7 2^-24 at any u: the factor and its product, v_exp_f32 (an ulp), 1 + e,
// v_rcp_f32 (an ulp). (Bounded: inf - inf would be a NaN; beyond 128 e is 0 or inf.)
__device__ __forceinline__ float sigmoid_f32(float u) {
    const float x = __builtin_amdgcn_fmed3f(-u, -1000.0f, 1000.0f);
    const float t = x * kLog2e;
    const float r = fmaf(x, 1.925963033500012e-8f, fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t) * fmaf(r, 0.6931471805599453f, 1.0f);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

}  // namespace ssd
