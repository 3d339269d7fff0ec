// ssd_step.hpp -- argument blocks and launchers of the operators around the
// scan (include/ssd_step.h). Host-side only types; pointers are device
// pointers.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "ssd_internal.hpp"

namespace ssd {

// Columns [n0, n1) of a product's output go to p [M, n1 - n0]. n0 is a
// multiple of 16, so a 16-column tile has one destination.
struct LinearSeg {
    void *p;
    int32_t n0, n1;
    int32_t bf16;
};

struct LinearArgs {
    int32_t M, N, K;
    int32_t lo, hi;           // columns of this launch (set by the launcher), lo % 16 == 0
    int32_t io_bf16;
    int32_t act;              // ssd_activation
    const void *x, *w;        // [M,K], [N,K]
    const float *bias;        // [N] or null
    const void *residual;     // [M,N] or null (one segment only)
    int32_t nseg;
    LinearSeg seg[3];
};

// Tiles of a product's launch at most: its threads (up to 768 a tile) are counted
// in 32 bits. A size whose 128 x 128 tiles are no more than this has a kernel.
constexpr int64_t kLinearMaxTiles = 1 << 22;

struct NormArgs {
    int64_t T;
    int32_t C, gs;            // channels of a row, channels of a group
    int32_t io_bf16, before;
    float eps;
    const void *y, *z;        // z may be null
    const float *w;
    void *out;
};

struct LogprobArgs {
    int64_t T;
    int32_t V, bf16, k;
    const void *logits;
    const int32_t *tokens;
    float *logprob, *entropy;  // entropy, rank may be null
    int32_t *rank;
    int32_t *top_ids;
    float *top_logprobs;
};

// A row of logits is cut into chunks, dealt to streams in turn; a wave runs whole streams.
constexpr int kLogprobStreams = 16, kLogprobChunk = 2048;

// Waves of a row (16 or 4; the bits are the same). 16 while all rows run at the same time
// (bf16 two to a compute unit: 512 rows of 50280 with top 8 in 18 against 24 us, 1024 in
// 33 against 33, 2048 in 62 against 52; fp32 one: 256 rows in 14 against 18 us, 512 in 28
// against 25), and in bf16 where every wave has four chunks or more and the launch's
// threads, 64 a wave, fit 32 bits (16 waves against 4, 600 to 4096 rows, no or 8
// alternatives, all or one token in 50 allowed: 0.66 to 1.01 of the time at 131072 to 262144
// columns, 0.74 to 1.04 at 65536 to 114688, 0.85 to 1.24 at 50280).
constexpr int logprob_waves(int64_t T, int32_t V, bool bf16) {
    if (T <= (bf16 ? 512 : 256))
        return 16;
    return bf16 && V >= 4 * kLogprobStreams * kLogprobChunk && T < (1 << 22) ? 16 : 4;
}

// A cache as the page kernels see it.
struct SlotMap {
    int32_t *pages;           // [slots, npp] or null
    int32_t npp, shift, num_pages, num_slots;
    int32_t Q;
    int32_t *buf_len;
    int64_t *boundary_pos;
    float *state;
    void *state_bf;
    void *buf_x, *buf_dt, *buf_B, *buf_C;
};

struct ReserveArgs {
    SlotMap c;
    int32_t n;
    const int32_t *slot_idx, *like_idx, *tokens;
    int32_t tokens_all;
    int32_t *granted;
};

// Bytes of one token's row in each buffer, and of one slot's state.
struct RowBytes {
    int32_t x, dt, bc;        // bc: B, and C alike
    int64_t state;            // fp32; the bf16 copy has half
};

struct CopyArgs {
    SlotMap dst, src;
    RowBytes r;
    int32_t n;
    const int32_t *dst_idx, *src_idx;
    int32_t *copied;
};

hipError_t launch_linear(const LinearArgs &a, hipStream_t stream);
hipError_t launch_gated_norm(const NormArgs &a, hipStream_t stream);
hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t stream);
hipError_t launch_pages_reserve(const ReserveArgs &a, hipStream_t stream);
hipError_t launch_pages_trim(const SlotMap &c, int32_t n, const int32_t *slot_idx,
                             hipStream_t stream);
hipError_t launch_cache_free(const SlotMap &c, const RowBytes &r, int32_t n,
                             const int32_t *slot_idx, hipStream_t stream);
hipError_t launch_cache_copy(const CopyArgs &a, hipStream_t stream);
// work: int32 [2 + num_pages] (move count, then from/to pairs)
hipError_t launch_pages_compact(const SlotMap &c, const RowBytes &r, int32_t *used, int32_t *work,
                                hipStream_t stream);

}  // namespace ssd
