// ssd_checks.hpp -- host-side argument checks shared by the C ABI layers
// (ssd_api.cpp, ssd_step_api.cpp): shapes, caches, alignment, status codes.
// All of them run before any HIP call.
#pragma once

#include "ssd_replay.h"

#include <stdint.h>

#include <vector>

#include "ssd_internal.hpp"

namespace ssd {
namespace checks {

inline bool pow2_in(int v, int lo, int hi) {
    if (v < lo || v > hi)
        return false;
    return (v & (v - 1)) == 0;
}

// bf16_state: the recurrent update also takes a bf16 state; everything that
// touches the replay cache requires fp32 ([RFC] section 4).
inline int check_shape(const ssd_shape *sh, Dims *d, bool bf16_state = false) {
    if (!sh)
        return SSD_ERR_NULL;
    if (sh->state_dtype != SSD_F32 && !(bf16_state && sh->state_dtype == SSD_BF16))
        return SSD_ERR_STATE_NOT_FP32;
    if ((sh->io_dtype != SSD_F32 && sh->io_dtype != SSD_BF16) ||
        (sh->dt_dtype != SSD_F32 && sh->dt_dtype != SSD_BF16))
        return SSD_ERR_DTYPE;
    if (sh->H <= 0 || sh->G <= 0 || sh->H % sh->G != 0)
        return SSD_ERR_SHAPE;
    if (!pow2_in(sh->chunk_size, 16, 256) || !pow2_in(sh->P, 16, 128) ||
        !pow2_in(sh->N, 16, 128) || sh->H > 65535)
        return SSD_ERR_UNSUPPORTED;
    d->H = sh->H;
    d->G = sh->G;
    d->P = sh->P;
    d->N = sh->N;
    d->Q = sh->chunk_size;
    d->io_bf16 = sh->io_dtype == SSD_BF16;
    d->dt_bf16 = sh->dt_dtype == SSD_BF16;
    d->softplus = sh->dt_softplus != 0;
    return SSD_OK;
}

// Arrays the kernels move in 16-byte pieces (NULL passes).
inline bool a16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <class... T>
bool all_a16(const T *...p) {
    return (a16(p) && ...);
}

// need_work = false: the call does not use the cache's work array (the
// decode entry point that brings its own)
inline int check_cache(const ssd_shape *sh, const ssd_replay_cache *c, bool need_work = true) {
    if (!c)
        return SSD_ERR_NULL;
    if (c->state_dtype != SSD_F32)
        return SSD_ERR_STATE_NOT_FP32;
    if (c->chunk_size != sh->chunk_size)
        return SSD_ERR_CHUNK_MISMATCH;
    if (!c->state || !c->state_bf || !c->buf_x || !c->buf_dt || !c->buf_B || !c->buf_len ||
        !c->boundary_pos || (need_work && !c->work))
        return SSD_ERR_NULL;
    if (c->num_slots <= 0)
        return SSD_ERR_SHAPE;
    if (c->buf_pages) {
        const int pt = c->page_tokens;
        if (pt < 16 || pt > c->chunk_size || (pt & (pt - 1)) != 0 || c->num_pages <= 0)
            return SSD_ERR_SHAPE;
    }
    if (!all_a16(c->state, c->state_bf, c->buf_x, c->buf_B, c->buf_C))
        return SSD_ERR_ALIGN;
    return SSD_OK;
}

// Buffer addressing of a checked cache.
inline ssd::BufMap buf_map(const ssd_replay_cache *c) {
    ssd::BufMap m = {};
    if (c->buf_pages) {
        m.pages = c->buf_pages;
        int sh = 0;
        while ((1 << sh) < c->page_tokens)
            ++sh;
        m.shift = sh;
        m.npp = c->chunk_size >> sh;
        m.num_pages = c->num_pages;
    }
    return m;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

inline size_t dtype_bytes(int dt) { return dt == SSD_BF16 ? 2 : 4; }

// Debug builds (SSD_DEBUG_CHECKS) also check that the slot_idx entries of a
// call that lie in [0, num_slots) are distinct: every kernel reads and writes
// a slot from one place per call, so a repeated slot is undefined behaviour
// the release build does not look for (it would need the device array on
// the host, a synchronising copy). Entries outside the range are the
// skipped positions some calls allow. Returns SSD_ERR_SHAPE on a repeat.
#ifdef SSD_DEBUG_CHECKS
inline int check_slots_distinct(const int32_t *slot_idx, int32_t n, int32_t num_slots) {
    if (!slot_idx || n <= 0 || num_slots <= 0)
        return SSD_OK;
    std::vector<int32_t> h((size_t)n);
    if (ssd::copy_to_host(h.data(), slot_idx, sizeof(int32_t) * (size_t)n) != hipSuccess)
        return SSD_ERR_HIP;
    std::vector<char> seen((size_t)num_slots, 0);
    for (int32_t v : h) {
        if (v < 0 || v >= num_slots)
            continue;
        if (seen[(size_t)v])
            return SSD_ERR_SHAPE;
        seen[(size_t)v] = 1;
    }
    return SSD_OK;
}
#else
inline int check_slots_distinct(const int32_t *, int32_t, int32_t) { return SSD_OK; }
#endif

}  // namespace checks
}  // namespace ssd
