// ssd_step_api.cpp -- the extern "C" entry points declared in
// include/ssd_step.h: host-side argument checks (all of them before any HIP
// call, so a rejected call launches nothing) and the translation into
// kernel argument blocks.
#include "ssd_step.h"

#include <cmath>
#include <limits>

#include "ssd_checks.hpp"
#include "ssd_step.hpp"

namespace {

using namespace ssd::checks;
using ssd::Dims;

constexpr int64_t kMaxI32 = std::numeric_limits<int32_t>::max();
constexpr int32_t kMaxPages = 1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 34;   // of a norm
constexpr int32_t kMaxList = (1 << 24) - 8;       // rows or entries with 256 threads each

bool known_dtype(int dt) { return dt == SSD_F32 || dt == SSD_BF16; }
bool natural(const void *p, int dt) { return (uintptr_t)p % dtype_bytes(dt) == 0; }

// What both projections share; the segments are the caller's.
int check_linear(int64_t M, int64_t N, int64_t K, int32_t io) {
    if (!known_dtype(io))
        return SSD_ERR_DTYPE;
    if (M < 0 || N < 0 || K < 1)
        return SSD_ERR_SHAPE;
    // (a tile's rows lie within 32-bit byte offsets of its first one, and row
    // numbers up to a tile past the end are whole numbers of 32 bits)
    if (M > kMaxI32 - 65536 || N > kMaxI32 - 65536 || K > (1 << 20) ||
        K % (io == SSD_BF16 ? 8 : 4) != 0)
        return SSD_ERR_UNSUPPORTED;
    if (((M + 127) / 128) * ((N + 127) / 128) > ssd::kLinearMaxTiles)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// The cache fields that the page and slot calls need (check_cache without
// the work array), as the kernels take them.
int slot_map(const ssd_shape *sh, const ssd_replay_cache *c, bool paged, Dims *d, ssd::SlotMap *m) {
    int st = check_shape(sh, d);
    if (st != SSD_OK)
        return st;
    if ((st = check_cache(sh, c, false)) != SSD_OK)
        return st;
    if (paged && !c->buf_pages)
        return SSD_ERR_NULL;
    const ssd::BufMap b = buf_map(c);
    if (b.pages && (c->num_pages > kMaxPages || (int64_t)c->num_slots * b.npp > kMaxI32))
        return SSD_ERR_UNSUPPORTED;
    *m = {};
    m->pages = const_cast<int32_t *>(b.pages);
    m->npp = b.npp;
    m->shift = b.shift;
    m->num_pages = b.num_pages;
    m->num_slots = c->num_slots;
    m->Q = c->chunk_size;
    m->buf_len = c->buf_len;
    m->boundary_pos = c->boundary_pos;
    m->state = c->state;
    m->state_bf = c->state_bf;
    m->buf_x = c->buf_x;
    m->buf_dt = c->buf_dt;
    m->buf_B = c->buf_B;
    m->buf_C = c->buf_C;
    return SSD_OK;
}

int row_bytes(const ssd_shape *sh, const Dims &d, ssd::RowBytes *r) {
    const int64_t io = (int64_t)dtype_bytes(sh->io_dtype);
    const int64_t x = (int64_t)d.H * d.P * io, bc = (int64_t)d.G * d.N * io;
    if (x > kMaxI32 / 512 || bc > kMaxI32 / 512)
        return SSD_ERR_UNSUPPORTED;   // a page's bytes fit 32 bits with room
    r->x = (int32_t)x;
    r->bc = (int32_t)bc;
    r->dt = d.H * (int32_t)dtype_bytes(sh->dt_dtype);
    r->state = (int64_t)d.H * d.P * d.N * (int64_t)sizeof(float);
    return SSD_OK;
}

}  // namespace

extern "C" {

int ssd_linear(int64_t M, int64_t N, int64_t K, int32_t io, int32_t out_dtype, int32_t act,
               const void *x, const void *w, const float *bias, const void *residual, void *out,
               hipStream_t stream) {
    int st = check_linear(M, N, K, io);
    if (st != SSD_OK)
        return st;
    if (!known_dtype(out_dtype))
        return SSD_ERR_DTYPE;
    if (act < SSD_ACT_NONE || act > SSD_ACT_RELU2)
        return SSD_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return SSD_OK;
    if (!x || !w || !out)
        return SSD_ERR_NULL;
    if (!all_a16(x, w) || !natural(bias, SSD_F32) || !natural(residual, io) ||
        !natural(out, out_dtype))
        return SSD_ERR_ALIGN;
    // in place only where a thread reads what it then writes
    if (residual == out && io != out_dtype)
        return SSD_ERR_DTYPE;
    ssd::LinearArgs a = {};
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.io_bf16 = io == SSD_BF16;
    a.act = act;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.nseg = 1;
    a.seg[0] = {out, 0, (int32_t)N, out_dtype == SSD_BF16};
    return hip_status(ssd::launch_linear(a, stream));
}

int ssd_in_proj(const ssd_shape *sh, int64_t M, int64_t d_model, const void *u, const void *w,
                const float *bias, void *z, void *xBC, void *dt, hipStream_t stream) {
    Dims d;
    int st = check_shape(sh, &d);
    if (st != SSD_OK)
        return st;
    const int64_t hp = (int64_t)d.H * d.P, cd = hp + 2 * (int64_t)d.G * d.N, N = hp + cd + d.H;
    if ((st = check_linear(M, N, d_model, sh->io_dtype)) != SSD_OK)
        return st;
    if (M == 0)
        return SSD_OK;
    if (!u || !w || !z || !xBC || !dt)
        return SSD_ERR_NULL;
    if (!all_a16(u, w) || !natural(bias, SSD_F32) || !natural(z, sh->io_dtype) ||
        !natural(xBC, sh->io_dtype) || !natural(dt, sh->dt_dtype))
        return SSD_ERR_ALIGN;
    ssd::LinearArgs a = {};
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)d_model;
    a.io_bf16 = d.io_bf16;
    a.act = SSD_ACT_NONE;
    a.x = u;
    a.w = w;
    a.bias = bias;
    a.nseg = 3;
    a.seg[0] = {z, 0, (int32_t)hp, d.io_bf16};
    a.seg[1] = {xBC, (int32_t)hp, (int32_t)(hp + cd), d.io_bf16};
    a.seg[2] = {dt, (int32_t)(hp + cd), (int32_t)N, d.dt_bf16};
    return hip_status(ssd::launch_linear(a, stream));
}

int ssd_gated_norm(const ssd_shape *sh, int64_t T, int32_t groups, float eps,
                   int32_t norm_before_gate, const void *y, const void *z, const float *w,
                   void *out, hipStream_t stream) {
    Dims d;
    int st = check_shape(sh, &d);
    if (st != SSD_OK)
        return st;
    if (T < 0 || groups < 1 || d.H % groups != 0 || !(eps >= 0.0f) || std::isinf(eps))
        return SSD_ERR_SHAPE;
    const int64_t C = (int64_t)d.H * d.P, gs = C / groups;
    // (at most a thread for four channels, whose number is one of 32 bits)
    if (gs > 32768 || T > kMaxElems / C)
        return SSD_ERR_UNSUPPORTED;
    if (T == 0)
        return SSD_OK;
    if (!y || !w || !out)
        return SSD_ERR_NULL;
    if (!all_a16(y, z, (const void *)out) || !a16(w))
        return SSD_ERR_ALIGN;
    ssd::NormArgs a = {};
    a.T = T;
    a.C = (int32_t)C;
    a.gs = (int32_t)gs;
    a.io_bf16 = d.io_bf16;
    a.before = norm_before_gate != 0;
    a.eps = eps;
    a.y = y;
    a.z = z;
    a.w = w;
    a.out = out;
    return hip_status(ssd::launch_gated_norm(a, stream));
}

int ssd_token_logprobs(int64_t T, int64_t V, int32_t dtype, const void *logits,
                       const int32_t *tokens, int32_t top_k, float *logprob, float *entropy,
                       int32_t *rank, int32_t *top_ids, float *top_logprobs, hipStream_t stream) {
    if (!known_dtype(dtype))
        return SSD_ERR_DTYPE;
    if (T < 0 || V < 1 || top_k < 0 || top_k > V)
        return SSD_ERR_SHAPE;
    // (indices up to a chunk past V stay within 32 bits, as do 256 threads a row; a row
    // gets 1024 only where those do too)
    if (T > kMaxList || V > kMaxI32 - 65536 || top_k > 64)
        return SSD_ERR_UNSUPPORTED;
    if (T == 0)
        return SSD_OK;
    if (!logits || !tokens || !logprob || (top_k > 0 && (!top_ids || !top_logprobs)))
        return SSD_ERR_NULL;
    if (!natural(logits, dtype))
        return SSD_ERR_ALIGN;
    ssd::LogprobArgs a = {};
    a.T = T;
    a.V = (int32_t)V;
    a.bf16 = dtype == SSD_BF16;
    a.k = top_k;
    a.logits = logits;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.rank = rank;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    return hip_status(ssd::launch_logprobs(a, stream));
}

int ssd_replay_pages_reserve(const ssd_shape *sh, const ssd_replay_cache *cache, int32_t n,
                             const int32_t *slot_idx, const int32_t *like_idx,
                             const int32_t *tokens, int32_t tokens_all, int32_t *granted,
                             hipStream_t stream) {
    Dims d;
    ssd::ReserveArgs a = {};
    int st = slot_map(sh, cache, true, &d, &a.c);
    if (st != SSD_OK)
        return st;
    if (n < 0 || (!slot_idx && n > cache->num_slots))
        return SSD_ERR_SHAPE;
    if ((int64_t)n * a.c.npp > kMaxI32)
        return SSD_ERR_UNSUPPORTED;
    if (n == 0)
        return SSD_OK;
    if ((st = check_slots_distinct(slot_idx, n, cache->num_slots)) != SSD_OK)
        return st;
    a.n = n;
    a.slot_idx = slot_idx;
    a.like_idx = like_idx;
    a.tokens = tokens;
    a.tokens_all = tokens_all;
    a.granted = granted;
    return hip_status(ssd::launch_pages_reserve(a, stream));
}

int ssd_replay_pages_trim(const ssd_shape *sh, const ssd_replay_cache *cache, int32_t n,
                          const int32_t *slot_idx, hipStream_t stream) {
    Dims d;
    ssd::SlotMap m;
    int st = slot_map(sh, cache, true, &d, &m);
    if (st != SSD_OK)
        return st;
    if (n < 0 || (!slot_idx && n > cache->num_slots))
        return SSD_ERR_SHAPE;
    if ((int64_t)n * m.npp > kMaxI32)
        return SSD_ERR_UNSUPPORTED;
    if (n == 0)
        return SSD_OK;
    if ((st = check_slots_distinct(slot_idx, n, cache->num_slots)) != SSD_OK)
        return st;
    return hip_status(ssd::launch_pages_trim(m, n, slot_idx, stream));
}

int ssd_replay_cache_free(const ssd_shape *sh, const ssd_replay_cache *cache, int32_t n,
                          const int32_t *slot_idx, hipStream_t stream) {
    Dims d;
    ssd::SlotMap m;
    ssd::RowBytes r;
    int st = slot_map(sh, cache, false, &d, &m);
    if (st != SSD_OK)
        return st;
    if ((st = row_bytes(sh, d, &r)) != SSD_OK)
        return st;
    if (n < 0 || (!slot_idx && n > cache->num_slots))
        return SSD_ERR_SHAPE;
    if (n > kMaxList)
        return SSD_ERR_UNSUPPORTED;
    if (n == 0)
        return SSD_OK;
    if ((st = check_slots_distinct(slot_idx, n, cache->num_slots)) != SSD_OK)
        return st;
    return hip_status(ssd::launch_cache_free(m, r, n, slot_idx, stream));
}

int ssd_replay_cache_copy(const ssd_shape *sh, const ssd_replay_cache *dst,
                          const ssd_replay_cache *src, int32_t n, const int32_t *dst_idx,
                          const int32_t *src_idx, int32_t *copied, hipStream_t stream) {
    Dims d;
    ssd::CopyArgs a = {};
    int st = slot_map(sh, dst, false, &d, &a.dst);
    if (st != SSD_OK)
        return st;
    if ((st = slot_map(sh, src, false, &d, &a.src)) != SSD_OK)
        return st;
    if ((st = row_bytes(sh, d, &a.r)) != SSD_OK)
        return st;
    if (n < 0)
        return SSD_ERR_SHAPE;
    if (n > kMaxList)
        return SSD_ERR_UNSUPPORTED;
    if (n == 0)
        return SSD_OK;
    if (!dst_idx || !src_idx || (dst->buf_C && !src->buf_C))
        return SSD_ERR_NULL;
    if ((st = check_slots_distinct(dst_idx, n, dst->num_slots)) != SSD_OK)
        return st;
    a.n = n;
    a.dst_idx = dst_idx;
    a.src_idx = src_idx;
    a.copied = copied;
    return hip_status(ssd::launch_cache_copy(a, stream));
}

size_t ssd_replay_pages_compact_workspace_bytes(const ssd_replay_cache *cache) {
    if (!cache || !cache->buf_pages || cache->num_pages <= 0)
        return 0;
    return ((size_t)cache->num_pages + 2) * sizeof(int32_t);
}

int ssd_replay_pages_compact(const ssd_shape *sh, const ssd_replay_cache *cache, int32_t *used,
                             void *workspace, size_t workspace_bytes, hipStream_t stream) {
    Dims d;
    ssd::SlotMap m;
    ssd::RowBytes r;
    int st = slot_map(sh, cache, true, &d, &m);
    if (st != SSD_OK)
        return st;
    if ((st = row_bytes(sh, d, &r)) != SSD_OK)
        return st;
    if (!used)
        return SSD_ERR_NULL;
    if (!workspace || workspace_bytes < ssd_replay_pages_compact_workspace_bytes(cache))
        return SSD_ERR_WORKSPACE;
    if ((uintptr_t)workspace % sizeof(int32_t) != 0)
        return SSD_ERR_ALIGN;
    return hip_status(ssd::launch_pages_compact(m, r, used, (int32_t *)workspace, stream));
}

}  // extern "C"
