// step_host_check.cpp -- the C ABI layer of the operators around the scan
// (csrc/ssd_step_api.cpp) on the CPU, built with AddressSanitizer and
// UndefinedBehaviorSanitizer and with the debug-build checks, against
// stand-ins for the kernel launchers: what an accepted call hands over, the
// limits on either side, and repeated slots.
//
// Exit status 0 when every expectation holds; a sanitizer report aborts.
#include <cstdio>
#include <cstring>

#include "ssd_step.h"
#include "ssd_step.hpp"

namespace {

int g_fail = 0;

#define EXPECT(cond)                                                           \
    do {                                                                       \
        if (!(cond)) {                                                         \
            std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__,  \
                         __LINE__, #cond);                                     \
            ++g_fail;                                                          \
        }                                                                      \
    } while (0)

int g_launches = 0;
ssd::LinearArgs g_linear;
ssd::NormArgs g_norm;
ssd::LogprobArgs g_logprobs;
ssd::ReserveArgs g_reserve;
ssd::CopyArgs g_copy;
ssd::SlotMap g_map;
ssd::RowBytes g_rows;

template <class T>
hipError_t seen(T &to, const T &a) {
    to = a;
    ++g_launches;
    return hipSuccess;
}
// launches since the last call
int launched() {
    const int n = g_launches;
    g_launches = 0;
    return n;
}

}  // namespace

namespace ssd {
hipError_t launch_linear(const LinearArgs &a, hipStream_t) { return seen(g_linear, a); }
hipError_t launch_gated_norm(const NormArgs &a, hipStream_t) { return seen(g_norm, a); }
hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t) { return seen(g_logprobs, a); }
hipError_t launch_pages_reserve(const ReserveArgs &a, hipStream_t) { return seen(g_reserve, a); }
hipError_t launch_pages_trim(const SlotMap &c, int32_t, const int32_t *, hipStream_t) {
    return seen(g_map, c);
}
hipError_t launch_cache_free(const SlotMap &c, const RowBytes &r, int32_t, const int32_t *,
                             hipStream_t) {
    g_rows = r;
    return seen(g_map, c);
}
hipError_t launch_cache_copy(const CopyArgs &a, hipStream_t) { return seen(g_copy, a); }
hipError_t launch_pages_compact(const SlotMap &c, const RowBytes &r, int32_t *, int32_t *,
                                hipStream_t) {
    g_rows = r;
    return seen(g_map, c);
}
hipError_t copy_to_host(void *dst, const void *src, size_t bytes) {
    std::memcpy(dst, src, bytes);
    return hipSuccess;
}
}  // namespace ssd

int main() {
    alignas(16) static char mem[256];
    void *const A = mem;
    float *const F = reinterpret_cast<float *>(mem);
    int32_t *const I = reinterpret_cast<int32_t *>(mem);

    // products: the arguments, in-place residuals, the largest sizes
    EXPECT(ssd_linear(3, 5, 16, SSD_BF16, SSD_F32, SSD_ACT_GELU, A, A, F, nullptr, A,
                      nullptr) == SSD_OK && launched() == 1);
    EXPECT(g_linear.M == 3 && g_linear.N == 5 && g_linear.K == 16 && g_linear.io_bf16 == 1 &&
           g_linear.act == SSD_ACT_GELU && g_linear.nseg == 1 && g_linear.seg[0].n0 == 0 &&
           g_linear.seg[0].n1 == 5 && g_linear.seg[0].bf16 == 0 && !g_linear.residual);
    EXPECT(ssd_linear(1, 536870912, 8, SSD_BF16, SSD_BF16, 0, A, A, nullptr, A, A, nullptr) ==
           SSD_OK && launched() == 1);
    EXPECT(ssd_linear(1, 536870913, 8, SSD_BF16, SSD_BF16, 0, A, A, nullptr, A, A, nullptr) ==
           SSD_ERR_UNSUPPORTED);
    EXPECT(ssd_linear(INT64_MAX, INT64_MAX, 8, SSD_BF16, SSD_BF16, 0, A, A, nullptr, A, A,
                      nullptr) == SSD_ERR_UNSUPPORTED);
    EXPECT(ssd_linear(1, 1, INT64_MAX, SSD_F32, SSD_F32, 0, A, A, nullptr, A, A, nullptr) ==
           SSD_ERR_UNSUPPORTED);
    EXPECT(launched() == 0);

    // the in-projection's three parts, each of its type, the largest head count
    ssd_shape sh = {4, 2, 16, 16, 64, SSD_BF16, SSD_F32, SSD_F32, 1};
    EXPECT(ssd_in_proj(&sh, 7, 24, A, A, nullptr, A, A, A, nullptr) == SSD_OK && launched() == 1);
    EXPECT(g_linear.N == 64 + 128 + 4 && g_linear.nseg == 3 && g_linear.seg[0].n1 == 64 &&
           g_linear.seg[1].n0 == 64 && g_linear.seg[1].n1 == 192 && g_linear.seg[2].n0 == 192 &&
           g_linear.seg[2].n1 == 196 && g_linear.seg[1].bf16 == 1 && g_linear.seg[2].bf16 == 0);
    ssd_shape wide = {65535, 65535, 128, 128, 64, SSD_BF16, SSD_BF16, SSD_F32, 1};
    EXPECT(ssd_in_proj(&wide, 1, 8, A, A, nullptr, A, A, A, nullptr) == SSD_OK &&
           launched() == 1 && g_linear.N == 65535 * (4 * 128 + 1));

    // the norm's groups and largest sizes
    EXPECT(ssd_gated_norm(&sh, 3, 4, 0.0f, 2, A, nullptr, F, A, nullptr) == SSD_OK &&
           launched() == 1 && g_norm.C == 64 && g_norm.gs == 16 && g_norm.before == 1 &&
           !g_norm.z);
    EXPECT(ssd_gated_norm(&sh, 1 << 28, 1, 0.0f, 0, A, A, F, A, nullptr) == SSD_OK &&
           launched() == 1);
    EXPECT(ssd_gated_norm(&sh, (1 << 28) + 1, 1, 0.0f, 0, A, A, F, A, nullptr) ==
           SSD_ERR_UNSUPPORTED);
    EXPECT(ssd_gated_norm(&sh, INT64_MAX, 1, 0.0f, 0, A, A, F, A, nullptr) ==
           SSD_ERR_UNSUPPORTED);

    EXPECT(ssd_token_logprobs(5, 50, SSD_BF16, A, I, 20, F, nullptr, nullptr, I, F, nullptr) ==
           SSD_OK && launched() == 1 && g_logprobs.V == 50 && g_logprobs.k == 20 &&
           !g_logprobs.rank && !g_logprobs.entropy);
    EXPECT(ssd_token_logprobs(INT64_MAX, 50, SSD_F32, A, I, 0, F, F, I, nullptr, nullptr,
                              nullptr) == SSD_ERR_UNSUPPORTED);

    // caches: the map, the bytes of a row, lists
    ssd_replay_cache c = {};
    c.state = F;
    c.state_bf = c.buf_x = c.buf_dt = c.buf_B = A;
    c.buf_len = I;
    c.boundary_pos = reinterpret_cast<int64_t *>(mem);
    c.num_slots = 3;
    c.chunk_size = 64;
    c.state_dtype = SSD_F32;
    c.buf_pages = I;
    c.page_tokens = 32;
    c.num_pages = 9;
    int32_t once[] = {0, -1, 2, -1, 7}, twice[] = {1, 0, 1};
    EXPECT(ssd_replay_pages_reserve(&sh, &c, 5, once, nullptr, nullptr, -3, nullptr, nullptr) ==
           SSD_OK && launched() == 1);
    EXPECT(g_reserve.n == 5 && g_reserve.tokens_all == -3 && g_reserve.c.npp == 2 &&
           g_reserve.c.shift == 5 && g_reserve.c.num_pages == 9 && g_reserve.c.Q == 64);
    EXPECT(ssd_replay_pages_trim(&sh, &c, 3, nullptr, nullptr) == SSD_OK && launched() == 1);
    EXPECT(ssd_replay_cache_free(&sh, &c, 5, once, nullptr) == SSD_OK && launched() == 1);
    EXPECT(g_rows.x == 128 && g_rows.bc == 64 && g_rows.dt == 16 && g_rows.state == 4096);
    EXPECT(ssd_replay_pages_compact(&sh, &c, I, A, 44, nullptr) == SSD_OK && launched() == 1);
    EXPECT(ssd_replay_pages_compact_workspace_bytes(&c) == 44);
    EXPECT(ssd_replay_pages_compact(&sh, &c, I, A, 43, nullptr) == SSD_ERR_WORKSPACE);
    ssd_replay_cache flat = c;
    flat.buf_pages = nullptr;
    EXPECT(ssd_replay_cache_copy(&sh, &flat, &c, 2, once, twice, I, nullptr) == SSD_OK &&
           launched() == 1 && !g_copy.dst.pages && g_copy.src.pages && g_copy.n == 2);
    // a slot twice: every list that is written through (sources may repeat)
    EXPECT(ssd_replay_pages_reserve(&sh, &c, 3, twice, nullptr, nullptr, 1, I, nullptr) ==
           SSD_ERR_SHAPE);
    EXPECT(ssd_replay_pages_trim(&sh, &c, 3, twice, nullptr) == SSD_ERR_SHAPE);
    EXPECT(ssd_replay_cache_free(&sh, &c, 3, twice, nullptr) == SSD_ERR_SHAPE);
    EXPECT(ssd_replay_cache_copy(&sh, &c, &c, 3, twice, once, I, nullptr) == SSD_ERR_SHAPE);
    EXPECT(ssd_replay_cache_copy(&sh, &c, &flat, 3, once, twice, I, nullptr) == SSD_OK &&
           launched() == 1);
    // buffered C that the source lacks
    flat.buf_C = A;
    EXPECT(ssd_replay_cache_copy(&sh, &flat, &c, 2, once, twice, I, nullptr) == SSD_ERR_NULL);
    // rows too wide for a 32-bit page
    ssd_shape huge = wide;
    huge.chunk_size = 64;
    EXPECT(ssd_replay_cache_free(&huge, &c, 1, nullptr, nullptr) == SSD_ERR_UNSUPPORTED);
    c.num_pages = (1 << 20) + 1;
    EXPECT(ssd_replay_pages_trim(&sh, &c, 3, nullptr, nullptr) == SSD_ERR_UNSUPPORTED);
    EXPECT(launched() == 0);

    std::printf("%d failed expectations\n", g_fail);
    return g_fail != 0;
}
