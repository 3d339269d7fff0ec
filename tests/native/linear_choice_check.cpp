// linear_choice_check.cpp -- the tile shapes that a product's launches take
// (csrc/ssd_linear_choice.hpp), on the CPU. Reads lines "bf16 M N K" (bf16 1 or
// 0; fp32 outputs) and prints "first second", second -1 for a single launch.
//
// Exit status 0 when every expectation holds.
#include <cstdio>
#include <iterator>

#include "ssd_linear_choice.hpp"

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

ssd::LinearArgs product(int bf16, long M, long N, long K) {
    alignas(16) static float out[4];
    ssd::LinearArgs a = {};
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.io_bf16 = bf16;
    a.nseg = 1;
    a.seg[0] = {out, 0, (int32_t)N, 0};
    return a;
}

int64_t tiles(const ssd::LinearShape &s, int64_t M, int64_t N) {
    return ((M + s.bm - 1) / s.bm) * ((N + s.bn - 1) / s.bn);
}

// A plan that a launch takes: whole columns, first part first, tiles counted in 32 bits.
void check(int bf16, const ssd::LinearArgs &a) {
    const ssd::LinearPlan p = ssd::linear_plan(a);
    const ssd::LinearShape *s = bf16 ? ssd::kLinearBF16 : ssd::kLinearF32;
    const int n = bf16 ? (int)std::size(ssd::kLinearBF16) : (int)std::size(ssd::kLinearF32);
    EXPECT(p.first >= 0 && p.first < n && p.second >= 0 && p.second < n);
    EXPECT(p.n1 > 0 && p.n1 <= a.N && (p.n1 == a.N || p.n1 % 16 == 0));
    EXPECT(tiles(s[p.first], a.M, p.n1) <= ssd::kLinearMaxTiles);
    EXPECT(p.n1 == a.N || tiles(s[p.second], a.M, a.N - p.n1) <= ssd::kLinearMaxTiles);
}

}  // namespace

int main() {
    const long sizes[] = {1, 15, 16, 17, 100, 256, 257, 1000, 4097, 10304, 50280, 65544, 262144,
                          536870912};
    for (int bf16 = 0; bf16 < 2; ++bf16)
        for (long M : sizes)
            for (long N : sizes)
                for (long K : {8L, 1000L, 4096L, 1048576L})
                    if (((M + 127) / 128) * ((N + 127) / 128) <= ssd::kLinearMaxTiles)
                        check(bf16, product(bf16, M, N, K));

    int bf16;
    long M, N, K;
    while (std::scanf("%d %ld %ld %ld", &bf16, &M, &N, &K) == 4) {
        const ssd::LinearArgs a = product(bf16, M, N, K);
        const ssd::LinearPlan p = ssd::linear_plan(a);
        std::printf("plan %d %d\n", p.first, p.n1 == a.N ? -1 : p.second);
    }
    std::printf("%d failed expectations\n", g_fail);
    return g_fail != 0;
}
