// step_choice_check.cpp -- the rules by which the operators around the scan
// choose a kernel, on the CPU.
//
// Exit status 0 when every expectation holds.
#include <cstdio>

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

}  // namespace

int main() {
    // log probabilities: 16 waves for few rows, or long ones in bf16, and a launch's
    // threads below 2^32 at every accepted size
    using ssd::logprob_waves;
    EXPECT(logprob_waves(512, 100, true) == 16 && logprob_waves(513, 100, true) == 4);
    EXPECT(logprob_waves(256, 100, false) == 16 && logprob_waves(257, 1 << 20, false) == 4);
    EXPECT(logprob_waves(4096, 131072, true) == 16 && logprob_waves(4096, 131071, true) == 4);
    const int64_t rows[] = {1, 600, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 24) - 8};
    const int32_t cols[] = {1, 131071, 131072, 2147483647 - 65536};
    for (int64_t T : rows)
        for (int32_t V : cols)
            for (int bf = 0; bf < 2; ++bf)
                EXPECT(T * 64 * logprob_waves(T, V, bf != 0) < (int64_t)1 << 32);

    std::printf("%d failed expectations\n", g_fail);
    return g_fail != 0;
}
