// ssd_linear_choice.hpp -- which tile shapes a product's launches take
// (ssd_linear.hip has the kernels, in the tables' order). Host only.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "ssd_step.hpp"

namespace ssd {

// All shapes give the same bits; the choice is for time alone. A shape's time
// is modelled as that of its rounds of tiles over the 256 compute units. A
// round takes fix (us) + K ns with as many workgroups on each compute unit as
// fit; a single round that is not full fix1 and ns1 with one on each, in between by
// the line through the two. In bf16 that counts no further down than the time of
// the arrays at 5.2 TB/s (but a fiftieth of it, for shapes that are all bound by
// them). In a single launch of one round, where nothing runs beside it, the epilogue
// counts when output rows do not start on 16 bytes (734 x 7643 x 320 against 7648
// columns: 14.9 against 12.0 us in 256 x 128 tiles, 11.7 against 10.3 in 128 x 128; fp32
// does not notice). Of 200 drawn sizes with odd columns that changes the choice for 20,
// at 0.81 to 1.05 of the time without it, 0.94 in the mean.
// The figures are fitted to 466 sizes in bf16 (1 to 8192 rows, 256 to 50280
// columns, K 256 to 4096) and 400 in fp32 (half the K), with weights that come from
// memory, as a model's do. On those above 6 us the shape that they pick is 1.2 % slower
// than the best one in the mean in bf16 (7 % at the 95th percentile), 1.2 % (6 %) in
// fp32. (profiles/linear_shapes_sweep.csv has every shape's time at each of them.)
struct LinearShape {
    int bm, bn;
    int fit;                 // workgroups that run on a compute unit at a time
    float fix1, ns1, fix, ns;
};
constexpr int kLinearUnits = 256;

struct LinearProblem {
    int64_t M, N, K;
    bool bf16, ragged;       // inputs; output rows that are not 16-byte aligned
};

inline float linear_time(const LinearShape &s, const LinearProblem &p) {
    const int64_t M = p.M, N = p.N, K = p.K;
    const int64_t tiles = ((M + s.bm - 1) / s.bm) * ((N + s.bn - 1) / s.bn);
    if (tiles > kLinearMaxTiles)
        return INFINITY;
    const int64_t round = kLinearUnits * s.fit;
    const float one = s.fix1 + (float)K * s.ns1 * 1e-3f, full = s.fix + (float)K * s.ns * 1e-3f;
    float t = one;
    if (tiles > round)
        t = (float)((tiles + round - 1) / round) * full;
    else if (s.fit > 1)
        t += (full - one) * (float)((tiles - 1) / kLinearUnits) / (float)(s.fit - 1);
    if (tiles <= round && p.ragged)
        t += 6e-5f * (float)(s.bm * s.bn);
    const float bytes = 2.0f * ((float)N * (float)K + (float)M * (float)K + (float)M * (float)N);
    return p.bf16 ? std::max(t, bytes / 5.2e6f) + 0.02f * t : t;
}

template <int S>
int best_linear_shape(const LinearShape (&s)[S], const LinearProblem &p, float *time) {
    int best = 0;
    *time = linear_time(s[0], p);
    for (int i = 1; i < S; ++i) {
        const float t = linear_time(s[i], p);
        if (t < *time) {
            *time = t;
            best = i;
        }
    }
    return best;
}

constexpr LinearShape kLinearBF16[] = {
    {16, 16, 3, 0.39f, 1.39f, 0.75f, 2.52f},    {16, 16, 2, 0.56f, 1.06f, 1.57f, 2.53f},
    {16, 32, 2, 0.60f, 1.33f, 1.66f, 3.36f},    {32, 32, 2, 0.58f, 2.61f, 1.14f, 3.59f},
    {64, 32, 1, 0.91f, 2.38f, 1.56f, 2.61f},    {64, 64, 2, 0.90f, 4.80f, 1.62f, 6.69f},
    {64, 64, 1, 1.32f, 3.94f, 2.37f, 3.69f},    {128, 64, 2, 0.89f, 6.66f, 2.05f, 10.17f},
    {128, 64, 1, 1.89f, 5.50f, 2.68f, 5.46f},   {128, 128, 2, 1.27f, 13.25f, 4.04f, 15.88f},
    {128, 128, 1, 2.74f, 8.41f, 3.57f, 9.25f},  {256, 128, 1, 5.34f, 11.83f, 6.43f, 12.30f},
    {256, 256, 1, 9.16f, 23.49f, 10.36f, 22.82f},
};

// fp32 is bound by the matrix instructions from 32 x 32 on (131 of 157 TFLOP/s
// peak in full rounds of 128 x 128): the shapes differ in how evenly the tiles divide.
constexpr LinearShape kLinearF32[] = {
    {16, 16, 3, 0.00f, 4.46f, 0.57f, 5.97f},    {32, 32, 2, 0.00f, 4.95f, 2.29f, 7.69f},
    {32, 32, 3, 0.00f, 6.46f, 1.57f, 11.64f},   {32, 64, 3, 0.00f, 11.44f, 2.36f, 20.28f},
    {64, 32, 3, 0.00f, 10.78f, 2.25f, 21.16f},  {64, 32, 1, 0.00f, 8.73f, 1.89f, 8.84f},
    {64, 64, 2, 0.00f, 20.37f, 2.00f, 30.86f},  {96, 64, 2, 0.06f, 26.22f, 2.13f, 43.62f},
    {128, 64, 3, 0.82f, 35.11f, 5.34f, 77.40f}, {128, 128, 2, 2.31f, 64.76f, 5.29f, 113.08f},
};

// Columns [0, n1) in shape `first`, the rest, if any, in shape `second`.
struct LinearPlan {
    int first, second;
    int64_t n1;
};

// One launch over all columns, or one over the columns of a shape's whole rounds
// and one, in a smaller shape, over the rest, where the last round would leave
// most of the device idle (8192 x 10304 x 2048 in 256 x 256 tiles: 5 rounds and 32
// tiles, 386 us; with the last 64 columns on their own 305; fp32 2048 x 10304 x 2048 715
// and 637). What the second launch has to save, in us: of the sizes of the fit 39 take
// two in bf16, at 0.94 of the one launch's time in the mean (0.77-1.12), 10 in fp32, at
// 0.96 (0.87-1.09). With 2 us in fp32 it was 77, at 1.04.
constexpr float kSecondLaunch[] = {15.0f, 4.0f};   // fp32, bf16
template <int S>
LinearPlan linear_plan(const LinearShape (&s)[S], const LinearProblem &all) {
    float best, rest_time;
    LinearPlan plan = {best_linear_shape(s, all, &best), 0, all.N};
    for (int i = 0; i < S; ++i) {
        const int64_t mt = (all.M + s[i].bm - 1) / s[i].bm, nt = (all.N + s[i].bn - 1) / s[i].bn;
        const int64_t round = kLinearUnits * s[i].fit;
        const int64_t cols = mt * nt / round * round / mt * s[i].bn;
        if (cols <= 0 || cols >= all.N)
            continue;
        LinearProblem part = all, rest = all;
        part.ragged = rest.ragged = false;   // (each runs beside the other)
        part.N = cols;
        rest.N = all.N - cols;
        const int j = best_linear_shape(s, rest, &rest_time);
        const float t = linear_time(s[i], part) + rest_time +
                        kSecondLaunch[all.bf16];
        if (t < best) {
            best = t;
            plan = {i, j, cols};
        }
    }
    return plan;
}

inline LinearPlan linear_plan(const LinearArgs &a) {
    const LinearSeg &o = a.seg[0];   // (of several, the others are as wide or few columns)
    const int bytes = o.bf16 ? 2 : 4;
    const LinearProblem all = {a.M, a.N, a.K, a.io_bf16 != 0,
                               a.io_bf16 && ((uintptr_t)o.p % 16 != 0 ||
                                             (int64_t)(o.n1 - o.n0) * bytes % 16 != 0)};
    return a.io_bf16 ? linear_plan(kLinearBF16, all) : linear_plan(kLinearF32, all);
}

}  // namespace ssd
