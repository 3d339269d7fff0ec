// ssd_linear.hip -- matrix product with bias, activation and residual in its
// epilogue: the mixer's projections (and any other linear layer of a step).
//   out[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
//
// Every output is an fp32 accumulation chain of matrix-core instructions over
// 64-byte steps of k, ascending from zero: one v_mfma_f32_16x16x32_bf16 for the
// step's 32 k in bf16, four v_mfma_f32_16x16x4_f32 for its 16 k in fp32 (the
// i-th takes k = i, 4 + i, 8 + i, 12 + i of the step), where a chain ends after 512 k
// and the chains are added in turn; k past K are zeros on both sides. An MFMA result
// element depends on its own row, its own column and its accumulator only, so every tile
// shape here gives the same bits, and a row's bits do not depend on the number of rows.
// (A wave has all of k: work comes from outputs alone, and few of them with a long k
// take the time of their sum.)
//
// The instruction's rows are output columns n and its columns are rows m of x:
// a lane then holds four consecutive n of one row.
//
// What bounds it, measured with copies that leave parts out: at 8192^3 (uniform values)
// the matrix instructions and LDS reads alone take 596 us, the loads alone 710,
// together 835 (1320 TFLOP/s; normal values 835-890, the library's product 743-764); the
// LDS serves both, 96 of its 128 bytes a cycle to the reads of 128 x 64 wave tiles and
// 32 to the loads at the matrix cores' full rate. 8192 x 10304 x 2048
// takes 302-320 us, card to card (1080-1150 TFLOP/s; the library 335-360). At 256 x 2048 x
// 4096 (one 64 x 32 tile per compute unit, one wave per SIMD, and as many that load) the
// reads and MFMAs alone take 10.9 us of a stream of launches, the loads alone 10.2 (13.8
// with w from memory), together 12.5 (14.5). A few rows stream w: 1 row x 50280 x 2048 in
// 41 us, 16 rows in 42 (206 MB, 4.9-5.0 TB/s).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <iterator>

#include "ssd_linear_choice.hpp"
#include "ssd_step.h"
#include "ssd_step.hpp"
#include "ssd_step_device.hpp"

namespace ssd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- epilogue ---------------------------------------------------------------

// f32: for an fp32 output. (Branches for the eight together: a switch for each of them
// and full divisions cost 4 us of 20 in 256 x 128 tiles.)
__device__ __forceinline__ void activate(float (&v)[8], int act, bool f32) {
    if (act == SSD_ACT_RELU2) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = v[i] <= 0.0f ? 0.0f : v[i] * v[i];   // (a NaN stays one)
        return;
    }
    if (act != SSD_ACT_SILU && act != SSD_ACT_GELU)
        return;
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        u[i] = v[i];
    if (act == SSD_ACT_GELU) {
        // 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), u = sqrt(2/pi)(v + 0.044715 v^3)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = 1.5957691216057308f * fmaf(0.044715f * v[i] * v[i], v[i], v[i]);
    }
    if (f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= sigmoid_f32(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= sigmoid_bf16(u[i]);
    }
}

// Columns n .. n + 7 of row m, n a multiple of 8: bias, activation, residual, one
// rounding, 16-byte accesses where the eight are all there (of any alignment:
// N may be odd).
__device__ __forceinline__ void store_eight(const LinearArgs &a, int m, int n, float (&v)[8]) {
    typedef f32x4 f32x4_u __attribute__((aligned(4)));
    typedef u32x4 u32x4_u __attribute__((aligned(2)));
    LinearSeg s = a.seg[0];
    if (a.nseg > 1 && n >= s.n1)
        s = n >= a.seg[1].n1 ? a.seg[2] : a.seg[1];
    const int64_t at = (int64_t)m * (s.n1 - s.n0) + (n - s.n0);
    const int cnt = a.hi - n;
    float r[8];
    if (cnt >= 8) {
        if (a.bias) {
            const f32x4 b0 = reinterpret_cast<const f32x4_u *>(a.bias + n)[0];
            const f32x4 b1 = reinterpret_cast<const f32x4_u *>(a.bias + n)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += b0[i];
                v[i + 4] += b1[i];
            }
        }
        if (a.residual) {
            if (a.io_bf16) {
                const u32x4 w = *reinterpret_cast<const u32x4_u *>(
                    static_cast<const uint16_t *>(a.residual) + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[2 * i] = __uint_as_float(w[i] << 16);
                    r[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            } else {
                const f32x4_u *p = reinterpret_cast<const f32x4_u *>(
                    static_cast<const float *>(a.residual) + at);
                const f32x4 r0 = p[0], r1 = p[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[i] = r0[i];
                    r[i + 4] = r1[i];
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < cnt && a.bias)
                v[i] += a.bias[n + i];
            if (i < cnt && a.residual)
                r[i] = a.io_bf16 ? IoBF16::ld(static_cast<const uint16_t *>(a.residual), at + i)
                                 : static_cast<const float *>(a.residual)[at + i];
        }
    }
    activate(v, a.act, !s.bf16);
    if (a.residual)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += r[i];
    if (cnt >= 8) {
        if (s.bf16) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = bf16_rne(v[2 * i]) | ((uint32_t)bf16_rne(v[2 * i + 1]) << 16);
            *reinterpret_cast<u32x4_u *>(static_cast<uint16_t *>(s.p) + at) = w;
        } else {
            f32x4_u *p = reinterpret_cast<f32x4_u *>(static_cast<float *>(s.p) + at);
            p[0] = (f32x4){v[0], v[1], v[2], v[3]};
            p[1] = (f32x4){v[4], v[5], v[6], v[7]};
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < cnt) {
            if (s.bf16)
                static_cast<uint16_t *>(s.p)[at + i] = bf16_rne(v[i]);
            else
                static_cast<float *>(s.p)[at + i] = v[i];
        }
}

// ---- tiles through LDS --------------------------------------------------------

// The wave's number as a scalar (what is computed from it then is, too).
__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

typedef __attribute__((address_space(3))) void lds_void;

// k of one fp32 chain. A longer sum is several, added in ascending order: the error of
// a chain grows with the root of its length (64 x 64 x 16384 in one: 2.3e-6 of the
// values' root mean square; in chains of 512, whatever K is: 4.1e-7), and where they
// end depends on K alone. It costs 1-4 % of the time (256 x 2048 x 4096: 43.2 -> 44.9 us).
// A bf16 step adds 32 products at a time; that stays one chain (1.8e-7 at K = 1024,
// 8.3e-7 at 16384).
constexpr int kChain = 512;

// A workgroup computes BM rows x BN columns, in (BM / WM) (BN / WN) waves of
// WM x WN each (16 x 16 tiles). Both operands pass through LDS in tiles of 2 BK
// bytes of k (BK bf16, BK / 2 fp32), S buffers in turn: the direct loads
// (global_load_lds, 16 bytes a lane) of the S - 1 tiles ahead run while the matrix
// cores work on this one. NL waves issue
// the loads; with APART waves of their own, where a compute unit has one small
// tile and the issue of the loads would hold up its few MFMAs (256 x 2048 x 4096 in
// 64 x 32 tiles: 15.8 us, 12.5 with four loading waves apart, 12.4 with eight).
// LDS layout: row r of a tile at 2 BK r bytes, its 16-byte piece c at c ^ (r % 8),
// so that the 16 rows that a fragment read touches spread over the banks. A
// direct load fills 1 KB in lane order, whole rows or more, so a lane fetches
// the piece that belongs at its place.
template <bool F32_, int BM_, int BN_, int WM_, int WN_, int BK_, int S_, int NL_ = 0,
          bool APART = false>
struct Tile {
    static constexpr bool F32 = F32_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, S = S_;
    static constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN;
    static constexpr int NL = NL_ ? NL_ : NW;
    static constexpr int L0 = APART ? NW : 0;             // the first wave that loads
    static constexpr int WAVES = L0 + NL > NW ? L0 + NL : NW;
    static constexpr int FM = WM / 16, FN = WN / 16;
    static constexpr int CHAIN = F32 ? 2 * kChain / BK : 0;   // tiles of a chain; 0: all
    static constexpr int PIECES = BK / 8;                 // 16-byte pieces of a row
    static constexpr int RPL = 64 / PIECES;               // rows of one direct load
    static constexpr int LX = BM / RPL / NL, LW = BN / RPL / NL;   // loads per wave
    static constexpr int BYTES = (BM + BN) * BK * 2, XBYTES = BM * BK * 2;
    // fp32 (two sets of sums): registers for as many waves a SIMD as the LDS has room for
    static constexpr int PER_SIMD = F32 ? 160 * 1024 / (S * BYTES) * WAVES / 4 : 1;
    static_assert(!F32 || 2 * kChain % BK == 0, "chains end with a tile, in every shape alike");
    static_assert(PIECES >= 8, "a row of the tile covers all eight places of swizzle()");
    static_assert(BM % (RPL * NL) == 0 && BN % (RPL * NL) == 0, "loads divide over the waves");
    static_assert(S * BYTES <= 160 * 1024, "LDS of a compute unit");
};

// One direct load of 1 KB: lane l's 16 bytes from base + off to LDS byte
// lds + 16 l. (An asm statement without register outputs: the compiler, which
// cannot tell the buffers apart, would wait for all loads in flight before
// each LDS read; the kernel waits at its barriers instead. m0 is an operand, so the
// compiler keeps track of it; the load may not follow its writing at once.)
__device__ __forceinline__ void direct_load(uint32_t lds, const char *base, uint32_t off) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "{m0}"(lds), "v"(off), "s"(base)
                 : "memory");
}

// Waits for this wave's direct loads except the newest N and its LDS reads,
// then for the workgroup.
template <int N>
__device__ __forceinline__ void loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// What a row's pieces are exchanged by: eight rows that are read together
// cover the 128 bytes of a bank row.
__device__ __forceinline__ int swizzle(int row) { return row & 7; }

template <class C>
struct TileLoader {
    const char *x, *w;                // the tile's first row
    uint32_t ox[C::LX], ow[C::LW];    // per-lane byte offsets of the wave's loads
    uint32_t lx, lw;                  // LDS offsets of the wave's loads in a buffer
    int nx;                           // loads of x that hold rows below M
    __device__ __forceinline__ TileLoader(const LinearArgs &a, int m0, int n0) {
        const int lane = threadIdx.x & 63, wave = wave_id() - C::L0;
        const uint32_t rb = row_bytes(a);
        x = static_cast<const char *>(a.x) + (int64_t)m0 * rb;
        w = static_cast<const char *>(a.w) + (int64_t)n0 * rb;
        // (rows past the end read the last row; what they give is not stored)
#pragma unroll
        for (int i = 0; i < C::LX; ++i)
            ox[i] = offset(wave * C::LX + i, lane, a.M - 1 - m0, rb);
#pragma unroll
        for (int i = 0; i < C::LW; ++i)
            ow[i] = offset(wave * C::LW + i, lane, a.hi - 1 - n0, rb);
        lx = 1024 * wave * C::LX;
        lw = C::XBYTES + 1024 * wave * C::LW;
        nx = (a.M - m0 + C::RPL - 1) / C::RPL - wave * C::LX;
    }
    // Byte offset of the lane's piece of load number i of an operand.
    __device__ static __forceinline__ int piece(int i, int lane) {
        const int row = i * C::RPL + lane / C::PIECES;
        return (lane % C::PIECES) ^ swizzle(row);
    }
    __device__ static __forceinline__ uint32_t offset(int i, int lane, int last, uint32_t rb) {
        const int row = i * C::RPL + lane / C::PIECES;
        return (uint32_t)min(row, last) * rb + 16 * piece(i, lane);
    }
    __device__ static __forceinline__ uint32_t row_bytes(const LinearArgs &a) {
        return (uint32_t)a.K * (C::F32 ? 4 : 2);
    }
    // Tile at byte kb of the rows, all 2 BK bytes of it there. Loads of x whose rows
    // are all past M are left out: those rows of the buffer feed columns of the
    // result that are not stored.
    __device__ __forceinline__ void load(char *buf, int64_t kb) const {
        const uint32_t lds = (uint32_t)(uintptr_t)(lds_void *)buf;
#pragma unroll
        for (int i = 0; i < C::LX; ++i)
            if (C::BM > 32 || i < nx)
                direct_load(lds + lx + 1024 * i, x + kb, ox[i]);
#pragma unroll
        for (int i = 0; i < C::LW; ++i)
            direct_load(lds + lw + 1024 * i, w + kb, ow[i]);
    }
    // The last tile when 2 BK does not divide a row (left: what is there, in units
    // of 2 bytes): pieces past the row fetch the tile's first piece instead, and
    // count as zeros when they are read.
    __device__ __forceinline__ void load_tail(char *buf, int64_t kb, int left) const {
        int lane = threadIdx.x & 63;
        const int wave = wave_id() - C::L0;
        if constexpr (C::F32)   // (no registers for these offsets through the loop before)
            asm volatile("" : "+v"(lane));
        const uint32_t lds = (uint32_t)(uintptr_t)(lds_void *)buf;
        const auto at = [&](uint32_t off, int i) {
            const int p = piece(i, lane);
            return 8 * p < left ? off : off - 16 * p;
        };
#pragma unroll
        for (int i = 0; i < C::LX; ++i)
            if (C::BM > 32 || i < nx)
                direct_load(lds + lx + 1024 * i, x + kb, at(ox[i], wave * C::LX + i));
#pragma unroll
        for (int i = 0; i < C::LW; ++i)
            direct_load(lds + lw + 1024 * i, w + kb, at(ow[i], wave * C::LW + i));
    }
};

// One step of a 16 x 16 tile: lane l's operands are 16 bytes of row (column) l % 16
// at byte 16 (l / 16) of the step.
template <bool F32>
__device__ __forceinline__ f32x4 mma_step(const u32x4 &w, const u32x4 &x, f32x4 acc) {
    if constexpr (F32) {
        const f32x4 fw = __builtin_bit_cast(f32x4, w), fx = __builtin_bit_cast(f32x4, x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fw[i], fx[i], acc, 0, 0, 0);
        return acc;
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    }
}

// NK steps of an LDS tile, from step k0: the w fragments of a step stay,
// the x fragments come in groups of two, and the reads of the group after next
// (and of its step's w) go out before this group's MFMAs. In the last, partial
// tile (TAIL) pieces from `left` on are zeros.
template <class C, int NK, bool TAIL = false>
__device__ __forceinline__ void tile_steps(const char *buf, f32x4 (&acc)[C::FM][C::FN],
                                           int k0 = 0, int left = 0) {
    constexpr int G = C::FM < 2 ? 1 : 2, NG = C::FM / G;
    constexpr int AHEAD = 2;   // groups read ahead
    constexpr int RX = AHEAD + 1, RW = 1 + (AHEAD + NG - 1) / NG;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15;
    const char *px = buf + ((wave % C::NWM) * C::WM + r) * (2 * C::BK);
    const char *pw = buf + C::XBYTES + ((wave / C::NWM) * C::WN + r) * (2 * C::BK);
    const auto piece = [&](int kk) { return 16 * ((4 * (k0 + kk) + (lane >> 4)) ^ swizzle(r)); };
    u32x4 x[RX][G], w[RW][C::FN];
    const auto fragment = [&](const char *p, int kk) {
        u32x4 f = *reinterpret_cast<const u32x4 *>(p + piece(kk));
        if (TAIL && 8 * (4 * (k0 + kk) + (lane >> 4)) >= left)
            f = (u32x4){0, 0, 0, 0};
        return f;
    };
    const auto read = [&](int s) {
        const int kk = s / NG, g = s % NG;
        if (g == 0)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                w[kk % RW][j] = fragment(pw + j * 16 * (2 * C::BK), kk);
#pragma unroll
        for (int i = 0; i < G; ++i)
            x[s % RX][i] = fragment(px + (g * G + i) * 16 * (2 * C::BK), kk);
    };
#pragma unroll
    for (int s = 0; s < AHEAD && s < NK * NG; ++s)
        read(s);
#pragma unroll
    for (int s = 0; s < NK * NG; ++s) {
        const int kk = s / NG, g = s % NG;
        if (s + AHEAD < NK * NG)
            read(s + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                acc[g * G + i][j] =
                    mma_step<C::F32>(w[kk % RW][j], x[s % RX][i], acc[g * G + i][j]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Which tile a workgroup computes. Workgroup b runs on XCD b % 8, whose L2 the
// others do not share. Tiles run down the rows, then along the columns. With
// eight row tiles or more, an XCD that takes every eighth tile sees an eighth of
// the rows of x. With fewer, it takes a run of tiles instead, all rows of an
// eighth of the columns, so that w, the larger operand then, goes to one XCD
// (256 x 2048 x 4096 as 64 x 32 tiles: 12.5 against 20.5 us; 8192 x 8192 x 8192
// the other way round: 835 against 1000 us).
__device__ __forceinline__ bool tile_of(int b, int mtiles, int ntiles, int &m, int &n) {
    const int t = mtiles < 8 ? (b & 7) * (int)(gridDim.x >> 3) + (b >> 3) : b;
    m = t % mtiles;
    n = t / mtiles;
    return n < ntiles;
}

template <class C>
__global__ __launch_bounds__(64 * C::WAVES, C::PER_SIMD)
void k_linear_tile(LinearArgs a, int mtiles, int ntiles) {
    constexpr int S = C::S, BK = C::BK;
    __shared__ __attribute__((aligned(1024))) char buf[S * C::BYTES];
    const int wave = wave_id();
    int m0, n0;
    if (!tile_of(blockIdx.x, mtiles, ntiles, m0, n0))
        return;
    m0 *= C::BM;
    n0 = a.lo + n0 * C::BN;
    const bool loads = C::NL == C::WAVES || (wave >= C::L0 && wave < C::L0 + C::NL);
    const bool works = C::NW == C::WAVES || wave < C::NW;
    const TileLoader<C> ld(a, m0, n0);
    f32x4 acc[C::FM][C::FN] = {}, total[C::FM][C::FN] = {};
    const auto end_chain = [&] {
        asm volatile("");   // (a branch: selections would wait for the sums after each tile)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                total[i][j] += acc[i][j];
                acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            }
    };
    const int k2 = a.K * (C::F32 ? 2 : 1);   // a row in units of 2 bytes
    const int full = k2 / BK, left = k2 % BK, tiles = full + (left != 0);
    const auto load = [&](int t, int slot) {
        if (C::F32 ? __builtin_expect(t < full, 1) : t < full)
            ld.load(buf + slot * C::BYTES, (int64_t)t * BK * 2);
        else
            ld.load_tail(buf + slot * C::BYTES, (int64_t)t * BK * 2, left);
    };
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
        if (t < tiles && loads)
            load(t, t);
    int slot = 0, ahead = S - 1;      // t % S and (t + S - 1) % S
    for (int t = 0; t < full; ++t) {
        // tile t is there when only the loads of the S - 2 tiles after it are in
        // flight (with loads left out fewer: that waits for more); past the
        // barrier every wave has read tile t - 1, whose buffer is loaded next
        if (C::BM > 32 && t + S - 2 < tiles)
            loads_barrier<(S - 2) * (C::LX + C::LW)>();
        else if (t + S - 2 < tiles)
            loads_barrier<(S - 2) * C::LW>();
        else
            loads_barrier<0>();
        if (t + S - 1 < tiles && loads)
            load(t + S - 1, ahead);
        if (works)
            tile_steps<C, BK / 32>(buf + slot * C::BYTES, acc);
        if constexpr (C::CHAIN > 0)
            if ((t + 1) % C::CHAIN == 0)
                end_chain();
        slot = slot + 1 == S ? 0 : slot + 1;
        ahead = ahead + 1 == S ? 0 : ahead + 1;
    }
    if (left) {
        loads_barrier<0>();
        if (works)
#pragma unroll 1
            for (int k = 0; k < left; k += 32)
                tile_steps<C, 1, true>(buf + slot * C::BYTES, acc, k / 32, left);
    }
    if constexpr (C::CHAIN > 0)
        end_chain();
    const auto &sum = *(C::CHAIN > 0 ? &total : &acc);
    __syncthreads();
    if (!works)
        return;
    // Epilogue through LDS, 32 of the wave's rows at a time in its own part of
    // the buffers, so that lanes store eight columns of a row together. (A row
    // is WN + 4 floats long: the 16 rows of a tile write to different banks.)
    constexpr int PITCH = C::WN + 4;
    constexpr int HALF = C::FM < 2 || 32 * PITCH * 4 * C::NW > S * C::BYTES ? 1 : 2;
    constexpr int PART = HALF * 16 * PITCH;
    static_assert(PART * 4 * C::NW <= S * C::BYTES, "fits the buffers");
    const int lane = threadIdx.x & 63;
    float *mine = reinterpret_cast<float *>(buf) + wave * PART;
    const int wm = m0 + (wave % C::NWM) * C::WM, wn = n0 + (wave / C::NWM) * C::WN;
#pragma unroll
    for (int h = 0; h < C::FM / HALF; ++h) {
#pragma unroll
        for (int i = 0; i < HALF; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                *reinterpret_cast<f32x4 *>(mine + (16 * i + (lane & 15)) * PITCH + 16 * j +
                                           4 * (lane >> 4)) = sum[h * HALF + i][j];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int e = lane; e < HALF * 16 * (C::WN / 8); e += 64) {
            const int row = e / (C::WN / 8), col = e % (C::WN / 8) * 8;
            const int m = wm + h * HALF * 16 + row, n = wn + col;
            if (m < a.M && n < a.hi) {
                const f32x4 v0 = *reinterpret_cast<const f32x4 *>(mine + row * PITCH + col);
                const f32x4 v1 = *reinterpret_cast<const f32x4 *>(mine + row * PITCH + col + 4);
                float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
                store_eight(a, m, n, v);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---- launches ---------------------------------------------------------------

// `each` launches the shape it is given over the columns of its arguments.
template <class F>
hipError_t by_columns(LinearArgs a, F each) {
    const LinearPlan plan = linear_plan(a);
    a.lo = 0;
    a.hi = (int32_t)plan.n1;
    const hipError_t e = each(plan.first, a);
    if (e != hipSuccess || plan.n1 == a.N)
        return e;
    a.lo = (int32_t)plan.n1;
    a.hi = a.N;
    return each(plan.second, a);
}

template <class C>
hipError_t launch_tile(const LinearArgs &a, hipStream_t stream) {
    const int64_t mt = (a.M + C::BM - 1) / C::BM, nt = (a.hi - a.lo + C::BN - 1) / C::BN;
    // (a multiple of 8: runs of tiles for the XCDs)
    const dim3 grid((unsigned)((mt * nt + 7) / 8 * 8));
    k_linear_tile<C><<<grid, dim3(64 * C::WAVES), 0, stream>>>(a, (int)mt, (int)nt);
    return hipGetLastError();
}

hipError_t linear_bf16(const LinearArgs &args, hipStream_t stream) {
    static_assert(std::size(kLinearBF16) == 13, "a kernel for each shape");
    return by_columns(args, [&](int shape, const LinearArgs &a) {
        switch (shape) {
        case 0: return launch_tile<Tile<false, 16, 16, 16, 16, 256, 3, 4>>(a, stream);
        case 1: return launch_tile<Tile<false, 16, 16, 16, 16, 256, 4, 8, true>>(a, stream);
        case 2: return launch_tile<Tile<false, 16, 32, 16, 16, 256, 3, 4, true>>(a, stream);
        case 3: return launch_tile<Tile<false, 32, 32, 16, 16, 256, 2, 4, true>>(a, stream);
        case 4: return launch_tile<Tile<false, 64, 32, 32, 16, 256, 3, 4, true>>(a, stream);
        case 5: return launch_tile<Tile<false, 64, 64, 32, 32, 64, 4>>(a, stream);
        case 6: return launch_tile<Tile<false, 64, 64, 32, 32, 128, 4, 4, true>>(a, stream);
        case 7: return launch_tile<Tile<false, 128, 64, 32, 32, 64, 3>>(a, stream);
        case 8: return launch_tile<Tile<false, 128, 64, 64, 32, 128, 3, 4, true>>(a, stream);
        case 9: return launch_tile<Tile<false, 128, 128, 32, 64, 64, 2>>(a, stream);
        case 10: return launch_tile<Tile<false, 128, 128, 64, 32, 64, 4, 4, true>>(a, stream);
        case 11: return launch_tile<Tile<false, 256, 128, 64, 64, 64, 3, 4, true>>(a, stream);
        default: return launch_tile<Tile<false, 256, 256, 128, 64, 64, 2>>(a, stream);
        }
    });
}

hipError_t linear_f32(const LinearArgs &args, hipStream_t stream) {
    static_assert(std::size(kLinearF32) == 10, "a kernel for each shape");
    return by_columns(args, [&](int shape, const LinearArgs &a) {
        switch (shape) {
        case 0: return launch_tile<Tile<true, 16, 16, 16, 16, 256, 3, 4>>(a, stream);
        case 1: return launch_tile<Tile<true, 32, 32, 16, 16, 256, 2, 8, true>>(a, stream);
        case 2: return launch_tile<Tile<true, 32, 32, 16, 16, 128, 3>>(a, stream);
        case 3: return launch_tile<Tile<true, 32, 64, 16, 16, 128, 2>>(a, stream);
        case 4: return launch_tile<Tile<true, 64, 32, 32, 16, 128, 2>>(a, stream);
        case 5: return launch_tile<Tile<true, 64, 32, 32, 16, 256, 3, 4, true>>(a, stream);
        case 6: return launch_tile<Tile<true, 64, 64, 32, 32, 128, 2>>(a, stream);
        case 7: return launch_tile<Tile<true, 96, 64, 32, 16, 128, 2, 4>>(a, stream);
        case 8: return launch_tile<Tile<true, 128, 64, 32, 32, 64, 2>>(a, stream);
        default: return launch_tile<Tile<true, 128, 128, 32, 64, 64, 2>>(a, stream);
        }
    });
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t stream) {
    return a.io_bf16 ? linear_bf16(a, stream) : linear_f32(a, stream);
}

}  // namespace ssd
