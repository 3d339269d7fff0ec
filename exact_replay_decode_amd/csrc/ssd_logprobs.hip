// ssd_logprobs.hip -- log probability, rank and entropy of one given token per
// row of logits, with the row's best alternatives, in one pass over the row.
//
// With m = max x, s = sum e^(x - m), u = sum e^(x - m) (x - m):
//   log p[i] = x[i] - m - log s,   entropy = log s - u / s.
// m, s and u are kept as running values (rescaled when m grows) per lane and
// joined at the end. A row is cut into chunks of 2048 elements, chunk c
// belongs to stream c % 16, and a wave runs whole streams: lane values over
// the stream's chunks in order, then a DPP tree over the wave, then the 16
// streams in order. So the sums' order depends on V alone, and a row's bits
// depend neither on the number of rows nor on how many waves share the row
// (4, or 16 when there are few rows).
//
// The best top_k: a wave keeps a list of candidates in LDS and a threshold (the
// worst of the best top_k it has seen), so an element costs a comparison of
// its lane's chunk maximum, which the softmax needs anyway. Its first chunk
// (and one with more candidates than the list has room for) sets the
// threshold to the top_k-th largest of the 64 lane maxima: at least top_k
// elements reach it. A list that would still overflow (many equal values) is
// cut to its best top_k element by element, read again from memory. Masked
// elements are no candidates: if fewer than top_k are left, the lists hold
// all of those and the lowest masked indices follow. Keys (value, then lower
// index) are unique 64-bit numbers, so the result does not depend on the
// order of any of this.
// rank counts the elements ahead of the token with one comparison each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_device.hpp"
#include "ssd_step.hpp"

namespace ssd {
namespace {

constexpr int kStreams = 16;
constexpr int kPerLane = 32;
constexpr int kChunkElems = 64 * kPerLane;
constexpr int kList = 256;        // candidates a wave keeps (at least top_k + 64)

// A wave's chunk: 32 elements per lane in 16-byte pieces, piece v of lane l at
// element (64 v + l) E. Rows start anywhere (V may be odd), so the loads are
// declared with the element's alignment only; the hardware takes them.
template <class IO>
struct Chunk;
template <>
struct Chunk<IoBF16> {
    static constexpr int E = 8;
    typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
    __device__ static __forceinline__ void unpack(const uint4 &u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = (__float_as_uint(f[2 * k]) >> 16) | (__float_as_uint(f[2 * k + 1]) & 0xffff0000u);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Chunk<IoF32> {
    static constexpr int E = 4;
    typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(4)));
    __device__ static __forceinline__ void unpack(const uint4 &u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    __device__ static __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

template <class IO>
struct Regs {
    static constexpr int E = Chunk<IO>::E, NV = kPerLane / E;
    uint4 r[NV];
    // elements past V are -inf
    __device__ __forceinline__ void load(const typename IO::T *row, int c, int V, int lane) {
        const int64_t base = (int64_t)c * kChunkElems + lane * E;
        if ((int64_t)(c + 1) * kChunkElems <= V) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const auto x = *reinterpret_cast<const typename Chunk<IO>::vec *>(
                    row + base + v * 64 * E);
                r[v] = make_uint4(x.x, x.y, x.z, x.w);
            }
            return;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int64_t i = base + v * 64 * E + j;
                f[j] = i < V ? IO::ld(row, i) : -INFINITY;
            }
            r[v] = Chunk<IO>::pack(f);
        }
    }
};

// ---- keys: value descending, then index ascending ----------------------------

__device__ __forceinline__ uint64_t key_of(float v, int i) {
    uint32_t b = __float_as_uint(v + 0.0f);   // -0 counts as +0
    b ^= (b >> 31) ? 0xffffffffu : 0x80000000u;
    return ((uint64_t)b << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float key_value(uint64_t k) {
    uint32_t b = (uint32_t)(k >> 32);
    b ^= (b >> 31) ? 0x80000000u : 0xffffffffu;
    return __uint_as_float(b);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

// The candidates of one wave. All members are the same in every lane.
struct TopList {
    uint64_t *keys;       // [kList] of LDS, this wave's own
    int n, k;
    float tau;            // an element counts when it is ahead of (tau, tau_i)
    int tau_i;
    __device__ __forceinline__ bool ahead(float x, int i) const {
        return x > tau || (x == tau && i < tau_i);
    }
    // Keep the best k in order, and raise the threshold to the worst of them.
    __device__ __forceinline__ void cut() {
        const int lane = threadIdx.x & 63;
        uint64_t mine[kList / 64];
        int rank[kList / 64] = {};
#pragma unroll
        for (int i = 0; i < kList / 64; ++i)
            mine[i] = lane + 64 * i < n ? keys[lane + 64 * i] : 0;
        for (int j = 0; j < n; ++j) {
            const uint64_t o = keys[j];
#pragma unroll
            for (int i = 0; i < kList / 64; ++i)
                rank[i] += o > mine[i];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kList / 64; ++i)
            if (lane + 64 * i < n && rank[i] < k)
                keys[rank[i]] = mine[i];
        __builtin_amdgcn_wave_barrier();
        if (n >= k) {
            n = k;
            const uint64_t w = keys[k - 1];
            tau = __uint_as_float(
                __builtin_amdgcn_readfirstlane(__float_as_uint(key_value(w))));
            tau_i = __builtin_amdgcn_readfirstlane(key_index(w));
        }
    }
    // Appends one element of every lane in m (there is room).
    __device__ __forceinline__ void append(uint64_t m, float x, int i) {
        if ((m >> (threadIdx.x & 63)) & 1)
            keys[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] =
                key_of(x, i);
        n += __popcll(m);
    }
    // Raises the threshold to the k-th largest of the lanes' values, when that
    // is higher: k elements at least are equal to it or above.
    __device__ __forceinline__ void raise(float lm) {
        const int lane = threadIdx.x & 63;
        int rank = 0;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lm), i));
            rank += o > lm || (o == lm && i < lane);
        }
        const uint64_t at = __ballot(rank == k - 1);
        if (!at)
            return;   // (a NaN among the maxima)
        const float v = __int_as_float(__builtin_amdgcn_readlane(
            __float_as_int(lm), (int)__ffsll((unsigned long long)at) - 1));
        if (v > tau) {
            tau = v;
            tau_i = INT32_MAX;
        }
    }
};

// v of the lane that DPP control CTRL names, v itself where there is none.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_or_own(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(
        __float_as_int(v), __float_as_int(v), CTRL, ROW_MASK, 0xf, false));
}
__device__ __forceinline__ float lane63(float v) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_or_own<0x111, 0xf>(v));
    v = fmaxf(v, dpp_or_own<0x112, 0xf>(v));
    v = fmaxf(v, dpp_or_own<0x114, 0xf>(v));
    v = fmaxf(v, dpp_or_own<0x118, 0xf>(v));
    v = fmaxf(v, dpp_or_own<0x142, 0xa>(v));
    v = fmaxf(v, dpp_or_own<0x143, 0xc>(v));
    return lane63(v);
}

// e^d by one v_exp_f32
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// Running maximum, sum and weighted sum. An empty one is (-inf, 0, 0).
struct Stat {
    float m, s, u;
    // Takes the values to the new maximum n >= m. (Steps beyond 200 leave
    // nothing in fp32; bounded, since s times the lowest finite value is not.)
    __device__ __forceinline__ void raise(float n) {
        const float d = m == -INFINITY ? 0.0f : fmaxf(m - n, -200.0f);
        const float f = exp_of(d);
        u = f * fmaf(s, d, u);
        s *= f;
        m = n;
    }
};

template <class IO, int NW, bool TOP>
__global__ __launch_bounds__(64 * NW) void k_logprobs(LogprobArgs a) {
    using T = typename IO::T;
    constexpr int E = Chunk<IO>::E, NV = Regs<IO>::NV;
    __shared__ uint64_t keys[NW][TOP ? kList : 1];
    __shared__ float st[kStreams][3];
    __shared__ int ln[NW], ahead_of[NW];
    __shared__ float fin[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = blockIdx.x;
    const int V = a.V;
    const T *row = static_cast<const T *>(a.logits) + t * V;
    const int tok = a.tokens[t];
    const bool valid = tok >= 0 && tok < V;
    const float tv = valid ? IO::ld(row, tok) + 0.0f : 0.0f;
    // x >= tv counts up to the token, x > tv, that is x >= the next float,
    // past it (the piece that holds the token is corrected below)
    const float tv_next = tv >= 0.0f ? __uint_as_float(__float_as_uint(tv) + 1)
                                     : (tv == -__uint_as_float(1)
                                            ? 0.0f
                                            : __uint_as_float(__float_as_uint(tv) - 1));
    const int nchunks = (V + kChunkElems - 1) / kChunkElems;

    // (-inf, 0): nothing that is masked is ahead of it
    TopList top = {keys[wave], 0, a.k, -INFINITY, 0};
    int ahead = 0;
    Regs<IO> cur, nxt;
    int stream = wave, c = wave;
    if (c < nchunks)
        cur.load(row, c, V, lane);
    Stat q = {-INFINITY, 0.0f, 0.0f};
    while (stream < kStreams) {
        // the chunk after this one: same stream, or the wave's next stream
        int nstream = stream, nc = c + kStreams;
        if (nc >= nchunks) {
            nstream = stream + NW;
            nc = nstream;
        }
        if (nstream < kStreams && nc < nchunks)
            nxt.load(row, nc, V, lane);
        if (c < nchunks) {
            float lm = -INFINITY;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[E];
                Chunk<IO>::unpack(cur.r[v], f);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    lm = fmaxf(lm, f[j]);
            }
            if constexpr (TOP) {
                if (top.n == 0)
                    top.raise(lm);
                if (__ballot(lm >= top.tau && lm > -INFINITY)) {
                    const int at = c * kChunkElems + lane * E;
                    const auto count = [&]() {
                        int n = 0;
#pragma unroll
                        for (int v = 0; v < NV; ++v) {
                            float f[E];
                            Chunk<IO>::unpack(cur.r[v], f);
#pragma unroll
                            for (int j = 0; j < E; ++j)
                                n += __popcll(__ballot(top.ahead(f[j], at + 64 * E * v + j)));
                        }
                        return n;
                    };
                    int n = count();
                    if (top.n + n > kList) {
                        top.raise(lm);
                        n = count();
                    }
                    if (top.n + n <= kList) {
#pragma unroll
                        for (int v = 0; v < NV; ++v) {
                            float f[E];
                            Chunk<IO>::unpack(cur.r[v], f);
#pragma unroll
                            for (int j = 0; j < E; ++j) {
                                const int i = at + 64 * E * v + j;
                                const uint64_t m = __ballot(top.ahead(f[j], i));
                                if (m)
                                    top.append(m, f[j], i);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int e = 0; e < kPerLane; ++e) {
                            const int i = at + 64 * E * (e / E) + e % E;
                            const float x = i < V ? IO::ld(row, i) : -INFINITY;
                            uint64_t m = __ballot(top.ahead(x, i));
                            if (top.n + __popcll(m) > kList) {
                                top.cut();
                                m = __ballot(top.ahead(x, i));
                            }
                            if (m)
                                top.append(m, x, i);
                        }
                    }
                }
            }
            if (lm > q.m)
                q.raise(lm);
            const float m = q.m == -INFINITY ? 0.0f : q.m;   // (-inf) - (-inf) kept out
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[E];
                Chunk<IO>::unpack(cur.r[v], f);
                const float least =
                    c * kChunkElems + (64 * v + lane) * E <= tok ? tv : tv_next;
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float d = f[j] - m;
                    const float e = exp_of(d);
                    q.s += e;
                    // a masked element's d is -inf, and 0 * -inf must be 0: below
                    // -200 e is 0 in fp32 already
                    q.u = fmaf(e, fmaxf(d, -200.0f), q.u);
                    ahead += __popcll(__ballot(f[j] >= least));
                }
            }
        }
        if (nstream != stream) {
            const float m = wave_max(q.m);
            if (m > q.m)
                q.raise(m);
            const float s = wave_scan_inclusive(q.s), u = wave_scan_inclusive(q.u);
            if (lane == 63) {
                st[stream][0] = m;
                st[stream][1] = s;
                st[stream][2] = u;
            }
            q = {-INFINITY, 0.0f, 0.0f};
        }
        stream = nstream;
        c = nc;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            cur.r[v] = nxt.r[v];
    }
    if constexpr (TOP)
        top.cut();
    if (lane == 0) {
        ln[wave] = top.n;
        ahead_of[wave] = ahead;
    }
    __syncthreads();

    if (wave == 0) {
        Stat z = {-INFINITY, 0.0f, 0.0f};
        for (int i = 0; i < kStreams; ++i) {
            Stat o = {st[i][0], st[i][1], st[i][2]};
            const float m = fmaxf(z.m, o.m);
            if (m > z.m)
                z.raise(m);
            if (m > o.m)
                o.raise(m);
            z.s += o.s;
            z.u += o.u;
        }
        const bool none = z.m == -INFINITY && z.s == 0.0f;   // nothing left, and no NaN
        const bool bad = !(z.s < INFINITY);                    // a NaN or +inf in the row
        const float ls = none ? 0.0f : logf(z.s);
        // of the piece that holds the token, the elements from the token on that
        // are no more than equal to it were counted; so were -inf paddings
        int over = 0;
        if (valid && lane < E) {
            const int i = tok / E * E + lane;
            const float x = i < V ? IO::ld(row, i) : -INFINITY;
            over = i >= tok && x == tv;
        }
        const int surplus = __popcll(__ballot(over));
        if (lane == 0) {
            const float nan = __uint_as_float(0x7fc00000u);
            a.logprob[t] = !valid || bad ? nan : (none || tv == -INFINITY ? -INFINITY
                                                                          : tv - z.m - ls);
            if (a.entropy)
                a.entropy[t] = bad ? nan : (none ? 0.0f : ls - z.u / z.s);
            if (a.rank) {
                int n = 0;
                for (int w = 0; w < NW; ++w)
                    n += ahead_of[w];
                a.rank[t] = !valid || bad ? -1 : n - surplus;
            }
            fin[0] = z.m;
            fin[1] = ls;
            fin[2] = bad ? 1.0f : 0.0f;
        }
    }
    if constexpr (!TOP)
        return;
    __syncthreads();
    const bool bad = fin[2] != 0.0f;
    int32_t *ids = a.top_ids + t * a.k;
    float *lps = a.top_logprobs + t * a.k;
    if (bad) {
        for (int i = threadIdx.x; i < a.k; i += 64 * NW) {
            ids[i] = -1;
            lps[i] = __uint_as_float(0x7fc00000u);
        }
        return;
    }
    // Join the waves' sorted lists: an element's place is its place in its own
    // list plus the elements ahead of it in the others.
    int left = 0;   // candidates in all lists
    for (int w = 0; w < NW; ++w)
        left += ln[w];
    if (lane < ln[wave]) {
        const uint64_t me = keys[wave][lane];
        int rank = lane;
        for (int w = 0; w < NW; ++w) {
            if (w == wave)
                continue;
            int lo = 0, hi = ln[w];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (keys[w][mid] > me)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            rank += lo;
        }
        if (rank < a.k) {
            ids[rank] = key_index(me);
            lps[rank] = key_value(me) - fin[0] - fin[1];
        }
    }
    // Fewer than top_k unmasked: all of them are in the lists, and the lowest
    // masked indices follow. Index i < 2 k is masked when no list has it, and
    // its place is left + i - (listed indices below i).
    if (left < a.k) {
        for (int i = threadIdx.x; i < 2 * a.k && i < V; i += 64 * NW) {
            int below = 0;
            bool listed = false;
            for (int w = 0; w < NW; ++w)
                for (int j = 0; j < ln[w]; ++j) {
                    const int o = key_index(keys[w][j]);
                    below += o < i;
                    listed |= o == i;
                }
            const int place = left + i - below;
            if (!listed && place < a.k) {
                ids[place] = i;
                lps[place] = -INFINITY;
            }
        }
    }
}

template <class IO>
hipError_t logprobs_impl(const LogprobArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)a.T);
    if (a.T <= 256) {
        if (a.k > 0)
            k_logprobs<IO, 16, true><<<grid, dim3(1024), 0, stream>>>(a);
        else
            k_logprobs<IO, 16, false><<<grid, dim3(1024), 0, stream>>>(a);
    } else {
        if (a.k > 0)
            k_logprobs<IO, 4, true><<<grid, dim3(256), 0, stream>>>(a);
        else
            k_logprobs<IO, 4, false><<<grid, dim3(256), 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t stream) {
    return a.bf16 ? logprobs_impl<IoBF16>(a, stream) : logprobs_impl<IoF32>(a, stream);
}

}  // namespace ssd
