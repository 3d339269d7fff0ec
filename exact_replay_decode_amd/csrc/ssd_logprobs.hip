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
// (4 or 16).
//
// The best top_k in short steps after the pass, from what the softmax needs
// anyway, the maxima of each lane's 32 elements of a chunk (a segment; kept in
// LDS): the lanes form 128 groups (64 for a small top_k), the top_k-th largest of
// the groups' maxima bounds the row's top_k-th best from below, and only the
// segments that reach it are read again (for top_k = 20 about 25), a wave two at a time. The
// candidates' places are counted. Keys (value, then lower index) are unique
// 64-bit numbers, so the result does not depend on the order of any of this.
// Masked elements are no candidates: when fewer than top_k are left, the lowest
// masked indices follow. A row with too many best values for the lists (equal
// ones) is read again element by element into sorted lists, one per wave, which
// are then joined.
// rank counts the elements ahead of the token with one comparison each.
//
// Measured: 4096 rows of 50280 bf16 in 84 us without alternatives (4.9 TB/s), where
// the vector unit's work (a row's elements at 48 cycles per 64) is 63 us; an operation
// an element fewer changed nothing, so the waits between chunks bound it. 512 rows of
// 131072 with one token in 500 allowed and top 8: 30-32 us, 4.2-4.5 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_device.hpp"
#include "ssd_step.hpp"

namespace ssd {
namespace {

constexpr int kStreams = kLogprobStreams;
constexpr int kPerLane = 32;
constexpr int kChunkElems = 64 * kPerLane;
static_assert(kChunkElems == kLogprobChunk, "a wave's chunk");
constexpr int kSegs = 1024;       // segments read again
constexpr int kCands = 1024;      // candidates (top_k = 64: 90 in the mean)

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
            w[k] = (__float_as_uint(f[2 * k]) >> 16) |
                   (__float_as_uint(f[2 * k + 1]) & 0xffff0000u);
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

// The candidates of one wave, for rows that overflow the short way. All members
// are the same in every lane. LIST >= top_k + 64.
template <int LIST>
struct TopList {
    uint64_t *keys;       // [LIST] of LDS, this wave's own
    int n, k;
    float tau;            // an element counts when it is ahead of (tau, tau_i)
    int tau_i;
    __device__ __forceinline__ bool ahead(float x, int i) const {
        return x > tau || (x == tau && i < tau_i);
    }
    // Keep the best k in order, and raise the threshold to the worst of them.
    __device__ __forceinline__ void cut() {
        const int lane = threadIdx.x & 63;
        uint64_t mine[LIST / 64];
        int rank[LIST / 64] = {};
#pragma unroll
        for (int i = 0; i < LIST / 64; ++i)
            mine[i] = lane + 64 * i < n ? keys[lane + 64 * i] : 0;
        for (int j = 0; j < n; ++j) {
            const uint64_t o = keys[j];
#pragma unroll
            for (int i = 0; i < LIST / 64; ++i)
                rank[i] += o > mine[i];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < LIST / 64; ++i)
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
};

// Place of a lane's entry in a list that *count numbers: one LDS atomic a wave.
__device__ __forceinline__ int append_at(uint64_t m, int *count) {
    int base = 0;
    if ((threadIdx.x & 63) == 0)
        base = atomicAdd(count, __popcll(m));
    return __builtin_amdgcn_readfirstlane(base) +
           __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                     __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

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

// The k-th largest of the lanes' values (no NaN among them), 1 <= k <= 64: the
// least value with fewer than k above it; of 64 values, and of 128.
__device__ __forceinline__ float wave_kth(float v, int k) {
    int above = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i)
        above += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)) > v;
    return -wave_max(above < k ? -v : -INFINITY);
}
__device__ __forceinline__ float wave_kth(float v, float w, int k) {
    int av = 0, aw = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
        const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), i));
        av += a > v;
        aw += a > w;
        av += b > v;
        aw += b > w;
    }
    return -wave_max(fmaxf(av < k ? -v : -INFINITY, aw < k ? -w : -INFINITY));
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

// Segment maxima of a wave: ORD rows of 64 lanes, row (its chunk's number / R).
template <int NW>
struct Segs {
    static constexpr int ORD = 64 / NW;
};

// (bf16: 64 registers and less than 20 KB of LDS, so that 32 waves share a compute unit:
// 2048 rows of 50280 with top 8 in 52 us, 60 with 28 waves)
template <class IO, int NW, bool TOP>
__global__ __launch_bounds__(64 * NW, sizeof(typename IO::T) == 2 ? 8 : 1)
void k_logprobs(LogprobArgs a) {
    using T = typename IO::T;
    constexpr int E = Chunk<IO>::E, NV = Regs<IO>::NV, ORD = Segs<NW>::ORD;
    constexpr int LIST = NW == 4 ? 256 : 128;
    // segment maxima; past the listing of the segments the candidates, or the lists
    __shared__ __attribute__((aligned(8))) float smax[TOP ? NW * ORD * 64 : 1];
    __shared__ uint16_t few[TOP ? kSegs : 1];       // segments
    uint64_t *cand = reinterpret_cast<uint64_t *>(smax);
    __shared__ float st[kStreams][3];
    __shared__ int ahead_of[NW], ln[NW];
    __shared__ float gm[128];
    __shared__ float fin[3];
    __shared__ int count[2];
    __shared__ float tau_row;
    static_assert(sizeof(uint64_t) * NW * LIST <= sizeof(float) * NW * ORD * 64, "in smax's place");
    static_assert(sizeof(uint64_t) * kCands <= sizeof(float) * NW * ORD * 64, "in smax's place");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    // chunks of a wave per row of its segment maxima
    const int wchunks = (kStreams / NW) * ((nchunks + kStreams - 1) / kStreams);
    const int R = (wchunks + ORD - 1) / ORD;
    if (TOP && threadIdx.x < 2)
        count[threadIdx.x] = 0;

    int ahead = 0, ord = 0;
    float best = -INFINITY, seg = -INFINITY;   // this lane's, over all chunks and this row's
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
                best = fmaxf(best, lm);
                seg = fmaxf(seg, lm);
                smax[(wave * ORD + ord / R) * 64 + lane] = seg;
                if (++ord % R == 0)
                    seg = -INFINITY;
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
    if (lane == 0)
        ahead_of[wave] = ahead;
    if constexpr (TOP) {
        // maxima of groups of NW / 2 lanes, in the group's last lane (DPP row
        // shifts reach the lanes below within 16)
        static_assert(NW == 4 || NW == 16, "128 groups");
        float g = fmaxf(best, dpp_or_own<0x111, 0xf>(best));
        if constexpr (NW == 16) {
            g = fmaxf(g, dpp_or_own<0x112, 0xf>(g));
            g = fmaxf(g, dpp_or_own<0x114, 0xf>(g));
        }
        if (lane % (NW / 2) == NW / 2 - 1)
            gm[(wave * 64 + lane) / (NW / 2)] = g;
    }
    __syncthreads();

    if (TOP && wave == 1) {
        // (64 groups bound a small top_k well enough; the other waves wait here: uniform
        // bf16 of 50280, top 8, 117 against 120 us for 4096 rows, 21.7 against 22.8 for 512)
        const float g = gm[2 * lane], h = gm[2 * lane + 1];
        const float tau = a.k <= 24 ? wave_kth(fmaxf(g, h), a.k) : wave_kth(g, h, a.k);
        if (lane == 0)
            tau_row = tau;
    }
    if (wave == 0) {
        // the streams' sums joined, a lane each
        Stat z = {-INFINITY, 0.0f, 0.0f};
        if (lane < kStreams)
            z = {st[lane][0], st[lane][1], st[lane][2]};
        const float m = wave_max(z.m);
        if (m > z.m)
            z.raise(m);
        z = {m, lane63(wave_scan_inclusive(z.s)), lane63(wave_scan_inclusive(z.u))};
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
    int32_t *ids = a.top_ids + t * a.k;
    float *lps = a.top_logprobs + t * a.k;
    if (fin[2] != 0.0f) {   // no distribution
        for (int i = threadIdx.x; i < a.k; i += 64 * NW) {
            ids[i] = -1;
            lps[i] = __uint_as_float(0x7fc00000u);
        }
        return;
    }
    // the segments that reach the bound
    const float tau = tau_row;
    const int ords = (ord + R - 1) / R;
    for (int o = 0; o < ords; ++o) {
        const float s = smax[(wave * ORD + o) * 64 + lane];
        const uint64_t m = __ballot(s >= tau && s > -INFINITY);
        if (m) {
            const int at = append_at(m, &count[0]);
            if (((m >> lane) & 1) && at < kSegs)
                few[at] = (uint16_t)((wave * ORD + o) * 64 + lane);
        }
    }
    __syncthreads();
    const int nsegs = count[0];
    if (nsegs <= kSegs) {
        // a wave reads two segments at a time: lane l element l % 32 of one
        for (int p = 2 * wave; p < nsegs; p += 2 * NW) {
            const int at = p + (lane >> 5);
            const uint32_t id = at < nsegs ? few[at] : 0;
            const int w = (int)(id >> 6) / ORD, o = (int)(id >> 6) % ORD, l = (int)(id & 63);
            const int j = lane & 31;
            // the wave's chunk number n is chunk n % per of its stream n / per
            for (int r = 0; r < R; ++r) {
                int n = o * R + r, sw = w;
                // (streams end at different chunks)
                for (;;) {
                    const int per = sw < nchunks ? (nchunks - sw + kStreams - 1) / kStreams : 0;
                    if (n < per || sw >= kStreams)
                        break;
                    n -= per;
                    sw += NW;
                }
                const int64_t i = (int64_t)(sw + n * kStreams) * kChunkElems +
                                  (64 * (j / E) + l) * E + j % E;
                const bool in = at < nsegs && sw < kStreams && i < V;
                const float x = in ? IO::ld(row, i) : -INFINITY;
                const uint64_t m = __ballot(x >= tau && x > -INFINITY);
                if (m) {
                    const int to = append_at(m, &count[1]);
                    if (((m >> lane) & 1) && to < kCands)
                        cand[to] = key_of(x, (int)i);
                }
            }
        }
    }
    __syncthreads();
    const int n = count[1];
    if (nsegs <= kSegs && n <= kCands) {
        for (int i = threadIdx.x; i < n; i += 64 * NW) {
            const uint64_t me = cand[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j)
                rank += cand[j] > me;
            if (rank < a.k) {
                ids[rank] = key_index(me);
                lps[rank] = key_value(me) - fin[0] - fin[1];
            }
        }
        // Fewer than top_k unmasked: all of them are candidates, and the lowest
        // masked indices follow. Index i < 2 k is masked when it is no candidate,
        // and its place is n + i - (candidates below i).
        if (n < a.k)
            for (int i = threadIdx.x; i < 2 * a.k && i < V; i += 64 * NW) {
                int below = 0;
                bool listed = false;
                for (int j = 0; j < n; ++j) {
                    const int o = key_index(cand[j]);
                    below += o < i;
                    listed |= o == i;
                }
                const int place = n + i - below;
                if (!listed && place < a.k) {
                    ids[place] = i;
                    lps[place] = -INFINITY;
                }
            }
        return;
    }

    // Too many for the lists (at least top_k elements are unmasked then): every
    // wave reads its chunks once more, one element a lane at a time.
    TopList<LIST> top = {reinterpret_cast<uint64_t *>(smax) + wave * LIST, 0, a.k, tau, INT32_MAX};
    for (int sw = wave; sw < kStreams; sw += NW)
        for (int ch = sw; ch < nchunks; ch += kStreams)
#pragma unroll 1
            for (int e = 0; e < kPerLane; ++e) {
                const int64_t i = (int64_t)ch * kChunkElems + (64 * (e / E) + lane) * E + e % E;
                const float x = i < V ? IO::ld(row, i) : -INFINITY;
                uint64_t m = __ballot(x > -INFINITY && top.ahead(x, (int)i));
                if (top.n + __popcll(m) > LIST) {
                    top.cut();
                    m = __ballot(x > -INFINITY && top.ahead(x, (int)i));
                }
                if (m)
                    top.append(m, x, (int)i);
            }
    top.cut();
    if (lane == 0)
        ln[wave] = top.n;
    __syncthreads();
    // Join the waves' sorted lists: an element's place is its place in its own
    // list plus the elements ahead of it in the others.
    const uint64_t *keys = reinterpret_cast<const uint64_t *>(smax);
    if (lane < ln[wave]) {
        const uint64_t me = keys[wave * LIST + lane];
        int rank = lane;
        for (int w = 0; w < NW; ++w) {
            if (w == wave)
                continue;
            int lo = 0, hi = ln[w];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (keys[w * LIST + mid] > me)
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
}

template <class IO>
hipError_t logprobs_impl(const LogprobArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)a.T);
    if (logprob_waves(a.T, a.V, sizeof(typename IO::T) == 2) == 16) {
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
