// ssd_pages.hip -- pages and slots of the exact-replay cache: handing pages
// out, taking them back, copying slots, squeezing the pool.
//
// The page table is the only record of who holds which page, so the two
// calls that need to know the free pages (reserve, compact) build a bitmap of
// the used ones from it, in the LDS of one 1024-thread workgroup: one bit a
// page, set with LDS atomic ORs (their order does not change the bits), then
// a prefix sum of the free counts finds the r-th free page by search. That
// keeps the answer a pure function of the table (lowest page first), with no
// free list that could disagree with it, and a table of 8192 entries is
// 32 KB, read once.
// That plan is latency, not bytes: 512 slots of 16 pages take 5.9 us (the table's
// one round trip beside the requests', the bits, two prefix sums, the search); with the
// requests' rows read an entry at a time, and before the table, 8.7; 128 requests that
// take 320 pages of a pool of 647, 7.0-7.7.
// The copies move whole 16-byte pieces, eight loads in flight per thread
// before the first store: 16 slots forked into 128 (272 MB written, 34 MB read) in
// 54-58 us, 5.3-5.7 TB/s, where a fill of that size takes 40; 71 MB of pages moved in
// 23-25 us, 5.6-6.2 TB/s of both directions.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssd_device.hpp"
#include "ssd_step.hpp"

namespace ssd {
namespace {

constexpr int kPlan = 1024;        // threads of the planning workgroup
constexpr int kCopy = 256;         // threads of the copying workgroups
constexpr int kPiece = 32768;      // bytes of state that one workgroup moves: eight
                                   // 16-byte pieces a thread, all in flight at once
constexpr int kRowGroup = 16;      // buffered rows that one workgroup moves (a page
                                   // holds a multiple of 16 rows)

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- copying ----------------------------------------------------------------

// n16 16-byte pieces, by the whole workgroup: eight loads in flight per thread
// before the first store. go() is asked between the first loads and the first
// store, so that what it waits for and the data are under way together; without
// it nothing is stored.
template <class Go>
__device__ __forceinline__ void copy16(void *dst, const void *src, int64_t n16, Go go) {
    constexpr int B = 8;
    u32x4 *d = static_cast<u32x4 *>(dst);
    const u32x4 *s = static_cast<const u32x4 *>(src);
    bool asked = false;
    for (int64_t base = 0; base < n16; base += B * kCopy) {
        const int64_t e0 = base + threadIdx.x;
        u32x4 v[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int64_t e = e0 + i * kCopy;
            v[i] = s[e < n16 ? e : n16 - 1];
        }
        if (!asked) {
            if (!go())
                return;
            asked = true;
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int64_t e = e0 + i * kCopy;
            if (e < n16)
                __builtin_nontemporal_store(v[i], d + e);
        }
    }
}
__device__ __forceinline__ void copy16(void *dst, const void *src, int64_t n16) {
    copy16(dst, src, n16, [] { return true; });
}

// n 2-byte elements (raw dt rows, whose arrays have natural alignment only).
__device__ __forceinline__ void copy2(void *dst, const void *src, int n) {
    uint16_t *d = static_cast<uint16_t *>(dst);
    const uint16_t *s = static_cast<const uint16_t *>(src);
    for (int e = threadIdx.x; e < n; e += kCopy)
        d[e] = s[e];
}

// Row of the buffers that holds position pos (a multiple of 16) of a slot.
__device__ __forceinline__ int64_t pool_row(const SlotMap &c, int slot, int pos) {
    if (!c.pages)
        return (int64_t)slot * c.Q + pos;
    const int page = c.pages[(int64_t)slot * c.npp + (pos >> c.shift)];
    return ((int64_t)page << c.shift) + (pos & ((1 << c.shift) - 1));
}

__device__ __forceinline__ bool page_ok(const SlotMap &c, int page) {
    return page >= 0 && page < c.num_pages;
}

// Whether the first n positions of a slot have pages.
__device__ __forceinline__ bool rows_ok(const SlotMap &c, int slot, int n) {
    if (!c.pages)
        return true;
    const int np = (n + (1 << c.shift) - 1) >> c.shift;
    bool bad = false;
    if ((int)threadIdx.x < np)   // at most Q / 16 = 16 pages
        bad = !page_ok(c, c.pages[(int64_t)slot * c.npp + threadIdx.x]);
    return !__syncthreads_or(bad);
}

// grid (n, parts): parts [0, ns) pieces of the state, [ns, ns + nb) of its
// bf16 copy, the rest 16 buffered rows each. The list runs along x, so that
// the copies of one source (a fork) read it at the same time.
__global__ __launch_bounds__(kCopy) void k_cache_copy(CopyArgs a, int ns, int nb) {
    // every XCD takes a run of entries: the copies of one source read it
    // through one L2
    const int b = (int)(blockIdx.x & 7) * (int)(gridDim.x >> 3) + (int)(blockIdx.x >> 3);
    int part = blockIdx.y;
    if (b >= a.n)
        return;
    const int d = a.dst_idx[b], s = a.src_idx[b];
    const bool in = d >= 0 && d < a.dst.num_slots && s >= 0 && s < a.src.num_slots;
    const bool same = in && a.dst.state == a.src.state && d == s;
    if (!in || same) {
        if (part == 0 && threadIdx.x == 0 && a.copied)
            a.copied[b] = same;
        return;
    }
    const int len = a.src.buf_len[s];
    const auto ok = [&] {
        return len >= 0 && len < a.src.Q && rows_ok(a.src, s, len) && rows_ok(a.dst, d, len);
    };
    if (part < ns + nb) {
        // [0, ns): fp32 state, [ns, ns + nb): the bf16 copy
        const bool bf = part >= ns;
        const int64_t size = bf ? a.r.state / 2 : a.r.state;
        const int64_t at = (int64_t)(bf ? part - ns : part) * kPiece;
        const char *src = bf ? static_cast<const char *>(a.src.state_bf)
                             : reinterpret_cast<const char *>(a.src.state);
        char *dst = bf ? static_cast<char *>(a.dst.state_bf)
                       : reinterpret_cast<char *>(a.dst.state);
        const int64_t n = size - at < kPiece ? size - at : kPiece;
        copy16(dst + d * size + at, src + s * size + at, n / 16, [&] {
            const bool go = ok();
            if (part == 0 && threadIdx.x == 0) {
                if (a.copied)
                    a.copied[b] = go;
                if (go) {
                    a.dst.buf_len[d] = len;
                    a.dst.boundary_pos[d] = a.src.boundary_pos[s];
                }
            }
            return go;
        });
        return;
    }
    if (!ok())
        return;
    part -= ns + nb;
    const int pos = part * kRowGroup;
    if (pos >= len)
        return;
    const int rows = len - pos < kRowGroup ? len - pos : kRowGroup;
    const int64_t rs = pool_row(a.src, s, pos), rd = pool_row(a.dst, d, pos);
    const auto at = [](void *p, int64_t byte) { return static_cast<char *>(p) + byte; };
    copy16(at(a.dst.buf_x, rd * a.r.x), at(a.src.buf_x, rs * a.r.x), (int64_t)rows * a.r.x / 16);
    copy16(at(a.dst.buf_B, rd * a.r.bc), at(a.src.buf_B, rs * a.r.bc),
           (int64_t)rows * a.r.bc / 16);
    if (a.dst.buf_C)
        copy16(at(a.dst.buf_C, rd * a.r.bc), at(a.src.buf_C, rs * a.r.bc),
               (int64_t)rows * a.r.bc / 16);
    copy2(at(a.dst.buf_dt, rd * a.r.dt), at(a.src.buf_dt, rs * a.r.dt), rows * a.r.dt / 2);
}

// grid (n, parts): zeros, and part 0 resets the slot's metadata and table row.
__global__ __launch_bounds__(kCopy) void k_cache_free(SlotMap c, RowBytes r, int n,
                                                      const int32_t *slot_idx, int ns) {
    const int b = blockIdx.x, part = blockIdx.y;
    const int s = slot_idx ? slot_idx[b] : b;
    if (s < 0 || s >= c.num_slots)
        return;
    if (part == 0) {
        if (c.pages)
            for (int i = threadIdx.x; i < c.npp; i += kCopy)
                c.pages[(int64_t)s * c.npp + i] = -1;
        if (threadIdx.x == 0) {
            c.buf_len[s] = 0;
            c.boundary_pos[s] = 0;
        }
    }
    const bool bf = part >= ns;
    const int64_t size = bf ? r.state / 2 : r.state;
    const int64_t at = (int64_t)(bf ? part - ns : part) * kPiece;
    char *dst = (bf ? static_cast<char *>(c.state_bf) : reinterpret_cast<char *>(c.state)) +
                s * size + at;
    const int64_t n16 = (size - at < kPiece ? size - at : kPiece) / 16;
    const u32x4 zero = {0, 0, 0, 0};
    for (int64_t e = threadIdx.x; e < n16; e += kCopy)
        reinterpret_cast<u32x4 *>(dst)[e] = zero;
}

__global__ __launch_bounds__(256) void k_pages_trim(SlotMap c, int n, const int32_t *slot_idx) {
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;   // n npp < 2^31
    const int b = (int)(i / (uint32_t)c.npp), e = (int)(i % (uint32_t)c.npp);
    if (b >= n)
        return;
    const int s = slot_idx ? slot_idx[b] : b;
    if (s < 0 || s >= c.num_slots)
        return;
    const int len = c.buf_len[s];
    if (len >= 0 && ((int64_t)e << c.shift) >= len)
        c.pages[(int64_t)s * c.npp + e] = -1;
}

// ---- planning ---------------------------------------------------------------

// Exclusive prefix sum over the workgroup of kPlan threads, of counts whose total is
// below 2^24 (exact in fp32, for the DPP scan); *total gets the sum. red: 16 ints of
// LDS, free on entry and on return.
__device__ __forceinline__ int block_exclusive(int v, int *red, int *total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int x = (int)wave_scan_inclusive((float)v);
    if (lane == 63)
        red[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlan / 64; ++w) {
        const int t = red[w];
        before += w < wave ? t : 0;
        all += t;
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// Place of the r-th set bit of the words word(0), word(1), .., of which thread t
// owns the `per` words from t per on and before[t] bits lie below: a search for
// the owner, a walk over its words, a binary search in the word.
template <class Word>
__device__ __forceinline__ int nth_bit(const int32_t *before, int r, int per, Word word) {
    int lo = 0, hi = kPlan - 1;   // last thread whose before[] is <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    r -= before[lo];
    int w = lo * per;
    uint32_t f = word(w);
    for (int k; r >= (k = __popc(f)); f = word(++w))
        r -= k;
    int at = 0;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const int k = __popc(f & ((1u << s) - 1u));
        if (r >= k) {
            r -= k;
            f >>= s;
            at += s;
        }
    }
    return w * 32 + at;
}

// The used pages as a bitmap in LDS, and the free ones by rank.
struct PageBits {
    uint32_t *bits;       // [words], a set bit is a used page
    int32_t *first;       // [kPlan]: free pages below thread t's words
    int words, per, num_pages, nfree;
    int head[8];          // the thread's first eight table entries

    // table entries i0, i0 + kPlan, ..; -1 past the end
    __device__ static __forceinline__ void load(const SlotMap &c, int64_t i0, int (&p)[8]) {
        const int64_t n = (int64_t)c.num_slots * c.npp;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            p[k] = i0 + k * kPlan < n ? c.pages[i0 + k * kPlan] : -1;
    }
    __device__ __forceinline__ void mark(const SlotMap &c, const int (&p)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (page_ok(c, p[k]))
                atomicOr(&bits[p[k] >> 5], 1u << (p[k] & 31));
    }
    // pages that exist in word w
    __device__ uint32_t valid(int w) const {
        const int left = num_pages - w * 32;
        return left >= 32 ? 0xffffffffu : (1u << left) - 1u;
    }
    __device__ PageBits(const SlotMap &c, uint32_t *bits_, int32_t *first_, int *red)
        : bits(bits_), first(first_), num_pages(c.num_pages) {
        words = (num_pages + 31) / 32;
        per = (words + kPlan - 1) / kPlan;
        // (eight entries a thread in flight, the first eight while the bits are
        // cleared: the table's latency, not its size, is what this costs)
        load(c, threadIdx.x, head);
        for (int w = threadIdx.x; w < words; w += kPlan)
            bits[w] = 0;
        __syncthreads();
        mark(c, head);
        const int64_t n = (int64_t)c.num_slots * c.npp;
        for (int64_t i0 = threadIdx.x + 8 * kPlan; i0 < n; i0 += 8 * kPlan) {
            int p[8];
            load(c, i0, p);
            mark(c, p);
        }
        __syncthreads();
        const int w0 = threadIdx.x * per, w1 = min(w0 + per, words);
        int free = 0;
        for (int w = w0; w < w1; ++w)
            free += __popc(~bits[w] & valid(w));
        first[threadIdx.x] = block_exclusive(free, red, &nfree);
        __syncthreads();
    }
    // the r-th free page, 0 <= r < nfree
    __device__ __forceinline__ int free_page(int r) const {
        return nth_bit(first, r, per, [&](int w) { return ~bits[w] & valid(w); });
    }
};

// A request: its slot (-1: skipped), and its table row, its length and its tokens as
// loaded. (A slot has 1, 2, 4, 8 or 16 pages; the row is fetched in 16-byte pieces,
// since 64 lanes read 64 rows.)
struct Request {
    int slot, len, tok;
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    i32x4 e[kMaxQ / 64];
    __device__ __forceinline__ Request(const ReserveArgs &a, int b)
        : slot(-1), len(0), tok(0), e{} {
        typedef i32x4 i32x4_u __attribute__((aligned(4)));
        const SlotMap &c = a.c;
        if (b >= a.n)
            return;
        const int s = a.slot_idx ? a.slot_idx[b] : b;
        const int like = a.like_idx ? a.like_idx[b] : s;
        if (s < 0 || s >= c.num_slots || like < 0 || like >= c.num_slots)
            return;
        const int32_t *row = c.pages + (int64_t)s * c.npp;
        if (c.npp >= 4) {
#pragma unroll
            for (int i = 0; i < kMaxQ / 64; ++i)
                e[i] = *reinterpret_cast<const i32x4_u *>(row + (4 * i < c.npp ? 4 * i : 0));
        } else {
            e[0] = (i32x4){row[0], row[c.npp - 1], -1, -1};
        }
        slot = s;
        len = c.buf_len[like];
        tok = a.tokens ? a.tokens[b] : a.tokens_all;
    }
    // The pages that its tokens span and that it lacks, as a bit mask; a slot that
    // cannot be served becomes -1.
    __device__ __forceinline__ int lack(const SlotMap &c) {
        if (slot < 0 || len < 0 || len >= c.Q) {
            slot = -1;
            return 0;
        }
        const int t = min(max(tok, 0), c.Q);
        const int pages = (min(len + t, c.Q) + (1 << c.shift) - 1) >> c.shift;
        int m = 0;
#pragma unroll
        for (int i = 0; i < kMaxQ / 16; ++i)
            if (i < pages && !page_ok(c, e[i / 4][i % 4]))
                m |= 1 << i;
        return m;
    }
};

__global__ __launch_bounds__(kPlan) void k_pages_reserve(ReserveArgs a) {
    extern __shared__ uint32_t bits[];
    __shared__ int32_t first[kPlan];
    __shared__ int red[kPlan / 64];
    const SlotMap c = a.c;
    // (the first requests' loads run beside the table's)
    Request q(a, threadIdx.x);
    const PageBits pb(c, bits, first, red);
    int asked = 0;   // pages asked for by the entries before this batch
    for (int b0 = 0; b0 < a.n; b0 += kPlan) {
        const int b = b0 + threadIdx.x;
        if (b0 > 0)
            q = Request(a, b);
        const int lack = q.lack(c);
        const int need = __popc(lack);
        int total;
        int r = asked + block_exclusive(need, red, &total);
        asked += total;
        const bool served = q.slot >= 0 && (need == 0 || r + need <= pb.nfree);
        if (served) {
            int32_t *row = c.pages + (int64_t)q.slot * c.npp;
            for (int m = lack; m; m &= m - 1)
                row[__ffs(m) - 1] = pb.free_page(r++);
        }
        if (b < a.n && a.granted)
            a.granted[b] = served;
    }
}

__global__ __launch_bounds__(kPlan) void k_compact_plan(SlotMap c, int32_t *used, int32_t *work) {
    extern __shared__ uint32_t bits[];
    __shared__ int32_t first[kPlan], high[kPlan];
    __shared__ int red[kPlan / 64];
    const PageBits pb(c, bits, first, red);
    const int U = c.num_pages - pb.nfree;
    // used bits of word w at or past page U
    const auto movers = [&](int w) {
        const int below = U - w * 32;
        return below >= 32 ? 0u : (below <= 0 ? bits[w] : bits[w] & ~((1u << below) - 1u));
    };
    const int w0 = threadIdx.x * pb.per, w1 = min(w0 + pb.per, pb.words);
    int mine = 0, moves;
    for (int w = w0; w < w1; ++w)
        mine += __popc(movers(w));
    high[threadIdx.x] = block_exclusive(mine, red, &moves);
    if (threadIdx.x == 0) {
        used[0] = U;
        work[0] = moves;
    }
    __syncthreads();
    // the j-th mover goes to the j-th free page; a thread each
    for (int j = threadIdx.x; j < moves; j += kPlan) {
        work[2 + 2 * j] = nth_bit(high, j, pb.per, movers);
        work[3 + 2 * j] = pb.free_page(j);
    }
    const int64_t n = (int64_t)c.num_slots * c.npp;
    int e[8];
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += 8 * kPlan) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            e[k] = pb.head[k];
        if (i0 >= 8 * kPlan)
            PageBits::load(c, i0, e);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int p = e[k];
            if (!page_ok(c, p) || p < U)
                continue;
            const int w = p >> 5, t = w / pb.per;
            int rank = high[t];
            for (int v = t * pb.per; v < w; ++v)
                rank += __popc(movers(v));
            rank += __popc(movers(w) & ((1u << (p & 31)) - 1u));
            c.pages[i0 + k * kPlan] = pb.free_page(rank);
        }
    }
}

// The listed moves, each page in pieces dealt to the workgroups in turn.
// The targets are pages that nothing reads, so the order does not matter.
__global__ __launch_bounds__(kCopy) void k_compact_move(SlotMap c, RowBytes r,
                                                        const int32_t *work) {
    const int moves = work[0], pt = 1 << c.shift;
    const int groups = pt / kRowGroup;
    const int64_t items = (int64_t)moves * groups;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int j = (int)(it / groups), g = (int)(it % groups);
        const int64_t rs = ((int64_t)work[2 + 2 * j] << c.shift) + g * kRowGroup;
        const int64_t rd = ((int64_t)work[3 + 2 * j] << c.shift) + g * kRowGroup;
        const auto at = [](void *p, int64_t byte) { return static_cast<char *>(p) + byte; };
        copy16(at(c.buf_x, rd * r.x), at(c.buf_x, rs * r.x), (int64_t)kRowGroup * r.x / 16);
        copy16(at(c.buf_B, rd * r.bc), at(c.buf_B, rs * r.bc), (int64_t)kRowGroup * r.bc / 16);
        if (c.buf_C)
            copy16(at(c.buf_C, rd * r.bc), at(c.buf_C, rs * r.bc),
                   (int64_t)kRowGroup * r.bc / 16);
        copy2(at(c.buf_dt, rd * r.dt), at(c.buf_dt, rs * r.dt), kRowGroup * r.dt / 2);
    }
}

// LDS bytes of the bitmap; above 64 KB (more than 524288 pages) the kernel
// has to ask for them.
template <class K>
hipError_t bitmap_bytes(K kernel, int num_pages, size_t *bytes) {
    *bytes = ((size_t)num_pages + 31) / 32 * sizeof(uint32_t);
    if (*bytes <= 48 * 1024)
        return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)*bytes);
}

int pieces(int64_t bytes) { return (int)((bytes + kPiece - 1) / kPiece); }

}  // namespace

hipError_t launch_pages_reserve(const ReserveArgs &a, hipStream_t stream) {
    size_t lds;
    const hipError_t e = bitmap_bytes(k_pages_reserve, a.c.num_pages, &lds);
    if (e != hipSuccess)
        return e;
    k_pages_reserve<<<dim3(1), dim3(kPlan), lds, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_pages_trim(const SlotMap &c, int32_t n, const int32_t *slot_idx,
                             hipStream_t stream) {
    const int64_t threads = (int64_t)n * c.npp;
    k_pages_trim<<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream>>>(c, n,
                                                                                   slot_idx);
    return hipGetLastError();
}

hipError_t launch_cache_free(const SlotMap &c, const RowBytes &r, int32_t n,
                             const int32_t *slot_idx, hipStream_t stream) {
    const int ns = pieces(r.state), nb = pieces(r.state / 2);
    k_cache_free<<<dim3(n, ns + nb), dim3(kCopy), 0, stream>>>(c, r, n, slot_idx, ns);
    return hipGetLastError();
}

hipError_t launch_cache_copy(const CopyArgs &a, hipStream_t stream) {
    const int ns = pieces(a.r.state), nb = pieces(a.r.state / 2);
    const int parts = ns + nb + a.src.Q / kRowGroup;
    k_cache_copy<<<dim3((a.n + 7u) / 8u * 8u, parts), dim3(kCopy), 0, stream>>>(a, ns, nb);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const SlotMap &c, const RowBytes &r, int32_t *used, int32_t *work,
                                hipStream_t stream) {
    size_t lds;
    hipError_t e = bitmap_bytes(k_compact_plan, c.num_pages, &lds);
    if (e != hipSuccess)
        return e;
    k_compact_plan<<<dim3(1), dim3(kPlan), lds, stream>>>(c, used, work);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    // at most half of the pages move; 2048 workgroups fill the device
    const int64_t most = (int64_t)(c.num_pages / 2) * ((1 << c.shift) / kRowGroup);
    if (most == 0)
        return hipSuccess;
    k_compact_move<<<dim3((unsigned)std::min<int64_t>(most, 2048)), dim3(kCopy), 0, stream>>>(
        c, r, work);
    return hipGetLastError();
}

}  // namespace ssd
