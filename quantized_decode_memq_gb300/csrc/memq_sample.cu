// memq_sample.cu -- memq_sample: one token a row of logits, from a given random number.
//
//   w_i = exp((l_i - max) / T), tokens in descending order of l, equal ones by index
//   top-k: the first k;  top-p: of those the shortest prefix with at least p of their weight;
//   min-p: of those the ones with w_i >= min_p;  then, in the order of indices, the first token whose
//   cumulative weight is above u times the total.
//
// What is kept is always a prefix of the order, so no row is sorted: a cut (a key and, among equal ones, an
// index) is found, and the draw runs over the kept tokens by index.
//
// A draw and a cut compare sums with a border, and with 1e5 tokens some border is near, so weights are formed to
// about 2^-41 and summed as 64-bit integers in units of 2^-44: sums do not depend on their order, and a token's
// probability is exact to 2^-41 of the largest one's.  (l - max) / T is a pair of f32, 2^-x a table of 512 powers
// times a polynomial, both in integers; below 2^-24 of the largest the hardware's exp2 is exact enough.
//
// A cluster of CTAs keeps a row in shared memory, so it is read once; the number of CTAs is chosen to fill
// the GPU with few rows and to let two CTAs share an SM with many.  Then, by what the row asks for:
//   greedy          the first of the largest
//   small top-k     The k-th largest of all is not below t if every one of the C CTAs has ceil(k / C) threads whose
//                   largest is t or more; what is t or more (usually little over k) is gathered and sorted by one CTA.
//   other top-k     The tokens are counted by steps of 1 / 25 of x = log2 of the largest's ratio, so the step that
//                   holds the cut is known; its tokens are gathered and sorted (finer steps when they are many).
//   top-p           The same with weights, added exactly, in 1536 steps of 1 / 64 (24 octaves).
//   then            One pass of weights over what is kept, the draw from the warps' sums; behind top-p, by the one CTA
//                   whose steps' sum holds the drawn place.
// bf16 logits have few values: top-p counts them and weighs each once, the draw looks them up (256 rows of 131072 169 us
// -> 111, f32 as before; from 8192 tokens a CTA, 256 rows of 16384 with top-p 55 -> 37, 4000 tokens a CTA gain nothing).
// Rows that defeat this are cut by bisection over keys, then over indices: thousands of equal logits at the cut, and a
// top-p that ends among weights below 2^-24 (which have no steps), as near 1 it does in steep rows and flat ones.
//
// us by what all rows ask for, greedy / top-k 50 / no cut / top-p 0.9:  1 x 32000 f32 3.5 / 8.7 / 7.4 / 23;  8 x 128259 f32
// 5.0 / 12 / 17 / 42;  256 x 131072 bf16 28 / 59 / 99 / 187, f32 49 / 89 / 156 / 343;  256 x 16384 bf16 with top-k 500 31.
// Top-p 0.999 with the cut behind the steps in some rows: 8 x 128259 355, 256 x 131072 bf16 1120, f32 880; in all rows (one
// token far above the others) 199, 1930 and 2370: bisection forms every weight up to 32 times.
// What bounds it: the load alone is 0.8 (256 x 131072 bf16, greedy: 2.4 TB/s, a CTA loads and then works), the exact weights 60
// instructions a token and pass (f32), counting 11 cycles a warp and token (shared atomics); of few rows, latency: eight
// cluster barriers of 1200 cycles, the sort by one CTA 7000 (8 x 128259: 80000 cycles, 37000 of them in the two passes).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>

#include "memq.h"
#include "memq_dev.cuh"
#include "memq_tc.cuh"

namespace memq {
namespace {

constexpr int kMaxWarps = 32;  // of a CTA: 512 threads, or 1024
constexpr int kMaxCtas = 8;
constexpr int kCap = 2048;   // tokens that are sorted
constexpr int kBins = 1536, kPerOctave = 64;  // steps of x, up to kCareful for weights
constexpr int kCountOctave = 25;              // and up to 60 for numbers of tokens
constexpr int kTable = 512;
constexpr int kUnitLog = 44;  // weights are integers in units of 2^-44
constexpr uint32_t kLeastKey = 0x007fffffu;  // of -infinity; NaN has key 0
constexpr int64_t kMaxVocab = 360000;
// bf16 logits: a table of the weights of ten binades of values, of either sign.
constexpr uint32_t kHalf = 10 * 128, kValues = 2 * kHalf;
constexpr int kTabled = 8192;  // tokens of a CTA from which it pays

// 2^(-j / 512) in units of 2^-62, formed by the compiler: the 512th root of 1/2 by nine square roots, then its powers.
struct Powers {
    unsigned long long at[kTable];
};
constexpr unsigned long long root_of(unsigned __int128 x) {  // floor of the square root
    unsigned __int128 r = 0;
    for (int b = 63; b >= 0; --b) {
        const unsigned __int128 t = r | (static_cast<unsigned __int128>(1) << b);
        if (t * t <= x) r = t;
    }
    return static_cast<unsigned long long>(r);
}
constexpr Powers make_powers() {
    Powers p{};
    unsigned long long step = 1ull << 62;  // 2^-1 in units of 2^-63
    for (int i = 0; i < 9; ++i) step = root_of(static_cast<unsigned __int128>(step) << 63);
    unsigned long long run = 1ull << 63;
    for (int j = 0; j < kTable; ++j) {
        p.at[j] = (run >> 1) + (run & 1);
        const unsigned __int128 next = static_cast<unsigned __int128>(run) * step;
        run = static_cast<unsigned long long>((next + (static_cast<unsigned __int128>(1) << 62)) >> 63);
    }
    return p;
}
__device__ const Powers g_powers = make_powers();

struct SampleArgs {
    const void *logits;
    int64_t stride;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *out;
    int vocab, slice;  // tokens of a row, of a CTA
};

struct __align__(16) Shared {
    unsigned long long table[kTable];           // g_powers
    union {
        struct {
            unsigned long long list[kCap];      // tokens: key << 32 | ~index; sorted, largest first
            unsigned long long weight[kCap];    // of the list
        };
        struct {
            union {
                unsigned long long value[kValues];  // bf16 values' weights
                uint32_t times[2 * kValues];        // and how often they are there
            };
            uint32_t lo[kBins], hi[kBins];      // weight of the steps of x
        } steps;
    };
    unsigned long long sums[kMaxCtas][kMaxWarps];  // of every CTA's warps
    unsigned long long pair[kMaxCtas][2];
    unsigned long long partial[kMaxCtas];       // weight of what every CTA keeps of the step that holds the cut
    unsigned long long warp64[2][kMaxWarps];
    unsigned long long cut;      // place of the last token that is kept
    unsigned long long before;   // weight ahead of the step that holds the cut
    uint32_t from_cta[kMaxCtas], bounds[kMaxCtas];
    uint32_t warp32[kMaxWarps];
    uint32_t count;              // tokens in the first CTA's list
    uint32_t found;
    int step;
};

// ------------------------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cta_count() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Nothing is stored to another CTA before it has begun.
__device__ __forceinline__ void cluster_arrive_entry() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_entry() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of `p` in CTA `rank`'s shared memory.
template <typename T>
__device__ __forceinline__ T *in_cta(T *p, uint32_t rank) {
    uint64_t r;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<T *>(r);
}

// ------------------------------------------------------------------------------ weights
struct Scale {
    float top;     // the largest logit
    float hi, lo;  // log2(e) / T
};

// x = (top - l) log2(e) / T, rounded to f32: monotone in l, so its steps are ranges of the order.
__device__ __forceinline__ float coarse(const Scale &s, float l) { return l == s.top ? 0.f : (s.top - l) * s.hi; }

// 2^-x of x >= kCareful: x is off by 2^-24 of it and exp2 by 2^-22 of it, below 2^-42 together.
constexpr float kCareful = 24.f;
__device__ __forceinline__ unsigned long long small_weight(float x) {  // 0 of 60 and more
    return x < 60.f ? static_cast<unsigned long long>(__float2uint_rn(ex2(static_cast<float>(kUnitLog) - x))) : 0ull;
}

// 2^-x in units of 2^-kUnitLog.
__device__ __forceinline__ unsigned long long careful_weight(const Scale &s, const unsigned long long *table, float l) {
    // the difference, exactly: dh + dl
    const float dh = __fsub_rn(s.top, l), bb = __fsub_rn(dh, s.top);
    const float dl = __fsub_rn(__fsub_rn(s.top, __fsub_rn(dh, bb)), __fadd_rn(l, bb));
    const float yh = fminf(__fmul_rn(dh, s.hi), kCareful);  // (of a larger one the result is not used)
    const float yl = __fmaf_rn(dh, s.hi, -yh) + __fmaf_rn(dh, s.lo, dl * s.hi);
    // the nearest multiple n of 2^-9
    const float big = 0x1.8p23f / kTable;
    const float t = __fadd_rn(yh, big);
    const int n = __float_as_int(t) - __float_as_int(big);
    const float rh = __fsub_rn(yh, __fsub_rn(t, big));
    // r = rh + yl as a pair
    const float r = __fadd_rn(rh, yl), rb = __fsub_rn(r, rh);
    const float rl = __fadd_rn(__fsub_rn(rh, __fsub_rn(r, rb)), __fsub_rn(yl, rb));
    // z = r ln 2, |z| < 2^-10.5; 1 - 2^-r = z - z^2/2 + z^3/6 - z^4/24
    const float kLn2 = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
    const float zh = __fmul_rn(r, kLn2);
    const float zl = __fmaf_rn(r, kLn2, -zh) + __fmaf_rn(r, kLn2Lo, rl * kLn2);
    const float q = zh * zh * __fmaf_rn(zh, __fmaf_rn(zh, 1.f / 24.f, -1.f / 6.f), 0.5f);
    const int a = __float2int_rn(zh * 0x1p41f) + __float2int_rn((zl - q) * 0x1p41f);  // below 2^30.6
    const int j = n & (kTable - 1), e = n >> 9;
    const unsigned long long p = table[j];
    const long long down = static_cast<long long>(static_cast<int>((p + 0x80000000ull) >> 32)) * a >> 9;
    const unsigned long long w = p - static_cast<unsigned long long>(down);
    const int shift = 62 - kUnitLog + e;
    return l == s.top ? 1ull << kUnitLog : (w + (1ull << (shift - 1))) >> shift;  // (infinity less itself is no number)
}
__device__ __forceinline__ unsigned long long weight_of(const Scale &s, const unsigned long long *table, float l) {
    const float x = coarse(s, l);
    return x < kCareful ? careful_weight(s, table, l) : small_weight(x);
}
// The weights of N tokens: a warp's lanes take the longer way together, all at once, if one of them has to.
template <int N>
__device__ __forceinline__ void weights_of(const Scale &s, const unsigned long long *table, const float (&l)[N],
                                           const float (&x)[N], unsigned long long (&w)[N]) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        w[j] = small_weight(x[j]);
        any = any || x[j] < kCareful;
    }
    if (__any_sync(kFullMask, any)) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned long long c = careful_weight(s, table, l[j]);
            if (x[j] < kCareful) w[j] = c;
        }
    }
}

// Few bf16 numbers lie between the largest logit and 24 octaves of weight below it: a table of them starts at
// the least magnitude, as bits, of `binades` up to the largest of any logit there.
__device__ __forceinline__ uint32_t table_base(const Scale &s, int binades) {
    const float far = fmaxf(fabsf(s.top), fabsf(s.top - __fdiv_rn(kCareful, s.hi)));
    return static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(far) >> 23) - (binades - 1), 0)) << 7;
}
// Of logits up to `after` and weights below `least` the entries are without weight.
template <int T>
__device__ __forceinline__ void make_values(const Scale &s, Shared &sh, uint32_t base, float after, unsigned long long least) {
    for (uint32_t i = threadIdx.x; i < kValues; i += T) {
        const uint32_t sign = i >= kHalf, bits = sign << 31 | (base + i - sign * kHalf) << 16;
        const float l = __uint_as_float(bits) + 0.f;
        unsigned long long e = l > s.top || l <= after ? 0ull : weight_of(s, sh.table, l);  // (none is above)
        sh.steps.value[i] = e < least ? 0ull : e;
    }
    __syncthreads();
}
// The sum of the weights of a group of tokens, of which the first n are there; what the table does not have is formed.
template <int N>
__device__ __forceinline__ unsigned long long sum_values(const Scale &s, const Shared &sh, uint32_t base, const float (&l)[N],
                                                         int n, float after, unsigned long long least) {
    uint32_t miss = 0;
    unsigned long long sum = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t bits = __float_as_uint(l[j]), at = (bits >> 16 & 0x7fffu) - base;
        if (j >= n) continue;
        if (at < kHalf) {
            sum += sh.steps.value[at + (bits >> 31) * kHalf];
        } else if (l[j] > after) {
            const float x = coarse(s, l[j]);
            if (x < kCareful) {
                miss |= 1u << j;
            } else {
                const unsigned long long w = small_weight(x);
                sum += w >= least ? w : 0ull;
            }
        }
    }
    while (__any_sync(kFullMask, miss != 0)) {
        const int now = __ffs(miss) - 1;
        float v = s.top;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j == now) v = l[j];
        const unsigned long long w = weight_of(s, sh.table, v);
        if (miss && w >= least) sum += w;
        miss &= miss - 1;
    }
    return sum;
}

// ------------------------------------------------------------------------------ reductions
__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

template <bool BF16, int T>
struct Row {
    const uint8_t *data;  // this CTA's tokens
    int len, first;       // their number, the first one's index
    int head;             // tokens ahead of the first 16-byte boundary
    static constexpr int kVec = BF16 ? 8 : 4;
    // f(i, value) of every token, in no order.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        const int body = (len - head) / kVec, tail = head + body * kVec, tid = threadIdx.x;
        if (tid < head) f(tid, at(tid));
        if (tail + tid < len && tid < kVec) f(tail + tid, at(tail + tid));
        const uint4 *from = reinterpret_cast<const uint4 *>(data + head * (BF16 ? 2 : 4));
        for (int i = tid; i < body; i += T) {
            float v[kVec];
            vec(from[i], v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) f(head + i * kVec + j, v[j]);
        }
    }
    // f(i, values, n) of groups of n <= kVec tokens next to one another in [from, to), a whole warp together (n = 0 for
    // lanes without any).
    template <typename F>
    __device__ __forceinline__ void walk(int from, int to, F f) const {
        const int lane = threadIdx.x & 31;
        // whole 16-byte groups, and a lane a token ahead of them and behind
        const int g0 = min(to, from + (((head - from) % kVec) + kVec) % kVec), groups = (to - g0) / kVec, tail = g0 + groups * kVec;
        float v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = 0.f;
        if (from < g0 || tail < to) {
            const int n0 = g0 - from, n1 = to - tail, i = lane < n0 ? from + lane : tail + lane - n0;
            const bool live = lane < n0 + n1;
            if (live) v[0] = at(i);
            f(i, v, live ? 1 : 0);
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(data + g0 * (BF16 ? 2 : 4));
        for (int g = 0; g < groups; g += 32) {
            const bool live = g + lane < groups;
            vec(live ? src[g + lane] : make_uint4(0, 0, 0, 0), v);
            f(g0 + (g + lane) * kVec, v, live ? kVec : 0);
        }
    }
    __device__ __forceinline__ static void vec(uint4 u, float (&v)[kVec]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (BF16) {
                v[(2 * j) % kVec] = __uint_as_float(w[j] << 16) + 0.f;
                v[(2 * j + 1) % kVec] = __uint_as_float(w[j] & 0xffff0000u) + 0.f;
            } else {
                v[j % kVec] = __uint_as_float(w[j]) + 0.f;
            }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        float v;
        if (BF16)
            v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(data)[i]) << 16);
        else
            v = reinterpret_cast<const float *>(data)[i];
        return v + 0.f;  // one zero
    }
};
__device__ __forceinline__ uint32_t key_of(float v) { return v == v ? order_bits(v) : 0u; }
__device__ __forceinline__ unsigned long long place_of(uint32_t key, int index) {
    return static_cast<unsigned long long>(key) << 32 | static_cast<uint32_t>(~index);
}

// Sum over the cluster of two 64-bit numbers a thread; all threads get the totals.
template <int T>
__device__ __forceinline__ void cluster_sum(Shared &sh, uint32_t rank, uint32_t ctas, unsigned long long &a,
                                            unsigned long long &b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_sum64(a);
    b = warp_sum64(b);
    if (lane == 0) {
        sh.warp64[0][warp] = a;
        sh.warp64[1][warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
        a = warp_sum64(lane < T / 32 ? sh.warp64[0][lane] : 0);
        b = warp_sum64(lane < T / 32 ? sh.warp64[1][lane] : 0);
        if (lane < static_cast<int>(ctas)) {
            unsigned long long *to = in_cta(&sh.pair[rank][0], lane);
            to[0] = a;
            to[1] = b;
        }
    }
    cluster_sync();
    a = b = 0;
    for (uint32_t r = 0; r < ctas; ++r) {
        a += sh.pair[r][0];
        b += sh.pair[r][1];
    }
    cluster_sync();  // the pairs may be written again
}

// The least key in (lo, hi] for which f holds, which it does for hi and what lies between; by half a warp, whose lanes
// differ from the other half's in what they ask for.
template <typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, F f) {
    const int lane = threadIdx.x & 15, half = threadIdx.x & 16;
#pragma unroll 1
    for (int round = 0; round < 8; ++round) {  // 16^8 keys
        const uint32_t step = (hi - lo - 1) / 16 + 1;
        const unsigned long long at = lo + static_cast<unsigned long long>(lane + 1) * step;
        const unsigned no = __ballot_sync(kFullMask, !f(at < hi ? static_cast<uint32_t>(at) : hi));
        lo += __popc(no >> half & 0xffffu) * step;
        hi = static_cast<uint32_t>(min(static_cast<unsigned long long>(hi), static_cast<unsigned long long>(lo) + step));
    }
    return hi;
}

// Sorts n places, largest first: few by counting the larger ones, many (padded with zeros to a power of two) in
// bitonic turns.
template <int T>
__device__ __forceinline__ void sort_list(Shared &sh, int n) {
    if (n <= 512) {
        unsigned long long mine = 0;
        int at = 0;
        if (static_cast<int>(threadIdx.x) < n) {
            mine = sh.list[threadIdx.x];
#pragma unroll 4
            for (int j = 0; j < n; ++j) at += sh.list[j] > mine;
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n) sh.list[at] = mine;
        __syncthreads();
        return;
    }
    int size = 32;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += T) sh.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int t = threadIdx.x; t < size / 2; t += T) {
                const int i = (t / j) * 2 * j + (t & (j - 1)), o = i + j;
                const unsigned long long a = sh.list[i], b = sh.list[o];
                if ((a < b) == ((i & k) == 0)) {
                    sh.list[i] = b;
                    sh.list[o] = a;
                }
            }
            __syncthreads();
        }
}

// Inclusive prefix sums of sh.weight[0 .. n), by the whole CTA.
template <int T>
__device__ __forceinline__ void scan_weights(Shared &sh, int n) {
    const int per = (n + T - 1) / T, i0 = threadIdx.x * per;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned long long s = 0;
    for (int i = i0; i < min(n, i0 + per); ++i) s += sh.weight[i];
    unsigned long long incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sh.warp64[0][warp] = incl;
    __syncthreads();
    unsigned long long run = incl - s;
    for (int w = 0; w < warp; ++w) run += sh.warp64[0][w];
    for (int i = i0; i < min(n, i0 + per); ++i) sh.weight[i] = run += sh.weight[i];
    __syncthreads();
}

// Appends a token to this CTA's list, which may be full.
__device__ __forceinline__ void append(Shared &sh, unsigned long long place) {
    const uint32_t at = atomicAdd(&sh.count, 1u);
    if (at < kCap) sh.list[at] = place;
}
// All CTAs' lists join the first one's, whose count is then of all.  (Appended there one by one a token waits for its
// place 1500 cycles.)
template <int T>
__device__ __forceinline__ void join_lists(Shared &sh, uint32_t rank) {
    __syncthreads();
    if (rank != 0) {
        Shared *first = in_cta(&sh, 0);
        const uint32_t n = sh.count;
        if (threadIdx.x == 0 && n > 0) sh.found = atomicAdd(&first->count, n);
        __syncthreads();
        const uint32_t at = sh.found;
        for (uint32_t i = threadIdx.x; i < min(n, static_cast<uint32_t>(kCap)) && at + i < kCap; i += T)
            first->list[at + i] = sh.list[i];
    }
    cluster_sync();
}

__device__ __forceinline__ float value_of(unsigned long long place) { return unorder_bits(static_cast<uint32_t>(place >> 32)); }
__device__ __forceinline__ int index_of(unsigned long long place) { return static_cast<int>(~static_cast<uint32_t>(place)); }

// f * total for f in [0, 1], rounded down, and whether something was dropped.
__device__ __forceinline__ unsigned long long part_of(float f, unsigned long long total, bool &rest) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max(static_cast<int>(bits >> 23), 1);
    const unsigned long long m = (bits & 0x7fffffu) | (bits >= 0x800000u ? 0x800000u : 0u);  // f = m 2^(e - 150)
    const unsigned long long lo = m * total, hi = __umul64hi(m, total);
    const int shift = 150 - e;  // 23 to 149
    rest = false;
    if (shift >= 128) {
        rest = (hi | lo) != 0;
        return 0;
    }
    if (shift >= 64) {
        rest = lo != 0 || (shift > 64 && (hi << (128 - shift)) != 0);
        return hi >> (shift - 64);
    }
    rest = (lo << (64 - shift)) != 0;
    return hi << (64 - shift) | lo >> shift;
}
// The least sum that reaches p of `total`; u of `total`, which the drawn token's sum is above.
__device__ __forceinline__ unsigned long long reach(float p, unsigned long long total) {
    bool rest;
    const unsigned long long n = part_of(p, total, rest);
    return n + rest;
}
__device__ __forceinline__ unsigned long long below(float u, unsigned long long total) {
    bool rest;
    return min(part_of(u, total, rest), total - 1);
}

// Of the sorted list's first n tokens: how many hold `need` of weight, at least one.  sh.weight has their sums.
__device__ __forceinline__ int first_reaching(const Shared &sh, int n, unsigned long long need) {
    int lo = 0, hi = n - 1;  // the first i with weight[i] >= need, the last at most
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sh.weight[mid] >= need) hi = mid; else lo = mid + 1;
    }
    return lo + 1;
}

template <bool BF16, int T>
__global__ void __launch_bounds__(T, 1024 / T) sample_kernel(const SampleArgs a) {
    constexpr int kWarps = T / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cta_rank(), ctas = cta_count();
    const int row_i = blockIdx.x / static_cast<int>(ctas);
    constexpr int kSize = BF16 ? 2 : 4;
    cluster_arrive_entry();
    griddep_launch_dependents();
    griddep_wait();
    const float temperature = a.temperature ? __ldcg(a.temperature + row_i) : 1.f;
    const int k_in = a.top_k ? __ldcg(a.top_k + row_i) : 0;
    const float p_in = a.top_p ? __ldcg(a.top_p + row_i) : 1.f, min_in = a.min_p ? __ldcg(a.min_p + row_i) : 0.f,
                u_in = __ldcg(a.u + row_i);

    // ------------------------------------------------------------------ the row into shared memory
    Row<BF16, T> row;
    row.first = min(a.vocab, static_cast<int>(rank) * a.slice);
    row.len = min(a.vocab, row.first + a.slice) - row.first;
    const uint8_t *src = static_cast<const uint8_t *>(a.logits) + (row_i * a.stride + row.first) * kSize;
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
    uint8_t *dst = smem + sizeof(Shared) + skew;
    row.data = dst;
    row.head = min(row.len, ((16 - skew) & 15) / kSize);
    float top = -INFINITY;  // of this thread's tokens
    bool any = false;       // one is a number
    {
        const int bytes = row.len * kSize, head = min(bytes, (16 - skew) & 15);
        const int body = (bytes - head) / 16, tail0 = head + body * 16;
        const auto look = [&](float v) {
            if (v == v) {
                top = fmaxf(top, v);
                any = true;
            }
        };
        const auto one = [&](int at) {
            if (BF16) {
                const uint16_t w = __ldcg(reinterpret_cast<const uint16_t *>(src + at));
                *reinterpret_cast<uint16_t *>(dst + at) = w;
                look(__uint_as_float(static_cast<uint32_t>(w) << 16));
            } else {
                const float w = __ldcg(reinterpret_cast<const float *>(src + at));
                *reinterpret_cast<float *>(dst + at) = w;
                look(w);
            }
        };
        if (tid * kSize < head) one(tid * kSize);
        if (tail0 + tid * kSize < bytes) one(tail0 + tid * kSize);
        const uint4 *from = reinterpret_cast<const uint4 *>(src + head);
        uint4 *to = reinterpret_cast<uint4 *>(dst + head);
#pragma unroll 8
        for (int i = tid; i < body; i += T) {
            const uint4 v = __ldcg(from + i);
            to[i] = v;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (BF16) {
                    look(__uint_as_float(w[j] << 16));
                    look(__uint_as_float(w[j] & 0xffff0000u));
                } else {
                    look(__uint_as_float(w[j]));
                }
            }
        }
    }
    for (int j = tid; j < kTable; j += T) sh.table[j] = __ldg(&g_powers.at[j]);
    if (tid == 0) sh.count = 0;
    cluster_wait_entry();
    const uint32_t my_top = any ? key_of(top + 0.f) : 0u;
    {
        const uint32_t m = __reduce_max_sync(kFullMask, my_top);
        if (lane == 0) sh.warp32[warp] = m;
        __syncthreads();
        if (warp == 0) {
            const uint32_t c = __reduce_max_sync(kFullMask, lane < kWarps ? sh.warp32[lane] : 0u);
            if (lane < static_cast<int>(ctas)) *in_cta(&sh.from_cta[rank], lane) = c;
        }
        cluster_sync();
    }
    uint32_t top_key = 0;
    for (uint32_t r = 0; r < ctas; ++r) top_key = max(top_key, sh.from_cta[r]);

    int k = k_in;
    if (k <= 0 || k > a.vocab) k = a.vocab;
    float p = p_in;
    if (!(p < 1.f)) p = 1.f;
    if (p <= 0.f) {
        p = 1.f;
        k = 1;
    }
    const float floor_p = fminf(fmaxf(min_in, 0.f), 1.f);
    const unsigned long long least = max(1ull, __float2ull_ru(floor_p * 0x1p44f));
    const float u = u_in > 0.f ? fminf(u_in, 1.f) : 0.f;

    // ------------------------------------------------------------------ greedy
    if (!(temperature > 0.f) || k == 1 || top_key <= kLeastKey) {
        uint32_t best = 0xffffffffu;
        if (my_top == top_key)
            row.each([&](int i, float v) {
                if (key_of(v) == top_key) best = min(best, static_cast<uint32_t>(row.first + i));
            });
        best = __reduce_min_sync(kFullMask, best);
        cluster_sync();  // the tops have been read
        if (lane == 0) sh.warp32[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = __reduce_min_sync(kFullMask, lane < kWarps ? sh.warp32[lane] : 0xffffffffu);
            if (lane == 0) *in_cta(&sh.from_cta[rank], 0) = best;
        }
        cluster_sync();
        if (rank == 0 && tid == 0) {
            for (uint32_t r = 1; r < ctas; ++r) best = min(best, sh.from_cta[r]);
            a.out[row_i] = static_cast<int>(best);
        }
        return;
    }
    Scale s;
    s.top = unorder_bits(top_key);
    {
        const float t = fminf(fmaxf(temperature, 1e-30f), 1e30f), kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;
        s.hi = __fdiv_rn(kLog2e, t);
        s.lo = __fdiv_rn(__fmaf_rn(-s.hi, t, kLog2e) + kLog2eLo, t);
    }

    // ------------------------------------------------------------------ top-k: few tokens, sorted
    const int each = (k + static_cast<int>(ctas) - 1) / static_cast<int>(ctas);
    unsigned long long cut_k = 0;  // what is kept has this place or a higher one; 0: everything
    if (k < a.vocab && each <= T / 2 && k <= kCap / 2) {
        // a key that `each` threads' largest reach, near the highest such: of the warps' largest where they are enough
        uint32_t lo = 0, hi = 0xffffffffu;
        if (each <= kWarps - 2) {
            __syncthreads();
            const uint32_t w = lane < kWarps ? sh.warp32[lane] : 0u;
            int above = 0;
#pragma unroll
            for (int j = 0; j < kWarps; ++j) {
                const uint32_t o = __shfl_sync(kFullMask, w, j);
                above += o > w || (o == w && j < lane);
            }
            lo = __shfl_sync(kFullMask, w, __ffs(__ballot_sync(kFullMask, lane < kWarps && above == each - 1)) - 1);
        } else {
            for (int bit = 0; bit < 32; ++bit) {
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                const int n = __syncthreads_count(my_top >= mid);
                if (n >= each) lo = mid; else hi = mid - 1;
                if (n >= each && n <= each + each / 8) break;
                if (lo == hi) break;
            }
        }
        if (tid < static_cast<int>(ctas)) *in_cta(&sh.bounds[rank], tid) = lo;
        cluster_sync();
        uint32_t bound = 0xffffffffu;
        for (uint32_t r = 0; r < ctas; ++r) bound = min(bound, sh.bounds[r]);
        bound = max(bound, kLeastKey + 1);  // masked tokens are never drawn, however few are left
        if (my_top >= bound)
            row.each([&](int i, float v) {
                const uint32_t key = key_of(v);
                if (key >= bound) append(sh, place_of(key, row.first + i));
            });
        join_lists<T>(sh, rank);
        const int n_all = static_cast<int>(in_cta(&sh, 0)->count);
        cluster_arrive();  // the count has been read
        if (n_all <= kCap) {
            if (rank == 0) {
                const int n = n_all;
                sort_list<T>(sh, n);
                const int m = min(n, k);
                unsigned long long w[kCap / T];  // of this thread's places
                for (int c = 0; c * T < m; ++c) {
                    const int i = c * T + tid;
                    if (i < m) sh.weight[i] = weight_of(s, sh.table, value_of(sh.list[i]));
                }
                __syncthreads();
                int kept = m;
                if (p < 1.f) {
#pragma unroll
                    for (int c = 0; c < kCap / T; ++c) w[c] = c * T + tid < m ? sh.weight[c * T + tid] : 0ull;
                    __syncthreads();
                    scan_weights<T>(sh, m);
                    kept = first_reaching(sh, m, reach(p, sh.weight[m - 1]));
                    __syncthreads();
#pragma unroll
                    for (int c = 0; c < kCap / T; ++c)
                        if (c * T + tid < m) sh.weight[c * T + tid] = w[c];
                    __syncthreads();
                }
                // min-p: weights fall along the list, so those that pass are its first ones
                int pass = 0;
                for (int i = tid; i < kept; i += T) pass += i == 0 || sh.weight[i] >= least;
                pass = __reduce_add_sync(kFullMask, pass);
                unsigned long long sum = 0;
                if (lane == 0) sh.warp32[warp] = pass;
                __syncthreads();
                kept = 0;
                for (int j = 0; j < kWarps; ++j) kept += static_cast<int>(sh.warp32[j]);
                for (int i = tid; i < kept; i += T) sum += sh.weight[i];
                sum = warp_sum64(sum);
                if (lane == 0) sh.warp64[0][warp] = sum;
                __syncthreads();
                sum = 0;
                for (int j = 0; j < kWarps; ++j) sum += sh.warp64[0][j];
                const unsigned long long goal = below(u, sum);
                if (kept > 128) {  // the least index up to which the sum passes the goal: every warp tries one
                    int from = 0, to = a.vocab - 1;
                    while (from < to) {
                        const int step = (to - from) / kWarps + 1, mid = min(to, from + (warp + 1) * step - 1);
                        unsigned long long part = 0;
                        for (int i = lane; i < kept; i += 32) part += index_of(sh.list[i]) <= mid ? sh.weight[i] : 0ull;
                        part = warp_sum64(part);
                        if (lane == 0) sh.warp32[warp] = part > goal;
                        __syncthreads();
                        const unsigned yes = __ballot_sync(kFullMask, lane < kWarps && sh.warp32[lane % kWarps] != 0);
                        from += (kWarps - __popc(yes)) * step;
                        to = min(to, from + step - 1);
                        __syncthreads();
                    }
                    if (tid == 0) a.out[row_i] = from;
                    kept = 0;
                }
                // a token's sum by index: of the kept ones with lower indices (which have the larger low words)
                for (int i = tid; i < kept; i += T) {
                    const uint32_t mine = static_cast<uint32_t>(sh.list[i]);
                    unsigned long long before = 0;
#pragma unroll 4
                    for (int j = 0; j < kept; ++j) before += static_cast<uint32_t>(sh.list[j]) > mine ? sh.weight[j] : 0ull;
                    if (before <= goal && goal < before + sh.weight[i]) a.out[row_i] = static_cast<int>(~mine);
                }
            }
            cluster_wait();
            return;
        }
        cluster_wait();
    }
    const auto in_k = [&](uint32_t key, int index) { return place_of(key, index) >= cut_k; };
    // a warp's tokens
    const int seg = (row.len + kWarps - 1) / kWarps, seg0 = min(row.len, warp * seg), seg1 = min(row.len, seg0 + seg);

    // f(value, times) of this CTA's bf16 tokens, counted: twenty binades of either sign, the others one by one.
    const bool tabled = BF16 && a.slice >= kTabled && fabsf(s.top) < 0x1p100f && 1.f / s.hi < 0x1p90f;
    const auto each_value = [&](auto f) {
        const uint32_t base = table_base(s, 20);
        for (int i = tid; i < static_cast<int>(2 * kValues); i += T) sh.steps.times[i] = 0;
        __syncthreads();
        row.walk(seg0, seg1, [&](int i0, const float(&v)[Row<BF16, T>::kVec], int n) {
#pragma unroll
            for (int j = 0; j < Row<BF16, T>::kVec; ++j) {
                if (j >= n || (cut_k != 0 && !in_k(key_of(v[j]), row.first + i0 + j))) continue;
                const uint32_t bits = __float_as_uint(v[j]), at = (bits >> 16 & 0x7fffu) - base;
                if (at < kValues)
                    atomicAdd(&sh.steps.times[at + (bits >> 31) * kValues], 1u);
                else
                    f(v[j], 1u);
            }
        });
        __syncthreads();
        for (uint32_t i = tid; i < 2 * kValues; i += T) {
            const uint32_t times = sh.steps.times[i], sign = i >= kValues;
            if (times) f(__uint_as_float(sign << 31 | (base + i - sign * kValues) << 16), times);
        }
    };

    // ------------------------------------------------------------------ top-k, then top-p
    // The same by numbers of tokens and by their weights.
    unsigned long long cut = 0;
    bool by_cta = false;  // what every CTA keeps is known
    // top-k by bisection over keys, then over indices
    const auto bisect_k = [&]() {
        uint32_t lo = 0, hi = top_key;  // the largest key that k tokens reach
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            unsigned long long n = 0, none = 0;
            row.each([&](int, float v) { n += key_of(v) >= mid; });
            cluster_sum<T>(sh, rank, ctas, n, none);
            if (n >= static_cast<unsigned long long>(k)) lo = mid; else hi = mid - 1;
        }
        unsigned long long above = 0, none = 0;
        row.each([&](int, float v) { above += key_of(v) > lo; });
        cluster_sum<T>(sh, rank, ctas, above, none);
        int from = 0, to = a.vocab - 1;  // the least index up to which enough equal ones lie
        while (from < to) {
            const int mid = (from + to) >> 1;
            unsigned long long n = 0;
            none = 0;
            row.each([&](int i, float v) { n += key_of(v) == lo && row.first + i <= mid; });
            cluster_sum<T>(sh, rank, ctas, n, none);
            if (above + n >= static_cast<unsigned long long>(k)) to = mid; else from = mid + 1;
        }
        cut = place_of(lo, from);
    };
    const auto find_cut = [&](auto what) {
        constexpr bool counting = decltype(what)::value;
        constexpr float octave = counting ? kCountOctave : kPerOctave, limit = counting ? 60.f : kCareful;
        unsigned long long total = 0, sure = 0;  // weight of all, and of what is surely kept
        bool sorted = false, beyond = false;
        int step0 = -1;  // the step that holds the cut, on the second level
        for (int level = 0; level < 2 && !sorted; ++level) {
            // A token's step: of 1 / octave, and within the one that holds the cut of 1 / (1536 octave).  Both are monotone in
            // l, whatever f32 rounds.
            const auto step_in = [&](float x) {
                const int b = static_cast<int>(x * octave);
                if (level == 0) return b;
                if (b != step0) return b < step0 ? -1 : kBins;
                return min(kBins - 1, max(0, static_cast<int>((x - step0 * (1.f / octave)) * (octave * kBins))));
            };
            for (int b = tid; b < 2 * kBins; b += T) sh.steps.lo[b] = 0;
            if (tid == 0) sh.count = 0;
            __syncthreads();
            // Small weights at once, into one sum: of 1e5 tokens up to 1e5 2^-24 of the largest, so that a cut lies there
            // where top-p leaves less, in steep rows as in flat ones.
            unsigned long long tail = 0, none = 0;
            const auto count = [&](int b, unsigned long long w) {
                const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.steps.lo[b], lo);
                const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old);
                if (hi) atomicAdd(&sh.steps.hi[b], hi);
            };
            if (BF16 && level == 0 && tabled)
                each_value([&](float l, uint32_t times) {
                    const float x = coarse(s, l);
                    if (!(x < 60.f)) return;
                    const unsigned long long w = (counting ? 1ull : weight_of(s, sh.table, l)) * times;
                    if (x >= limit)
                        tail += w;
                    else
                        count(step_in(x), w);
                });
            else
                row.walk(seg0, seg1, [&](int i0, const float(&v)[Row<BF16, T>::kVec], int n) {
                    float x[Row<BF16, T>::kVec];
                    unsigned long long w[Row<BF16, T>::kVec];
#pragma unroll
                    for (int j = 0; j < Row<BF16, T>::kVec; ++j) {
                        x[j] = coarse(s, v[j]);
                        // (NaN, -infinity: nothing)
                        if (j >= n || !(x[j] < 60.f) || (cut_k != 0 && !in_k(key_of(v[j]), row.first + i0 + j))) x[j] = 100.f;
                        if (level > 0 && (x[j] >= limit || step_in(x[j]) < 0 || step_in(x[j]) >= kBins)) x[j] = 100.f;
                    }
                    if (!counting) weights_of(s, sh.table, v, x, w);
#pragma unroll
                    for (int j = 0; j < Row<BF16, T>::kVec; ++j) {
                        if (counting) w[j] = x[j] < 60.f;
                        if (x[j] >= limit)
                            tail += w[j];
                        else
                            count(step_in(x[j]), w[j]);
                    }
                });
            cluster_sum<T>(sh, rank, ctas, tail, none);
            // Every CTA adds all CTAs' weights of its share of the steps (all of them by every one would be 12 KB from
            // each of the others: 13 us with 8); their sums tell in whose share the cut lies.  All loads are out at once.
            constexpr int kFetch = (kBins + T - 1) / T;
            const int share = kBins / static_cast<int>(ctas), per = (share + T - 1) / T;
            const int mine0 = tid * per, b0 = static_cast<int>(rank) * share + mine0;
            unsigned long long mass[kFetch], own = 0;
#pragma unroll
            for (int j = 0; j < kFetch; ++j) {
                const int i = j * T + tid, r = i / share;
                if (i < kBins) {
                    const Shared *other = in_cta(&sh, r);
                    const int b = static_cast<int>(rank) * share + i - r * share;
                    mass[j] = static_cast<unsigned long long>(other->steps.hi[b]) << 32 | other->steps.lo[b];
                }
            }
#pragma unroll
            for (int j = 0; j < kFetch; ++j)
                if (j * T + tid < kBins) sh.list[j * T + tid] = mass[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kFetch; ++j) {
                mass[j] = 0;
                if (j < per && mine0 + j < share)
                    for (uint32_t r = 0; r < ctas; ++r) mass[j] += sh.list[static_cast<int>(r) * share + mine0 + j];
                own += mass[j];
            }
            unsigned long long incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long up = __shfl_up_sync(kFullMask, incl, o);
                if (lane >= o) incl += up;
            }
            if (lane == 31) sh.warp64[0][warp] = incl;
            __syncthreads();
            unsigned long long run = incl - own, share_sum = 0;
            for (int w = 0; w < kWarps; ++w) {
                const unsigned long long x = sh.warp64[0][w];
                if (w < warp) run += x;
                share_sum += x;
            }
            if (tid < static_cast<int>(ctas)) *in_cta(&sh.pair[rank][0], tid) = share_sum;
            cluster_sync();  // and all steps have been read
            unsigned long long all = 0;
            for (uint32_t r = 0; r < ctas; ++r) {
                if (r == rank) run += all;
                all += sh.pair[r][0];
            }
            if (level == 0) total = all + tail;
            const unsigned long long goal = counting ? static_cast<unsigned long long>(k) : reach(p, total);
            const unsigned long long need = goal - sure;  // at least 1: the cut lies behind what is sure
            beyond = need > all;                          // in the tail
            if (beyond) {
                cluster_sync();  // the sums have been read: what comes next writes them again
                break;
            }
#pragma unroll
            for (int j = 0; j < kFetch; ++j) {
                if (run < need && need <= run + mass[j])
                    for (uint32_t r = 0; r < ctas; ++r) {
                        Shared *other = in_cta(&sh, r);
                        other->step = b0 + j;
                        other->before = run;
                    }
                run += mass[j];
            }
            cluster_sync();
            const int step = sh.step;
            sure += sh.before;
            unsigned long long ahead = 0;  // what this CTA keeps of the steps ahead
            for (int b = tid; b < step; b += T) ahead += static_cast<unsigned long long>(sh.steps.hi[b]) << 32 | sh.steps.lo[b];
            ahead = warp_sum64(ahead);
            if (lane == 0) sh.warp64[1][warp] = ahead;
            // the step's logits are a range: its least, and the least behind it (if it is not the first)
            if (warp == 0) {
                const uint32_t key = first_key(kLeastKey, top_key, [&](uint32_t key) {
                    return step_in(coarse(s, unorder_bits(key))) <= step - (lane >> 4);
                });
                if ((lane & 15) == 0) sh.bounds[lane >> 4] = key;
            }
            __syncthreads();
            const float least_v = unorder_bits(sh.bounds[0]);
            const float most_v = step_in(0.f) < step ? unorder_bits(sh.bounds[1] - 1) : s.top;
            row.each([&](int i, float v) {
                if (v >= least_v && v <= most_v) {
                    const uint32_t key = key_of(v);
                    if (cut_k == 0 || in_k(key, row.first + i)) append(sh, place_of(key, row.first + i));
                }
            });
            join_lists<T>(sh, rank);
            if (tid < static_cast<int>(ctas)) {
                ahead = 0;
                for (int w = 0; w < kWarps; ++w) ahead += sh.warp64[1][w];
                in_cta(&sh, tid)->pair[rank][1] = ahead;
            }
            const int n_all = static_cast<int>(in_cta(&sh, 0)->count);
            if (n_all <= kCap) {
                sorted = true;
                by_cta = !counting && level == 0 && least == 1;
                if (rank == 0) {
                    sort_list<T>(sh, n_all);
                    for (int i = tid; i < n_all; i += T)
                        sh.weight[i] = counting ? 1ull : weight_of(s, sh.table, value_of(sh.list[i]));
                    __syncthreads();
                    scan_weights<T>(sh, n_all);
                    const int kept = first_reaching(sh, n_all, goal - sure);
                    if (tid < static_cast<int>(ctas)) *in_cta(&sh.cut, tid) = sh.list[kept - 1];
                    if (warp < static_cast<int>(ctas)) {  // a warp adds up what a CTA keeps of the step
                        unsigned long long of_cta = 0;
                        for (int i = lane; i < kept; i += 32)
                            if (index_of(sh.list[i]) / a.slice == warp) of_cta += sh.weight[i] - (i ? sh.weight[i - 1] : 0ull);
                        of_cta = warp_sum64(of_cta);
                        if (lane < static_cast<int>(ctas)) *in_cta(&sh.partial[warp], lane) = of_cta;
                    }
                }
            }
            cluster_sync();
            if (sorted) cut = max(cut, sh.cut);
            step0 = step;
        }
        if (counting) {
            // (behind 60 octaves no token has a weight, so nothing is cut)
            if (!sorted && !beyond) bisect_k();
            cut_k = cut;
            return;
        }
        if (!sorted) {  // thousands of equal tokens: bisection over keys, by weight
            const unsigned long long need = reach(p, total);
            uint32_t lo = kLeastKey, hi = top_key;
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                unsigned long long w = 0, none = 0;
                row.each([&](int i, float v) {
                    const uint32_t key = key_of(v);
                    if (key >= mid && in_k(key, row.first + i)) w += weight_of(s, sh.table, v);
                });
                cluster_sum<T>(sh, rank, ctas, w, none);
                if (w >= need) lo = mid; else hi = mid - 1;
            }
            unsigned long long above = 0, none = 0;
            row.each([&](int i, float v) {
                const uint32_t key = key_of(v);
                if (key > lo && in_k(key, row.first + i)) above += weight_of(s, sh.table, v);
            });
            cluster_sum<T>(sh, rank, ctas, above, none);
            const unsigned long long one = max(1ull, weight_of(s, sh.table, unorder_bits(lo)));
            const unsigned long long ties = need > above ? (need - above + one - 1) / one : 1ull;
            int from = 0, to = a.vocab - 1;
            while (from < to) {
                const int mid = (from + to) >> 1;
                unsigned long long n = 0;
                none = 0;
                row.each([&](int i, float v) {
                    n += key_of(v) == lo && row.first + i <= mid && in_k(lo, row.first + i);
                });
                cluster_sum<T>(sh, rank, ctas, n, none);
                if (n >= ties) to = mid; else from = mid + 1;
            }
            cut = max(cut, place_of(lo, from));
        }
    };
    if (k < a.vocab) find_cut(std::true_type{});
    if (p < 1.f) find_cut(std::false_type{});

    // ------------------------------------------------------------------ the draw
    // A warp's tokens are consecutive, so its sum's place among the others is its place by index.
    const float cut_v = cut ? value_of(cut) : -INFINITY;
    const int cut_i = cut ? index_of(cut) : 0x7fffffff;
    const auto keep = [&](float v, int i) { return v > cut_v || (v == cut_v && row.first + i <= cut_i); };
    const auto kept_weight = [&](int i) -> unsigned long long {
        const float v = row.at(i);
        if (!keep(v, i)) return 0ull;
        const unsigned long long w = weight_of(s, sh.table, v);
        return w >= least ? w : 0ull;
    };
    unsigned long long mine = 0, goal = 0;
    if (by_cta) {  // the steps' weights tell whose token it is: the others are done
        unsigned long long total = 0, first = 0, mine_all = 0;
        for (uint32_t r = 0; r < ctas; ++r) total += sh.pair[r][1] + sh.partial[r];
        goal = below(u, total);
        for (uint32_t r = 0; r < ctas; ++r) {
            const unsigned long long w = sh.pair[r][1] + sh.partial[r];
            if (r < rank) first += w;
            if (r == rank) mine_all = w;
        }
        if (goal < first || goal >= first + mine_all) return;
        goal -= first;
    }
    const float after = cut ? cut_v : -INFINITY;
    const uint32_t base = table_base(s, 10);
    if (tabled) make_values<T>(s, sh, base, after, least);
    const unsigned long long cut_w = cut ? weight_of(s, sh.table, cut_v) : 0ull;
    row.walk(seg0, seg1, [&](int i0, const float(&v)[Row<BF16, T>::kVec], int n) {
        float x[Row<BF16, T>::kVec];
        unsigned long long w[Row<BF16, T>::kVec];
        if (tabled) {
            mine += sum_values(s, sh, base, v, n, after, least);
#pragma unroll
            for (int j = 0; j < Row<BF16, T>::kVec; ++j)
                if (v[j] == cut_v && row.first + i0 + j <= cut_i && j < n && cut_w >= least) mine += cut_w;
            return;
        }
#pragma unroll
        for (int j = 0; j < Row<BF16, T>::kVec; ++j) {
            x[j] = coarse(s, v[j]);
            if (j >= n || !(x[j] < 60.f) || !keep(v[j], i0 + j)) x[j] = 100.f;
        }
        weights_of(s, sh.table, v, x, w);
#pragma unroll
        for (int j = 0; j < Row<BF16, T>::kVec; ++j)
            if (w[j] >= least) mine += w[j];
    });
    mine = warp_sum64(mine);
    if (by_cta) {
        if (lane == 0) sh.sums[rank][warp] = mine;
        __syncthreads();
    } else {
        if (lane < static_cast<int>(ctas)) *in_cta(&sh.sums[rank][warp], lane) = mine;
        cluster_sync();
    }
    // The warp whose sum passes the goal: its CTA's warps share its tokens, then one goes through what is left.  A lane
    // holds four of the cluster's sums.
    constexpr int kEach = kMaxCtas * kWarps / 32;
    unsigned long long some[kEach], incl = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int k = lane * kEach + j;
        const bool there = by_cta ? k / kWarps == static_cast<int>(rank) : k < static_cast<int>(ctas) * kWarps;
        some[j] = there ? sh.sums[k / kWarps][k % kWarps] : 0ull;
        incl += some[j];
    }
    const unsigned long long own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += up;
    }
    const unsigned long long of_all = __shfl_sync(kFullMask, incl, 31);
    if (!by_cta) goal = below(u, of_all);
    const int at = __ffs(__ballot_sync(kFullMask, incl > goal)) - 1;
    unsigned long long before = incl - own;
    int place = lane * kEach;
#pragma unroll
    for (int j = 0; j < kEach - 1; ++j) {
        if (before + some[j] > goal) break;
        before += some[j];
        ++place;
    }
    before = __shfl_sync(kFullMask, before, at);
    place = __shfl_sync(kFullMask, place, at);
    const uint32_t r = static_cast<uint32_t>(place / kWarps);
    const int w = place % kWarps;
    if (r != rank) return;
    const int from = min(row.len, w * seg), to = min(row.len, from + seg), part = (to - from + kWarps - 1) / kWarps;
    const int part0 = min(to, from + warp * part), part1 = min(to, part0 + part);
    mine = 0;
    for (int i = part0 + lane; i < part1; i += 32) mine += kept_weight(i);
    mine = warp_sum64(mine);
    if (lane == 0) sh.warp64[0][warp] = mine;
    __syncthreads();
    for (int j = 0; j < warp; ++j) before += sh.warp64[0][j];
    if (goal < before || goal >= before + mine) return;
    for (int i0 = part0; i0 < part1; i0 += 32) {
        incl = i0 + lane < part1 ? kept_weight(i0 + lane) : 0ull;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long up = __shfl_up_sync(kFullMask, incl, o);
            if (lane >= o) incl += up;
        }
        const unsigned over = __ballot_sync(kFullMask, before + incl > goal);
        if (over) {
            if (lane == 0) a.out[row_i] = row.first + i0 + __ffs(over) - 1;
            return;
        }
        before += __shfl_sync(kFullMask, incl, 31);
    }
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

constexpr int kMaxDevices = 64;

bool allow(void (*kern)(const SampleArgs), int smem) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
}

// SM count and opt-in shared memory of the current device, after allowing the kernels all of it.
bool device_info(int &sms, int &smem) {
    static std::atomic<int> sm_cache[kMaxDevices], smem_cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < kMaxDevices && (sms = sm_cache[dev].load(std::memory_order_acquire)) > 0) {
        smem = smem_cache[dev].load(std::memory_order_relaxed);
        return true;
    }
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        !allow(sample_kernel<false, 512>, smem) || !allow(sample_kernel<true, 512>, smem) ||
        !allow(sample_kernel<false, 1024>, smem) || !allow(sample_kernel<true, 1024>, smem))
        return false;
    if (dev < kMaxDevices) {
        smem_cache[dev].store(smem, std::memory_order_relaxed);
        sm_cache[dev].store(sms, std::memory_order_release);
    }
    return true;
}

}  // namespace
}  // namespace memq

extern "C" int memq_sample(int dtype, const void *logits, int64_t stride, const float *temperature, const int32_t *top_k,
                           const float *top_p, const float *min_p, const float *u, int32_t *out, int64_t rows,
                           int64_t vocab, void *stream) {
    using namespace memq;
    if ((dtype != MEMQ_F32 && dtype != MEMQ_BF16) || rows < 0 || rows > (1 << 20) || vocab < 1 || vocab > kMaxVocab ||
        stride < 0 || stride > (int64_t{1} << 40))
        return MEMQ_ERR_SHAPE;
    if (rows == 0) return MEMQ_OK;
    if (!logits || !u || !out) return MEMQ_ERR_NULL;
    const int size = dtype == MEMQ_F32 ? 4 : 2;
    if (misaligned(logits, size) || misaligned(temperature, 4) || misaligned(top_k, 4) || misaligned(top_p, 4) ||
        misaligned(min_p, 4) || misaligned(u, 4) || misaligned(out, 4))
        return MEMQ_ERR_ALIGN;
    int sms = 0, smem = 0;
    if (!device_info(sms, smem)) return MEMQ_ERR_LAUNCH;
    SampleArgs a{logits, stride, temperature, top_p, min_p, u, top_k, out, static_cast<int>(vocab), 0};
    // As many CTAs a row as fill the GPU, and so many that two of them fit on an SM, if a cluster has as many.
    const auto slice_of = [&](int ctas) { return static_cast<int>(((vocab + ctas - 1) / ctas + 15) / 16 * 16); };
    const auto bytes_of = [&](int ctas) { return static_cast<int>(sizeof(Shared)) + slice_of(ctas) * size + 16; };
    int ctas = 1;
    while (ctas < kMaxCtas && (bytes_of(ctas) > smem / 2 || (rows * ctas * 2 <= sms && slice_of(ctas) > 2048))) ctas *= 2;
    if (bytes_of(ctas) > smem) return MEMQ_ERR_SHAPE;
    a.slice = slice_of(ctas);
    // A CTA that has its SM to itself takes all the threads that two would (us with 512 / 1024: 32 x 128259 bf16 top-p
    // 52 / 43, no cut 30 / 19; 64 x 32000 19 / 15; 8 x 128259 f32 42.5 / 42.0), unless its tokens are few (4000 of 1 x 32000:
    // 23 / 26).
    const bool wide = rows * ctas <= sms && a.slice > 8192;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
    cfg.blockDim = dim3(wide ? 1024 : 512);
    cfg.dynamicSmemBytes = static_cast<size_t>(bytes_of(ctas));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    using Kernel = void (*)(const SampleArgs);
    static constexpr Kernel kKernels[2][2] = {{sample_kernel<false, 512>, sample_kernel<false, 1024>},
                                              {sample_kernel<true, 512>, sample_kernel<true, 1024>}};
    return cudaLaunchKernelEx(&cfg, kKernels[dtype == MEMQ_BF16][wide], a) == cudaSuccess
               ? MEMQ_OK
               : MEMQ_ERR_LAUNCH;
}
