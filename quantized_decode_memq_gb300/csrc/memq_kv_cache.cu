// memq_kv_cache.cu -- the paged E4M3 cache of keys and values: memq_kv_cache_append quantises rows as
// it writes them, memq_kv_cache_read returns the values that cached rows stand for.
//
// The 16 tokens of a block share a scale per kv head, a power of two: the least with max |x| <= 448 scale.
// E4M3 codes are floating-point numbers, so a finer scale would gain nothing but the last 15% of their
// range; a power of two makes every product and quotient with it exact, the rows of a block that is filled
// in several calls among them: when a later row needs a larger scale, the codes of the earlier ones move
// down by whole binades and lose bits only below 2^-6.
//
// A warp serves the rows of one block and head, keys in its lower half and values in its upper: a lane
// holds D / 16 elements of each row, so inputs are read once, a row's codes leave as 16 lanes x 8 bytes and
// the maximum is one reduction a block.  16381 rows of bf16, 8 kv heads of 128: 24.4 us (26 without the
// prefetch), 4.1 TB/s of what is read and written (67 + 34 MB), bound by a block's work behind its loads, with none of the
// next one's in flight (issue 42%, DRAM 33%); of f32 42.6 us, 3.9 TB/s; 256 single rows of f32 6.6 us.
//
// A read is latency: slot, then codes and scale, of rows that lie anywhere (16381 rows of 8 x 128 11.4 us each pool, 4.4
// TB/s of codes and bf16; to f32 20.4 us).
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "memq.h"
#include "memq_dev.cuh"
#include "memq_tc.cuh"

namespace memq {
namespace {

__device__ unsigned int g_kv_fault = 0;
constexpr unsigned int kFaultInput = 32;  // a slot was outside the pool

constexpr int kBlock = 16;  // tokens that share a scale
constexpr int kAppendThreads = 128, kAppendWarps = kAppendThreads / 32;
constexpr int kReadThreads = 256;
constexpr int kLeast = -100;  // exponent of the least scale

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

struct AppendArgs {
    const void *k, *v;
    int64_t k_stride, v_stride;  // elements from one token's row to the next
    const int32_t *slots;
    uint8_t *k_cache, *v_cache;
    float *k_scales, *v_scales;
    int64_t n, pool;
    int n_kv, page_shift, window;
};

// E elements of a row, as they come: 16 rows of bf16 take 64 registers a lane and leave room for four CTAs on an SM
// (as f32 they took 128: one CTA, and loads, work and stores of a block did not overlap).
template <int E, bool BF16>
struct Elems {
    static constexpr int kWords = BF16 ? E / 2 : E;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        const uint8_t *src = static_cast<const uint8_t *>(p) + at * (BF16 ? 2 : 4);
        if constexpr (kWords == 2) {
            const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(src));
            w[0] = u.x;
            w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(src) + i);
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (BF16)
            return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else
            return __uint_as_float(w[i]);
    }
    // max |x| as bits: infinities and NaN lie above all numbers.
    __device__ __forceinline__ uint32_t largest() const {
        if constexpr (BF16) {
            uint32_t m = 0;  // two 16-bit maxima
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            return max(m << 16, m & 0xffff0000u);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        }
    }
};

template <int E>
__device__ __forceinline__ void store_codes(uint8_t *at, const uint32_t (&c)[E / 4]) {
    if (E == 8)
        *reinterpret_cast<uint2 *>(at) = make_uint2(c[0], c[E / 4 - 1]);
    else
        *reinterpret_cast<uint32_t *>(at) = c[0];
}

// The row's codes: those of x * inv, or for a row that is not finite NaN (keys) or 0 (values).
template <int E, bool BF16>
__device__ __forceinline__ void store_row(uint8_t *at, const Elems<E, BF16> &r, float inv, bool fin, bool keys) {
    uint32_t c[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        c[i] = f32x2_to_e4m3x2(r.at(4 * i) * inv, r.at(4 * i + 1) * inv) |
               f32x2_to_e4m3x2(r.at(4 * i + 2) * inv, r.at(4 * i + 3) * inv) << 16;
        if (!fin) c[i] = keys ? 0x7f7f7f7fu : 0u;
    }
    store_codes<E>(at, c);
}

// e of the least power of two with top <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exponent(uint32_t b) {  // of the bits of `top`
    const int k = static_cast<int>(b >> 23) - 127;
    return max(kLeast, (b & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7);
}
__device__ __forceinline__ float power_of_two(int e) {  // -149 <= e <= 127
    return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAppendThreads, BF16 || D == 64 ? 4 : 2) kv_append_kernel(const AppendArgs a) {
    constexpr int E = D / 16;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, half = lane >> 4, part = lane & 15;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t r0 = unit / a.n_kv * a.window;
    const int h = static_cast<int>(unit % a.n_kv);
    if (r0 >= a.n) return;
    const int64_t r_end = min(a.n, r0 + a.window);
    const auto block_of = [&](int64_t r) -> int64_t {  // of row r; -1 for none
        if (r < 0 || r >= a.n) return -1;
        const int64_t s = __ldcg(a.slots + r);
        return s < 0 || s >= a.pool ? -1 : s / kBlock;
    };
    if (a.window > 1 && r0 + part < a.n) {  // the rows are on their way to L2 while the slots are looked up
        const uint8_t *row = static_cast<const uint8_t *>(half ? a.v : a.k) +
                             ((r0 + part) * (half ? a.v_stride : a.k_stride) + h * D) * (BF16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < D * (BF16 ? 2 : 4); i += 128) prefetch_l2(row + i);
    }
    // rows of this window that begin a block
    const int64_t mine = r0 + lane < r_end ? r0 + lane : -1;
    if (h == 0 && mine >= 0 && __ldcg(a.slots + mine) >= a.pool) atomicOr(&g_kv_fault, kFaultInput);
    const int64_t my_block = block_of(mine);
    unsigned leads = __ballot_sync(kFullMask, my_block >= 0 && my_block != block_of(mine - 1));
    const void *src = half ? a.v : a.k;
    const int64_t stride = half ? a.v_stride : a.k_stride;
    uint8_t *cache = half ? a.v_cache : a.k_cache;
    float *scales = half ? a.v_scales : a.k_scales;
    const int page = 1 << a.page_shift;
    while (leads) {
        const int l = __ffs(leads) - 1;
        leads &= leads - 1;
        const int64_t r = r0 + l, block = __shfl_sync(kFullMask, my_block, l);
        // the rows behind it in the same block
        int64_t count = 0;
        for (;;) {
            const unsigned same = __ballot_sync(kFullMask, block_of(r + count + lane) == block);
            const int n = same == kFullMask ? 32 : __ffs(~same) - 1;
            count += n;
            if (n < 32) break;
        }
        const int64_t first_slot = block * kBlock;
        const int64_t plane = (first_slot >> a.page_shift) * a.n_kv + h;
        const int in_page = static_cast<int>(first_slot & (page - 1));
        uint8_t *rows = cache + (plane * page + in_page) * D + part * E;
        float *scale_at = scales + plane * (page / kBlock) + in_page / kBlock;
        const float old = __ldcg(scale_at);

        const int64_t at0 = r * stride + h * D + part * E;
        const int n0 = static_cast<int>(min(count, static_cast<int64_t>(kBlock)));
        Elems<E, BF16> x[kBlock];
        const int slot = lane < n0 ? __ldcg(a.slots + r + lane) & (kBlock - 1) : -1;
#pragma unroll
        for (int i = 0; i < kBlock; ++i)
            if (i < n0) x[i].load(src, at0 + i * stride);
        uint32_t top = 0;
        unsigned fin = 0, written = 0;
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            if (i < n0) {
                const uint32_t m = x[i].largest();
                const bool f = __all_sync(kFullMask, m < 0x7f800000u);
                if (f) top = max(top, m);
                fin |= static_cast<unsigned>(f) << i;
                written |= 1u << __shfl_sync(kFullMask, slot, i);
            }
        }
        for (int64_t i = kBlock; i < count; ++i) {  // more rows than places: some are named twice
            Elems<E, BF16> y;
            y.load(src, at0 + i * stride);
            const uint32_t m = y.largest();
            if (__all_sync(kFullMask, m < 0x7f800000u)) top = max(top, m);
            written |= 1u << (__ldcg(a.slots + r + i) & (kBlock - 1));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));
        int e = scale_exponent(top);
        // Rows that are there keep their values; offset 0 starts a block afresh.  A scale that no call
        // of this kind left there (not a power of two) is rounded up to one.
        const bool held = !(written & 1u) && old > 0.f && old < INFINITY;
        if (held) {
            const uint32_t b = __float_as_uint(old);
            const int eo = static_cast<int>(b >> 23) - 127 + ((b & 0x7fffffu) != 0);
            e = min(max(e, eo), 127);
        }
        const float scale = power_of_two(e), inv = power_of_two(-e);
        if (held && scale != old) {
            const float ratio = __fdiv_rn(old, scale);
#pragma unroll 4
            for (int i = 0; i < kBlock; ++i) {
                if (written >> i & 1u) continue;
                uint32_t c[E / 4];
#pragma unroll
                for (int j = 0; j < E / 4; ++j) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16x2x2(__ldcg(reinterpret_cast<const uint32_t *>(rows + i * D + 4 * j)), lo, hi);
                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    c[j] = f32x2_to_e4m3x2(p.x * ratio, p.y * ratio) | f32x2_to_e4m3x2(q.x * ratio, q.y * ratio) << 16;
                }
                store_codes<E>(rows + i * D, c);
            }
        }
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            if (i < n0)
                store_row(rows + __shfl_sync(kFullMask, slot, i) * D, x[i], inv, (fin >> i & 1u) != 0, half == 0);
        }
        for (int64_t i = kBlock; i < count; ++i) {
            Elems<E, BF16> y;
            y.load(src, at0 + i * stride);
            const bool f = __all_sync(kFullMask, y.largest() < 0x7f800000u);
            store_row(rows + (__ldcg(a.slots + r + i) & (kBlock - 1)) * D, y, inv, f, half == 0);
        }
        if (part == 0) *scale_at = scale;
    }
}

struct ReadArgs {
    const uint8_t *cache;
    const float *scales;
    const int32_t *slots;
    void *out;
    int64_t n, pool;
    int n_kv, page_shift;
};

// A thread returns 16 values of each of kTurns rows' parts, whose loads are out together: a part's slot, then its codes
// and scale.
constexpr int kTurns = 2;

template <int D, bool BF16>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
    constexpr int P = D / 16;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t parts = a.n * a.n_kv * P;
    const int page = 1 << a.page_shift;
    int64_t at[kTurns], slot[kTurns];
    int head[kTurns];
    uint4 code[kTurns];
    float scale[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        at[t] = (static_cast<int64_t>(blockIdx.x) * kTurns + t) * kReadThreads + threadIdx.x;
        const int64_t row = parts >> 32 ? at[t] / (a.n_kv * P) : static_cast<uint32_t>(at[t]) / static_cast<uint32_t>(a.n_kv * P);
        const int rest = static_cast<int>(at[t] - row * (a.n_kv * P));
        head[t] = rest / P;
        slot[t] = at[t] < parts ? __ldcg(a.slots + row) : -1;
        if (slot[t] >= a.pool) {
            if (rest == 0) atomicOr(&g_kv_fault, kFaultInput);
            slot[t] = -1;
        }
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        code[t] = make_uint4(0, 0, 0, 0);
        scale[t] = 0.f;
        if (slot[t] >= 0) {
            const int in_page = static_cast<int>(slot[t] & (page - 1));
            const int64_t plane = (slot[t] >> a.page_shift) * a.n_kv + head[t];
            code[t] = __ldcg(reinterpret_cast<const uint4 *>(a.cache + (plane * page + in_page) * D) + at[t] % P);
            scale[t] = __ldcg(a.scales + plane * (page / kBlock) + in_page / kBlock);
        }
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        if (at[t] >= parts) continue;
        const uint32_t w[4] = {code[t].x, code[t].y, code[t].z, code[t].w};
        float o[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(w[j], lo, hi);
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            o[4 * j] = x.x * scale[t];
            o[4 * j + 1] = x.y * scale[t];
            o[4 * j + 2] = y.x * scale[t];
            o[4 * j + 3] = y.y * scale[t];
        }
        if (BF16) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.out) + 2 * at[t];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(o[8 * i + 2 * j], o[8 * i + 2 * j + 1]);
                dst[i] = *reinterpret_cast<uint4 *>(b);
            }
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.out) + 4 * at[t];
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
    }
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool sizes_ok(int dtype, int64_t n, int n_kv, int d, int64_t n_pages, int page_size) {
    return (dtype == MEMQ_F32 || dtype == MEMQ_BF16) && n >= 0 && n <= (1 << 24) && n_kv >= 1 && n_kv <= 1024 &&
           (d == 64 || d == 128) && page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0 &&
           n_pages >= 0 && n_pages <= 0x7fffffffLL / page_size / n_kv;
}

template <typename Args>
int launch(void (*kern)(const Args), int64_t ctas, int threads, void *stream, const Args &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}

}  // namespace
}  // namespace memq

// Internal: this translation unit's device fault word (not part of the public header).
int memq_internal_fault_kv(unsigned int *out, bool clear) {
    if (cudaMemcpyFromSymbol(out, memq::g_kv_fault, sizeof(unsigned int)) != cudaSuccess) return 1;
    if (!clear) return 0;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(memq::g_kv_fault, &zero, sizeof(zero)) == cudaSuccess ? 0 : 1;
}

extern "C" int memq_kv_cache_append(int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                    const int32_t *slots, uint8_t *k_cache, float *k_scales, uint8_t *v_cache,
                                    float *v_scales, int64_t n, int n_kv, int d, int64_t n_pages, int page_size,
                                    void *stream) {
    using namespace memq;
    if (!sizes_ok(dtype, n, n_kv, d, n_pages, page_size)) return MEMQ_ERR_SHAPE;
    if (n == 0) return MEMQ_OK;
    const int64_t size = dtype == MEMQ_F32 ? 4 : 2, most = int64_t{1} << 40;
    if (k_stride < 0 || v_stride < 0 || k_stride > most || v_stride > most) return MEMQ_ERR_SHAPE;
    if (!k || !v || !slots || !k_cache || !k_scales || !v_cache || !v_scales) return MEMQ_ERR_NULL;
    if (misaligned(k, 16) || misaligned(v, 16) || (n > 1 && ((k_stride * size) % 16 || (v_stride * size) % 16)) ||
        misaligned(slots, 4) || misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(k_scales, 4) ||
        misaligned(v_scales, 4))
        return MEMQ_ERR_ALIGN;
    // A warp looks for its blocks among 16 rows (a prompt has one or two there), or serves the one row that it
    // has when rows are few: a decode step's rows lie in different blocks, which would wait for one another.  us with one
    // row / 16 rows a warp, 8 kv heads of 128: 256 rows of bf16 in as many blocks 4.5 / 32, of a prompt 4.5 / 4.3; 2048
    // rows 22 / 36 and 10.6 / 6.3; 4096 rows 42 / 37 and 17.5 / 6.7; f32, 2048 rows 40 / 36 and 17.6 / 6.9.
    const int window = n * n_kv <= 16384 ? 1 : kBlock;
    AppendArgs a{k, v, k_stride, v_stride, slots, k_cache, v_cache, k_scales, v_scales, n, n_pages * page_size, n_kv,
                 __builtin_ctz(static_cast<unsigned>(page_size)), window};
    const int64_t units = (n + window - 1) / window * n_kv, ctas = (units + kAppendWarps - 1) / kAppendWarps;
    const bool b = dtype == MEMQ_BF16;
    return launch<AppendArgs>(d == 128 ? (b ? kv_append_kernel<128, true> : kv_append_kernel<128, false>)
                                       : (b ? kv_append_kernel<64, true> : kv_append_kernel<64, false>),
                              ctas, kAppendThreads, stream, a);
}

extern "C" int memq_kv_cache_read(int dtype, const uint8_t *cache, const float *scales, const int32_t *slots, void *out,
                                  int64_t n, int n_kv, int d, int64_t n_pages, int page_size, void *stream) {
    using namespace memq;
    if (!sizes_ok(dtype, n, n_kv, d, n_pages, page_size)) return MEMQ_ERR_SHAPE;
    if (n == 0) return MEMQ_OK;
    if (!cache || !scales || !slots || !out) return MEMQ_ERR_NULL;
    if (misaligned(cache, 16) || misaligned(scales, 4) || misaligned(slots, 4) || misaligned(out, 16))
        return MEMQ_ERR_ALIGN;
    ReadArgs a{cache, scales, slots, out, n, n_pages * page_size, n_kv, __builtin_ctz(static_cast<unsigned>(page_size))};
    const int64_t parts = n * n_kv * (d / 16), ctas = (parts + kTurns * kReadThreads - 1) / (kTurns * kReadThreads);
    if (ctas > 0x7fffffffLL) return MEMQ_ERR_SHAPE;
    const bool b = dtype == MEMQ_BF16;
    return launch<ReadArgs>(d == 128 ? (b ? kv_read_kernel<128, true> : kv_read_kernel<128, false>)
                                     : (b ? kv_read_kernel<64, true> : kv_read_kernel<64, false>),
                            ctas, kReadThreads, stream, a);
}
