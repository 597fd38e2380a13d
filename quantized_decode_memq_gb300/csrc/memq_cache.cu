// memq_cache.cu -- the paged E4M3 latent cache: memq_mla_cache_append quantises rows as it writes
// them, memq_mla_cache_read returns the values that cached rows stand for.
//
// A row is the latent vector and its decoupled position part, side by side, under one f32 scale:
//   scale = max |x| / 448 (the largest E4M3 value),  code = e4m3(x / scale)
// One scale a row serves both parts: E4M3 keeps its relative precision of 2^-4 down to 2^-14 of the
// row's largest, and a single scale lets the attention fold it into the key's weight.
//
// A warp serves a row: a lane holds four consecutive elements of each 128-wide piece, so the row is
// read once and its maximum is one warp reduction.  At 16381 rows of 576 bf16 (they fit in L2) the write
// takes 9.8 us, 2.9 TB/s, and is bound by its divisions (7.4 us without them; codes from a reciprocal need
// a test for the middles between codes and took 11.3); the read takes 7.0 us, 4.1 TB/s, bound by the latency
// of scattered rows.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "memq.h"
#include "memq_dev.cuh"
#include "memq_tc.cuh"

namespace memq {
namespace {

__device__ unsigned int g_cache_fault = 0;
constexpr unsigned int kFaultInput = 32;  // a slot index was outside the pool

constexpr int kCacheThreads = 256;
constexpr int kCacheWarps = kCacheThreads / 32;
constexpr int kMaxPieces = 5;  // 512 latent elements and the position part

template <bool BF16>
__device__ __forceinline__ float4 load4(const void *p, int64_t i) {
    if (BF16) {
        const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i));
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    }
    return __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
}

template <bool BF16>
__global__ void __launch_bounds__(kCacheThreads)
    cache_append_kernel(const void *latent, const void *k_pe, const int32_t *__restrict__ slots, uint8_t *cache,
                        float *scales, int64_t n, int rank, int rope, int64_t pool) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kCacheWarps + (threadIdx.x >> 5);
    if (r >= n) return;
    const int64_t slot = __ldcg(slots + r);
    const int pieces = rank / 128;
    float4 v[kMaxPieces];
    float amax = 0.f;
    bool fin = true;
#pragma unroll
    for (int c = 0; c < kMaxPieces; ++c) {
        v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < pieces) v[c] = load4<BF16>(latent, r * rank + c * 128 + lane * 4);
        if (c == kMaxPieces - 1 && lane * 4 < rope) v[c] = load4<BF16>(k_pe, r * rope + lane * 4);
    }
#pragma unroll
    for (int c = 0; c < kMaxPieces; ++c) {
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v[c].x), fabsf(v[c].y)), fmaxf(fabsf(v[c].z), fabsf(v[c].w))));
        fin = fin && isfinite(v[c].x) && isfinite(v[c].y) && isfinite(v[c].z) && isfinite(v[c].w);
    }
    if (slot < 0) return;  // a padded row
    if (slot >= pool) {
        if (lane == 0) atomicOr(&g_cache_fault, kFaultInput);
        return;
    }
    fin = __all_sync(kFullMask, fin);
    const float scale = __fdiv_rn(warp_max(amax), 448.f);
    const bool zero = !fin || scale == 0.f;
    uint8_t *dst = cache + slot * (rank + rope);
#pragma unroll
    for (int c = 0; c < kMaxPieces; ++c) {
        const bool tail = c == kMaxPieces - 1;
        if (c < pieces || (tail && lane * 4 < rope)) {
            uint32_t code = 0;
            if (!zero)
                code = f32x2_to_e4m3x2(__fdiv_rn(v[c].x, scale), __fdiv_rn(v[c].y, scale)) |
                       f32x2_to_e4m3x2(__fdiv_rn(v[c].z, scale), __fdiv_rn(v[c].w, scale)) << 16;
            *reinterpret_cast<uint32_t *>(dst + (tail ? rank : c * 128) + lane * 4) = code;
        }
    }
    if (lane == 0) scales[slot] = fin ? scale : NAN;
}

template <bool BF16>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const uint8_t *cache, const float *scales, const int32_t *__restrict__ slots, void *out, int64_t n,
                      int width, int64_t pool) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kCacheWarps + (threadIdx.x >> 5);
    if (r >= n) return;
    int64_t slot = __ldcg(slots + r);
    if (slot >= pool) {
        if (lane == 0) atomicOr(&g_cache_fault, kFaultInput);
        slot = -1;
    }
    const float scale = slot >= 0 ? __ldcg(scales + slot) : 0.f;
    const uint8_t *src = cache + slot * width;
    uint32_t code[kMaxPieces];
#pragma unroll
    for (int c = 0; c < kMaxPieces; ++c) {
        const int i = c * 128 + lane * 4;
        code[c] = slot >= 0 && i < width ? __ldcg(reinterpret_cast<const uint32_t *>(src + i)) : 0u;
    }
#pragma unroll
    for (int c = 0; c < kMaxPieces; ++c) {
        const int i = c * 128 + lane * 4;
        if (i >= width) break;
        uint32_t lo, hi;
        e4m3x4_to_f16x2x2(code[c], lo, hi);
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        const float4 o = make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
        if (BF16) {
            __nv_bfloat162 p[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + r * width + i) = *reinterpret_cast<uint2 *>(p);
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(out) + r * width + i) = o;
        }
    }
}

bool rank_ok(int rank) { return rank == 128 || rank == 256 || rank == 512; }
bool rope_ok(int rope) { return rope == 0 || rope == 32 || rope == 64 || rope == 128; }
bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

template <typename K, typename... A>
int launch_rows(K kern, int64_t n, void *stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((n + kCacheWarps - 1) / kCacheWarps));
    cfg.blockDim = dim3(kCacheThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}

bool sizes_ok(int dtype, int64_t n, int kv_rank, int d_rope, int64_t pool) {
    return (dtype == MEMQ_F32 || dtype == MEMQ_BF16) && n >= 0 && n <= 0x7fffffffLL && rank_ok(kv_rank) &&
           rope_ok(d_rope) && pool >= 0 && pool <= 0x7fffffffLL;
}

}  // namespace
}  // namespace memq

// Internal: this translation unit's device fault word (not part of the public header).
int memq_internal_fault_cache(unsigned int *out, bool clear) {
    if (cudaMemcpyFromSymbol(out, memq::g_cache_fault, sizeof(unsigned int)) != cudaSuccess) return 1;
    if (!clear) return 0;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(memq::g_cache_fault, &zero, sizeof(zero)) == cudaSuccess ? 0 : 1;
}

extern "C" int memq_mla_cache_append(int dtype, const void *latent, const void *k_pe, const int32_t *slots,
                                     uint8_t *cache, float *scales, int64_t n, int kv_rank, int d_rope, int64_t pool,
                                     void *stream) {
    using namespace memq;
    if (!sizes_ok(dtype, n, kv_rank, d_rope, pool)) return MEMQ_ERR_SHAPE;
    if (n == 0) return MEMQ_OK;
    if (!latent || (d_rope > 0 && !k_pe) || !slots || !cache || !scales) return MEMQ_ERR_NULL;
    const uintptr_t al = dtype == MEMQ_F32 ? 16 : 8;
    if (misaligned(latent, al) || (d_rope > 0 && misaligned(k_pe, al)) || misaligned(slots, 4) ||
        misaligned(cache, 16) || misaligned(scales, 4))
        return MEMQ_ERR_ALIGN;
    return dtype == MEMQ_BF16
               ? launch_rows(cache_append_kernel<true>, n, stream, latent, k_pe, slots, cache, scales, n, kv_rank, d_rope, pool)
               : launch_rows(cache_append_kernel<false>, n, stream, latent, k_pe, slots, cache, scales, n, kv_rank, d_rope, pool);
}

extern "C" int memq_mla_cache_read(int dtype, const uint8_t *cache, const float *scales, const int32_t *slots,
                                   void *out, int64_t n, int kv_rank, int d_rope, int64_t pool, void *stream) {
    using namespace memq;
    if (!sizes_ok(dtype, n, kv_rank, d_rope, pool)) return MEMQ_ERR_SHAPE;
    if (n == 0) return MEMQ_OK;
    if (!cache || !scales || !slots || !out) return MEMQ_ERR_NULL;
    if (misaligned(out, dtype == MEMQ_F32 ? 16 : 8) || misaligned(slots, 4) || misaligned(cache, 16) ||
        misaligned(scales, 4))
        return MEMQ_ERR_ALIGN;
    const int width = kv_rank + d_rope;
    return dtype == MEMQ_BF16
               ? launch_rows(cache_read_kernel<true>, n, stream, cache, scales, slots, out, n, width, pool)
               : launch_rows(cache_read_kernel<false>, n, stream, cache, scales, slots, out, n, width, pool);
}
