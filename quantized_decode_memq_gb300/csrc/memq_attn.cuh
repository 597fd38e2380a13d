// memq_attn.cuh -- what the kernels of memq_attn_paged share: their arguments, the sequences' sizes, the
// partial results that they leave in the workspace.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "memq.h"
#include "memq_attn_owner.cuh"
#include "memq_dev.cuh"
#include "memq_tc.cuh"

namespace memq {

constexpr unsigned int kAttnFaultWait = 64;   // a bounded wait expired
constexpr unsigned int kAttnFaultInput = 32;  // a length or page index was out of range

namespace {
__device__ unsigned int g_attn_fault = 0;  // (one translation unit includes this)
}

constexpr int kAttnBlock = 16;  // keys that share a scale
constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxCached = 1 << 30;  // rows a sequence
constexpr int kAttnMaxGrid = 256;
constexpr float kAttnUnset = -1e30f;  // a reference before the first visible key
constexpr float kAttnLog2e = 1.4426950408889634f;
// Weights are 2^kAttnTop at the reference: f16 keeps eleven bits of them down to 2^-14 and steps of 2^-24
// below.  The reference moves when a score exceeds it by kAttnSlack (65504 is the largest f16), which costs a pass
// over the accumulators: with a slack of 2 most tiles of a short run had one.
constexpr float kAttnTop = 9.f;
constexpr float kAttnSlack = 6.f;
constexpr float kAttnLeastScale = 0x1p-100f;  // a smaller scale of values counts as this
// Value scales below 2^kAttnLeastLog count as that in the reference.  The sum of weights is of p / vs, each at most
// 2^(kAttnTop + kAttnSlack - kAttnLeastLog) = 2^95: 2^30 of them stay below 2^125, and the reciprocal is a normal number.
// (At -60 weights of rows whose scales are all below 2^-70 lost bits, and from 2^-95 on all of them.)
constexpr float kAttnLeastLog = -80.f;

struct AttnArgs {
    const void *q;
    int64_t q_stride;  // elements from one token's row to the next
    const uint8_t *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int32_t *table, *kv_len, *cu_q;
    void *out;
    AttnOwner *owner;  // one a run
    float2 *stats;     // [2 * run + piece][row] (reference, sum of weights)
    float *part;       // [2 * run + piece][row][d]
    int n_tok, n_seq, nh, n_kv, group, n_pages, page_shift, max_pages;
    int rows_from, rows_to;  // sequences with t * group in this range are served
    int out_bf16;
    int by_item;  // owners are noted by item, not by run
    int behind_tiles;  // the launch before this one is the other kernel's, of the same call
    float scale_log2;
};

struct AttnSeq {
    int start, t, kv;
};

// The sequence's lengths, clamped to what the arrays hold.
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &a, int c0, int c1, int kv) {
    AttnSeq s;
    s.start = min(max(c0, 0), a.n_tok);
    s.t = min(max(c1, s.start), a.n_tok) - s.start;
    s.kv = static_cast<int>(
        min(static_cast<long long>(max(kv, 0)), static_cast<long long>(a.max_pages) << a.page_shift));
    return s;
}

// The pool's row, among all pages and heads, of key `key` of a sequence whose page it lies in.
__device__ __forceinline__ int attn_row(const AttnArgs &a, int page, int head, int key) {
    if (page < 0 || page >= a.n_pages) {
        atomicOr(&g_attn_fault, kAttnFaultInput);
        page = 0;
    }
    return ((page * a.n_kv + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
}

// log2 of a scale, exact for powers of two; not a number or infinite as it is.
__device__ __forceinline__ float attn_log2(float v) {
    const uint32_t bits = __float_as_uint(v);
    const float l = static_cast<float>(static_cast<int>(bits >> 23) - 127) + __log2f(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
    return v < INFINITY ? l : v;
}

// What two f32 have beyond their f16x2.
__device__ __forceinline__ uint32_t attn_rest(float a, float b, uint32_t hi) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return f32x2_to_f16x2(a - h.x, b - h.y);
}

// out element offset of row `rr` of a (sequence, kv head).
__device__ __forceinline__ int64_t attn_out_at(const AttnArgs &a, int start, int head, int rr, int d) {
    const int tok = rr / a.group;
    return ((static_cast<int64_t>(start) + tok) * a.nh + head * a.group + (rr - tok * a.group)) * d;
}

}  // namespace memq
