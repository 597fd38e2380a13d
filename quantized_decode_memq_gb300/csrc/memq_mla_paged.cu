// memq_mla_paged.cu -- memq_mla_attn_paged: causal attention of a chunk of new tokens per
// sequence over a paged E4M3 latent cache, queries and outputs in the latent space.
//
//   s_j  = scale * scales_j * (q . codes_j)            j <= position of the query's token
//   out  = sum_j softmax(s)_j * scales_j * codes_j[:kv_rank]
//
// All heads read one latent vector per cached token, so a tile of 64 query rows (heads of one
// token, or heads x tokens when there are few heads) shares every key.  The products are formed
// transposed,
//   S^T [128 keys x 64 rows]  = C [128 x width] . Q^T
//   O^T [kv_rank x 64 rows]  += C[:, :kv_rank]^T [kv_rank x 128] . P^T
// because the f32 accumulator of 64 rows then takes kv_rank / 128 x 64 TMEM columns (256 of 512
// at rank 512) and both products read the cache's codes as they lie in memory: the same TMA-loaded
// tile is the K-major A operand of the first product and the MN-major A operand of the second, with
// no conversion or transposition in between.
//
// kind::f8f6f4 multiplies 8-bit operands exactly and adds in f32, so the operands that are not
// codes are sums of two 8-bit terms, each with its own product into the same accumulator (twice
// the operations at twice the 16-bit rate), or of three:
//   q = 2^e (hi + lo), both E4M3, e per row: a bf16 value exactly down to 2^-10 of the row's largest,
//       below that an absolute 2^-17 of it.  Of an f32 query hi + mid (E4M3) + lo (E5M2): its f16 form, 2^-11,
//       down to 2^-10 of the largest, an absolute 2^-20 below.
//   p = hi (E4M3) + lo (E5M2), with p in (0, 2^8.8] and 8 at the reference: a relative 1.13 x 2^-8 at most
//       (about 2^-9.6 rms) down to 2^-6, an absolute 2^-14 below that, steps of 2^-16 from 2^-14 on, and
//       0 below 2^-17: E5M2 carries small weights that a second E4M3 term would flush.  For f32 outputs a third
//       term, E5M2 too: a relative 2^-11 down to 2^-6, an absolute 2^-17 below.
//   8 sequences of 8 tokens over 8192 rows (rank 512, rope 64), us: bf16 85, f32 outputs 119, f32 queries 128,
//   both 145; relative error of 2048 rows against 64 bits with both 3.5e-4.
// The codes are bit fields of f16 numbers: E4M3 of v is bits 14..7 of f16(v / 256), E5M2 of v the high byte
// of f16(v), so a split needs one conversion per pair of numbers and integer operations.
// The key's scale is folded into its weight (p_j = 2^8 exp2(s_j + log2 scales_j - R - 7)), so R, the
// running reference, bounds what the 8-bit terms must hold; the sum of weights is kept apart in f32.
// R moves, and the accumulators are rescaled, only when a score exceeds it by 5.8, so that a tile needs one
// vote instead of 64 maxima over its keys, or when a look at a tile's codes finds a query all of whose
// weights are below 2^-8: thousands of small weights behind one large one (a sink) carry a part of the
// sum that must not be lost.  The f32 accumulators take a reference that comes down as well as one that
// goes up.  The look comes two tiles after a reference went up far, and every 16 tiles.
//
// One CTA per SM.  The 128-key tiles of all (sequence, token group, head block) items form one list
// that is cut into equal runs, one per CTA; every CTA derives its run from the lengths on the device
// (nothing of the plan is on the host, so a captured graph serves other lengths).  An item that
// spans CTAs leaves f32 partial accumulators in the workspace, and combine_kernel adds them in CTA
// order: results do not depend on timing.  Starting an item (its queries, the first tile's references,
// the accumulators' way out) costs as much as several tiles and counts as
// kStart tiles in the list.
//
// Warps 0-7 are the softmax warps (thread = key x half of the columns), warp 8 issues the TMA copies
// of 128 x 128-byte pieces into a ring, one thread of warp 9 the products.  S^T is double buffered: the
// scores of tile i + 1 are computed while the softmax of tile i runs.
//
// Shared memory's bandwidth bounds a tile: an m128 product of 32-byte rows reads 4 KB of codes and 32
// bytes per column at 128 bytes a cycle (48 cycles at n = 64, where the arithmetic takes 32; 64 at n =
// 128, where both do).  So both query terms are one product of 128 columns, S_hi and S_lo, which the
// softmax warps add; the accumulators of the outputs leave no room in TMEM for the same there.  At
// rank 512, rope 64: 18 x 64 + 32 x 48 cycles, and 576 for the copies that fill the ring; a tile takes
// 3480.  64 heads, rank 512, rope 64, bf16: 2048 new tokens over 8192 rows 1.69 ms, 1.21 PFLOP/s (62% of the
// bf16 peak; moves of the references take 0.1 ms of it); 48 single tokens over up to 16384 rows 89 us, 4.9 TB/s
// once it runs, of which starts and partial accumulators take 30; 8 tokens over 32768 rows 49 us.
//
// Codes of a cached row are finite by the cache's contract (a row that was not finite carries a
// NaN scale); rows past the end of a sequence may hold anything and are zeroed in shared memory
// before the second product, whose zero weights would otherwise meet NaN codes.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "memq.h"
#include "memq_dev.cuh"
#include "memq_phases.cuh"
#include "memq_tc.cuh"

namespace memq {
namespace {

__device__ unsigned int g_paged_fault = 0;
constexpr unsigned int kFaultWait = 16;   // a bounded wait expired
constexpr unsigned int kFaultInput = 32;  // a length or page index was out of range

constexpr int kRows = 64;       // query rows per tile
constexpr int kKeys = 128;      // keys per tile
constexpr int kPiece = 16384;   // bytes of one 128 x 128 ring slot
constexpr int kMaxSlots = 12;
constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 10 * 32;
constexpr int kMaxSeqs = 4096;
constexpr int kMaxGrid = 256;
constexpr int kMaxCached = 1 << 30;  // rows a sequence: key indices rounded up to a tile stay in 31 bits
constexpr float kLog2e = 1.4426950408889634f;
// Tiles that starting an item counts as (us, 0 / 3 / 6 / 9: 8 tokens over 32768 rows 63 / 56 / 53 / 53, 48
// single tokens 103 / 95 / 92 / 94; rank 256, whose tiles are shorter, is best at 4 to 5).
constexpr int kStart = 5;
constexpr float kUnset = -1e30f;  // the reference before the first visible key
// log2 of how far a score may exceed the reference, before kOver more: weights end at 2^8.8, E4M3's largest is
// 448.  Less slack keeps more bits of small weights and moves the references more often (2048 tokens over 8192
// rows, slack 4 / 5 / 6 us: 1737 / 1707 / 1676; wider scores cost more, twice as wide 2140, at 7 without
// looks 1780).
constexpr float kSlack = 5.0f;
constexpr float kOver = 0.8f;
// References come down on a look, to a tile's maxima that lie more than kKeep (log2) below them, but no more
// than kDepth below the highest that they were: the sums' range, and less than 2^-36 of the largest weight
// lost there.  Tiles between two looks, 8 / 16: 1721 / 1707 us, 1614 without any.
constexpr int kLook = 16;
constexpr float kKeep = 4.0f;
constexpr float kDepth = 16.0f;
constexpr float kJump = 0x1p-8f;  // a reference that went up by 8 calls for a look: codes keep 2^-8 above that
constexpr float kLeastScale = 0x1p-64f;  // smaller scales of a row count as this in the outputs
constexpr int kScoreCol = 256;    // TMEM: accumulators in columns 0..255, scores after them

// An item that several CTAs share, noted by the CTA that holds its start (`rows` is 0 otherwise).
struct __align__(16) Owner {
    long long row0;      // first output row
    unsigned char rows;  // 1 to 64
    unsigned char tail;  // its first partial is slot 2 cta + tail; the others are slots 2 c of the
    short last;          // CTAs c up to this one
    int pad;
};
static_assert(sizeof(Owner) == 16, "one load");

struct PagedArgs {
    const void *q_lat, *q_pe;
    const float *scales;
    const int32_t *table, *kv_len, *cu_q;
    void *out;
    Owner *owner;
    float2 *stats;  // [slot][row] (reference, sum of weights)
    float *part;    // [slot][row][rank]
    int n_tok, n_seq, nh, rank, rope, n_pages, page_shift, box, max_pages;
    int group;  // tokens per item
    int heads_per, head_blocks;
    int slots;
    int out_bf16;
    float scale_log2;
};

struct Item {
    int seq, start, t, kv;  // sequence, its first token row, new tokens, cached rows
    int tok, block;         // first token of the group, head block
    int vis, tiles;         // keys that its last token sees, tiles
};

struct Control {
    uint32_t tops[kRows];  // column maxima of a tile (order_bits); 0 between uses
    float ref[kRows], peak[kRows];  // the columns' references, the highest that they were
    alignas(16) uint32_t near[kSoftmaxWarps];  // bit 8 (c % 4) + c / 4: column c has a weight of 2^-8 or more
    float row_scale[kRows];
    alignas(16) float shrink[kRows], minus[kRows];  // what a move of the references means to a column
    uint64_t full[kMaxSlots], freed[kMaxSlots];
    uint64_t rope_full, rope_free, scale_full[2], scale_free[2], score_full[2];
    uint64_t weights_ready, out_done, q_ready, drain;
    uint32_t tmem;
    int first_off;
    Item first;  // of the run
    Item next;   // after the softmax warps' current one
    long long first_pos;
    long long warp_sum[kThreads / 32];
};
static_assert(sizeof(Control) <= 2048, "the control block has 2 KB of shared memory");

// Shared memory, from a 1024-byte boundary: Q terms (per 128 latent dims hi, lo; rope hi, lo; of f32 queries the third
// terms, per 128 latent dims and rope), P terms, the rope piece, the ring, the scales of two tiles, the control block.
__host__ __device__ constexpr int smem_weights_off(bool q3, int rank, int rope) { return (q3 ? 3 : 2) * kRows * (rank + rope); }
__host__ __device__ constexpr int smem_ring_off(bool q3, bool p3, int rank, int rope) {
    return smem_weights_off(q3, rank, rope) + (p3 ? 3 : 2) * kKeys * kRows + kKeys * rope;
}
__host__ __device__ constexpr int smem_tail() { return 2 * kKeys * 4 + 2048; }

__device__ __forceinline__ void item_sizes(const PagedArgs &a, Item &it) {
    const int last = min(it.tok + a.group, it.t) - 1;
    it.vis = max(0, min(it.kv, it.kv - it.t + last + 1));
    it.tiles = max(1, (it.vis + kKeys - 1) / kKeys);
}

// The sequence's lengths, clamped to what the arrays hold.
__device__ __forceinline__ void seq_sizes(const PagedArgs &a, int c0, int c1, int kv, Item &it) {
    it.start = min(max(c0, 0), a.n_tok);
    it.t = min(max(c1, it.start), a.n_tok) - it.start;
    it.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)),
                                 static_cast<long long>(a.max_pages) << a.page_shift));
}

__device__ __forceinline__ void next_item(const PagedArgs &a, Item &it) {
    if (++it.block < a.head_blocks) return;
    it.block = 0;
    it.tok += a.group;
    if (it.tok >= it.t) {
        it.tok = 0;
        do {
            if (++it.seq >= a.n_seq) {  // not with offsets that stand still: an item without rows and keys
                it.seq = a.n_seq;
                it.t = it.kv = 0;
                break;
            }
            seq_sizes(a, __ldcg(a.cu_q + it.seq), __ldcg(a.cu_q + it.seq + 1), __ldcg(a.kv_len + it.seq), it);
        } while (it.t == 0);
    }
    item_sizes(a, it);
}

// The item's rows of q and out: consecutive (token, head) rows.
__device__ __forceinline__ int64_t item_row0(const PagedArgs &a, const Item &it) {
    return (static_cast<int64_t>(it.start) + it.tok) * a.nh + it.block * a.heads_per;
}
__device__ __forceinline__ int item_rows(const PagedArgs &a, const Item &it) {
    if (it.tok >= it.t) return 0;
    return a.head_blocks > 1 ? min(a.heads_per, a.nh - it.block * a.heads_per) : min(a.group, it.t - it.tok) * a.nh;
}

// x / y of non-negative numbers; a 64-bit division costs some 500 cycles.
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}

// Waits for a barrier phase; after one wait expired, none is made any more, and the fault word says so.
// A warp whose wait expired frees no buffer any more, so that nothing is announced on a barrier whose last
// phase is not over: the copies stop and what is in flight is awaited, the products stop, and the softmax
// warps run to their end on whatever is there.
struct Waiter {
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        if (!dead && !warp_wait_bounded(bar, parity)) {
            dead = true;
            if ((threadIdx.x & 31) == 0) atomicOr(&g_paged_fault, kFaultWait);
        }
    }
};

// The same for a single thread.
struct ThreadWaiter {
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        if (dead || mbar_try_wait(bar, parity)) return;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (clock64() - t0 > kWaitCycles) {
                dead = true;
                atomicOr(&g_paged_fault, kFaultWait);
                return;
            }
        }
    }
};

__device__ __forceinline__ void prefetch_l2(const uint8_t *p, int64_t bytes, int lane) {
    for (int64_t i = lane * 128; i < bytes; i += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
}

// Byte offset of element `i` of row `r` in an operand of `row_bytes`-byte swizzled rows.
__device__ __forceinline__ int swizzled(int r, int i, int row_bytes) {
    const int x = row_bytes == 128 ? r & 7 : row_bytes == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
    return r * row_bytes + (i ^ (x << 4));
}

// E4M3 codes of 256 times the four f16 numbers in (-2, 2) of a and b, which have at most three
// fraction bits: bits 13..7 behind the sign.
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t a, uint32_t b) {
    return __byte_perm(a << 1, b << 1, 0x7531) | (__byte_perm(a, b, 0xfdb9) & 0x80808080u);
}

// Of four codes of weights, a bit 0 in the place of each that is 2^-8 or more (code 4).
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return (w + 0x7c7c7c7cu) >> 7 & 0x01010101u; }

// Byte offset of element `e` of row r in the hi terms, and how far behind its lo term lies: the lo terms
// are rows 64 to 127 of the same operand.
__device__ __forceinline__ int q_lat_at(int r, int e) { return (e >> 7) * (2 * kRows * 128) + swizzled(r, e & 127, 128); }
__device__ __forceinline__ int q_pe_at(const PagedArgs &a, int r, int e) { return 2 * a.rank * kRows + swizzled(r, e, a.rope); }
constexpr int kLatLo = kRows * 128;
// The same of the third terms.
__device__ __forceinline__ int q3_lat_at(const PagedArgs &a, int r, int e) {
    return 2 * kRows * (a.rank + a.rope) + (e >> 7) * (kRows * 128) + swizzled(r, e & 127, 128);
}
__device__ __forceinline__ int q3_pe_at(const PagedArgs &a, int r, int e) {
    return 2 * kRows * (a.rank + a.rope) + a.rank * kRows + swizzled(r, e, a.rope);
}

// 256 times the two f16 numbers of a, which are small enough; E5M2 codes of the four of a and b, the high
// bytes of which are rounded.
__device__ __forceinline__ uint32_t times256(uint32_t a) { return mul_f16x2(a, 0x5c005c00u); }
__device__ __forceinline__ uint32_t e5m2_bits(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }
// To the nearest multiple of three fraction bits.
__device__ __forceinline__ uint32_t round3(uint32_t f) { return (f + 0x00400040u) & 0xff80ff80u; }

// hi and lo terms of four query elements, given as two pairs of f16 in (-1, 1].
__device__ __forceinline__ void split4(uint32_t f0, uint32_t f1, uint32_t &hi, uint32_t &lo) {
    const uint32_t h0 = round3(f0), h1 = round3(f1);
    hi = e4m3_bits(h0, h1);
    lo = e4m3_bits(sub_f16x2(f0, h0) + 0x00400040u, sub_f16x2(f1, h1) + 0x00400040u);
}
// Three terms hold the eleven bits of an f16 number exactly, four, four and three of them, down to 2^-10.
__device__ __forceinline__ void split4(uint32_t f0, uint32_t f1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const uint32_t h0 = round3(f0), h1 = round3(f1), r0 = sub_f16x2(f0, h0), r1 = sub_f16x2(f1, h1);
    const uint32_t m0 = round3(r0), m1 = round3(r1);
    hi = e4m3_bits(h0, h1);
    mid = e4m3_bits(m0, m1);
    lo = e5m2_bits(times256(sub_f16x2(r0, m0)) + 0x00800080u, times256(sub_f16x2(r1, m1)) + 0x00800080u);
}
__device__ __forceinline__ uint32_t scaled_pair(uint32_t a, uint32_t b, uint64_t by) {
    const float2 x = unpack2(mul2(bits2(a, b), by));
    return f32x2_to_f16x2(x.x, x.y);
}
__device__ __forceinline__ uint32_t scaled_bf16(uint32_t w, uint64_t by) { return scaled_pair(w << 16, w & 0xffff0000u, by); }

// Eight bf16, parked in the places of their terms -> the terms.
__device__ __forceinline__ void split_parked(uint8_t *hi, uint8_t *lo, uint64_t by) {
    uint2 *h = reinterpret_cast<uint2 *>(hi), *l = reinterpret_cast<uint2 *>(lo);
    const uint2 w0 = *h, w1 = *l;
    uint2 th, tl;
    split4(scaled_bf16(w0.x, by), scaled_bf16(w0.y, by), th.x, tl.x);
    split4(scaled_bf16(w1.x, by), scaled_bf16(w1.y, by), th.y, tl.y);
    *h = th;
    *l = tl;
}
__device__ __forceinline__ void split_f32(uint8_t *hi, uint8_t *mid, uint8_t *lo, uint4 v, uint64_t by) {
    split4(scaled_pair(v.x, v.y, by), scaled_pair(v.z, v.w, by), *reinterpret_cast<uint32_t *>(hi),
           *reinterpret_cast<uint32_t *>(mid), *reinterpret_cast<uint32_t *>(lo));
}

// Maxima of |x| as bits: infinities and NaN lie above all numbers.
__device__ __forceinline__ __nv_bfloat162 max_bf16(__nv_bfloat162 m, uint4 v) {
    const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&v);
    return __hmax2_nan(__hmax2_nan(m, __hmax2_nan(__habs2(x[0]), __habs2(x[1]))),
                       __hmax2_nan(__habs2(x[2]), __habs2(x[3])));
}
__device__ __forceinline__ uint32_t max_f32(uint32_t m, uint4 v) {
    return max(max(m, v.x & 0x7fffffffu), max(v.y & 0x7fffffffu, max(v.z & 0x7fffffffu, v.w & 0x7fffffffu)));
}

// What a row's largest |x| (its upper 16 bits) makes of it: 2^e with max / 2^e in [1/2, 1) is divided out.
// Tiny rows keep a normal reciprocal; a row that is not finite, or past 2^126, gets a NaN scale, and
// what its codes hold then does not matter to the others.
__device__ __forceinline__ uint64_t row_factor(uint32_t top, float &scale) {
    const int e = min(max(static_cast<int>(top >> 7), 32), 252);
    scale = top < 0x7e80u ? __uint_as_float(static_cast<uint32_t>(e - 7) << 23) : NAN;
    const float inv = __uint_as_float(static_cast<uint32_t>(253 - e) << 23);
    return pack2(inv, inv);
}
__device__ __forceinline__ uint32_t max_of8(uint32_t v) {  // over the 8 lanes of a row
    v = max(v, __shfl_xor_sync(kFullMask, v, 1));
    v = max(v, __shfl_xor_sync(kFullMask, v, 2));
    return max(v, __shfl_xor_sync(kFullMask, v, 4));
}

// The 64 query rows of an item -> their 8-bit terms and scales in shared memory; rows past `rows` are
// zeros.  Eight lanes read 128 consecutive bytes of a row; a lane serves rows r and r + 1.  Two passes,
// for the row's maximum comes first.  Eight bf16 fill the 8 + 8 bytes of their terms, so the first pass
// parks them there and the second splits them in place; f32 queries are read a second time, from L2.
// Many loads are out at once and the code stays short: unrolled over registers it was half the kernel,
// and fetching it took longer than running it.  On the first item the producer starts its copies when
// the first loads are out; behind a ring of cache rows in the memory's queues they took 10 us and more.
__device__ __forceinline__ void stage_bf16(const PagedArgs &a, Control *ctl, uint8_t *smem, int64_t row0, int rows, int r,
                                           int q, bool first) {
    const int pieces = a.rank / 128;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 v[2][4][2], w[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const bool live = r + k < rows;
        const int64_t row = row0 + r + k;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q_lat) + row * a.rank) + q;
        const uint4 *pe = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q_pe) + row * a.rope) + q;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) v[k][c][j] = live && c < pieces ? __ldcg(src + c * 16 + j * 8) : zero;
#pragma unroll
        for (int j = 0; j < 2; ++j) w[k][j] = live && (q + 8 * j) * 8 < a.rope ? __ldcg(pe + j * 8) : zero;
    }
    if (first) named_bar_arrive(4, kSoftmaxWarps * 32 + 32);
    uint64_t by[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int rk = r + k;
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint8_t *at = smem + swizzled(rk, (q + 8 * j) * 8, 128);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c < pieces) {
                    top = max_bf16(top, v[k][c][j]);
                    uint8_t *hi = at + c * (2 * kRows * 128);
                    *reinterpret_cast<uint2 *>(hi) = make_uint2(v[k][c][j].x, v[k][c][j].y);
                    *reinterpret_cast<uint2 *>(hi + kLatLo) = make_uint2(v[k][c][j].z, v[k][c][j].w);
                }
            }
            if ((q + 8 * j) * 8 < a.rope) {
                top = max_bf16(top, w[k][j]);
                uint8_t *hi = smem + q_pe_at(a, rk, (q + 8 * j) * 8);
                *reinterpret_cast<uint2 *>(hi) = make_uint2(w[k][j].x, w[k][j].y);
                *reinterpret_cast<uint2 *>(hi + kRows * a.rope) = make_uint2(w[k][j].z, w[k][j].w);
            }
        }
        const uint32_t t = *reinterpret_cast<const uint32_t *>(&top);
        float scale;
        by[k] = row_factor(max_of8(max(t & 0x7fffu, (t >> 16) & 0x7fffu)), scale);
        if (q == 0) ctl->row_scale[rk] = scale;
    }
    int at[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) at[k][j] = swizzled(r + k, (q + 8 * j) * 8, 128);
#pragma unroll 1
    for (int c = 0; c < pieces; ++c) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint8_t *hi = smem + c * (2 * kRows * 128) + at[k][j];
                split_parked(hi, hi + kLatLo, by[k]);
            }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (int u = q; u * 8 < a.rope; u += 8) {
            uint8_t *hi = smem + q_pe_at(a, r + k, u * 8);
            split_parked(hi, hi + kRows * a.rope, by[k]);
        }
}

__device__ __forceinline__ void stage_f32(const PagedArgs &a, Control *ctl, uint8_t *smem, int64_t row0, int rows, int r,
                                          int q, bool first) {
    const int pieces = a.rank / 128;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 *src[2], *pe[2];
    bool live[2];
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        live[k] = r + k < rows;
        const int64_t row = row0 + r + k;
        src[k] = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q_lat) + row * a.rank) + q;
        pe[k] = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q_pe) + row * a.rope) + q;
    }
#pragma unroll 1
    for (int c = 0; c < pieces; c += 2) {
        uint4 v[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = live[k] && c + (j >> 2) < pieces ? __ldcg(src[k] + c * 32 + j * 8) : zero;
        if (first) named_bar_arrive(4, kSoftmaxWarps * 32 + 32);
        first = false;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) top[k] = max_f32(top[k], v[k][j]);
    }
    for (int u = q; u * 4 < a.rope; u += 8) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (live[k]) top[k] = max_f32(top[k], __ldcg(pe[k] + (u - q)));
    }
    uint64_t by[2];
    uint4 v[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float scale;
        by[k] = row_factor(max_of8(top[k]) >> 16, scale);
        if (q == 0) ctl->row_scale[r + k] = scale;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[k][j] = live[k] ? __ldcg(src[k] + j * 8) : zero;
    }
#pragma unroll 1
    for (int c = 0; c < pieces; ++c) {
        uint4 next[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                next[k][j] = live[k] && c + 1 < pieces ? __ldcg(src[k] + (c + 1) * 32 + j * 8) : zero;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = c * 128 + (q + 8 * j) * 4;
                uint8_t *hi = smem + q_lat_at(r + k, e);
                split_f32(hi, hi + kLatLo, smem + q3_lat_at(a, r + k, e), v[k][j], by[k]);
                v[k][j] = next[k][j];
            }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (int u = q; u * 4 < a.rope; u += 8) {
            uint8_t *hi = smem + q_pe_at(a, r + k, u * 4);
            split_f32(hi, hi + kRows * a.rope, smem + q3_pe_at(a, r + k, u * 4),
                      live[k] ? __ldcg(pe[k] + (u - q)) : zero, by[k]);
        }
}

template <bool F32>
__device__ __forceinline__ void stage_q(const PagedArgs &a, Control *ctl, uint8_t *smem, int64_t row0, int rows,
                                        int tid, bool first) {
    // rows r and r + 1; the warp's other rows lie 2 and 4 apart, so that the swizzle keeps them off
    // each other's banks
    const int r = (tid >> 5) * 8 + ((tid >> 3) & 1) * 4 + ((tid >> 4) & 1) * 2, q = tid & 7;
    if (F32)
        stage_f32(a, ctl, smem, row0, rows, r, q, first);
    else
        stage_bf16(a, ctl, smem, row0, rows, r, q, first);
}

// Sum over the 32 lanes of v[c], for every c, in lane c (a fixed tree).
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = (lane & o) != 0;
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(kFullMask, send, o);
        }
    }
    return v[0];
}

// Maximum over the 32 lanes of v[c], for every c, in lane c.
__device__ __forceinline__ float column_maxima(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = (lane & o) != 0;
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = fmaxf(keep, __shfl_xor_sync(kFullMask, send, o));
        }
    }
    return v[0];
}

// Q3: f32 queries, three terms of them.  P3: f32 outputs, three terms of the weights.
template <bool Q3, bool P3>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap map_lat, const __grid_constant__ CUtensorMap map_rope,
                      const PagedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFullMask, tid >> 5, 0);  // uniform
    const int pieces = a.rank / 128;
    uint8_t *weights = smem + smem_weights_off(Q3, a.rank, a.rope);
    uint8_t *ring = smem + smem_ring_off(Q3, P3, a.rank, a.rope);
    uint8_t *rope_k = ring - kKeys * a.rope;
    float *tile_scale = reinterpret_cast<float *>(ring + a.slots * kPiece);
    Control *ctl = reinterpret_cast<Control *>(tile_scale + 2 * kKeys);

    griddep_launch_dependents();
    if (tid == 0) {
        tma_prefetch_map(&map_lat);
        if (a.rope) tma_prefetch_map(&map_rope);
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->freed[i], 1);
        }
        mbar_init(&ctl->rope_full, 1);
        mbar_init(&ctl->rope_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->scale_full[i], 1);
            mbar_init(&ctl->scale_free[i], kSoftmaxWarps);
            mbar_init(&ctl->score_full[i], 1);
        }
        mbar_init(&ctl->weights_ready, kSoftmaxWarps);
        mbar_init(&ctl->out_done, 1);
        mbar_init(&ctl->q_ready, kSoftmaxWarps);
        mbar_init(&ctl->drain, 1);
        mbar_init_fence();
    }
    if (tid < kRows) ctl->tops[tid] = 0;
    if (warp == kMmaWarp) tmem_alloc(&ctl->tmem, 512);
    griddep_wait();

    // ------------------------------------------------------------------ this CTA's run of tiles
    int32_t *cu = reinterpret_cast<int32_t *>(ring), *kvl = cu + a.n_seq + 1;
    bool descends = false;
    for (int i = tid; i <= a.n_seq; i += kThreads) {
        const bool seq = i < a.n_seq;
        const int c0 = __ldcg(a.cu_q + i), c1 = seq ? __ldcg(a.cu_q + i + 1) : a.n_tok;
        const int kv = seq ? __ldcg(a.kv_len + i) : 0;
        cu[i] = c0;
        if (seq) kvl[i] = kv;
        if (c0 < 0 || c0 > c1 || kv < 0 || kv > (static_cast<long long>(a.max_pages) << a.page_shift))
            atomicOr(&g_paged_fault, kFaultInput);
        descends = descends || (seq && c0 > c1);
    }
    // Offsets that descend would name tokens again and again, n_seq / 2 times at worst: nothing is done then.
    const int n_seq = __syncthreads_or(descends) ? 0 : a.n_seq;
    // Thread i counts the tiles of the groups whose last token lies in its slice of the tokens.
    const int slice = (a.n_tok + kThreads - 1) / kThreads;
    const int tok_lo = min(a.n_tok, tid * slice), tok_hi = min(a.n_tok, tok_lo + slice);
    int seq0 = 0;
    {
        int hi = n_seq;  // first sequence that ends after tok_lo
        while (seq0 < hi) {
            const int mid = (seq0 + hi) >> 1;
            if (cu[mid + 1] <= tok_lo) seq0 = mid + 1; else hi = mid;
        }
    }
    long long run_lo = -1, run_hi = 0, per = 0;
    long long before = 0, own = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        long long sum = before;  // pass 0: this slice's tiles; pass 1: find the run's first tile
        if (pass == 1 && (run_lo < before || run_lo >= before + own)) break;
        Item it{};
        for (it.seq = seq0; it.seq < n_seq && cu[it.seq] < tok_hi; ++it.seq) {
            seq_sizes(a, cu[it.seq], cu[it.seq + 1], kvl[it.seq], it);
            const int k0 = max(tok_lo - it.start, 0), k1 = min(tok_hi - it.start, it.t);
            for (it.tok = a.group == 1 ? k0 : k0 / a.group * a.group; min(it.tok + a.group, it.t) <= k1 && it.tok < it.t;
                 it.tok += a.group) {
                item_sizes(a, it);
                const int units = it.tiles + kStart;
                const long long n = static_cast<long long>(units) * a.head_blocks;
                if (pass == 1 && sum <= run_lo && run_lo < sum + n) {
                    const int at = static_cast<int>(run_lo - sum);  // less than 2^25 units x 16 blocks
                    it.block = a.head_blocks == 1 ? 0 : at / units;
                    const int off = max(0, at - it.block * units - kStart);
                    ctl->first = it;
                    ctl->first_off = off;
                    ctl->first_pos = sum + it.block * units + kStart + off;
                }
                sum += n;
            }
        }
        if (pass == 0) {
            long long incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(kFullMask, incl, o);
                if (lane >= o) incl += up;
            }
            if (lane == 31) ctl->warp_sum[warp] = incl;
            __syncthreads();
            own = sum;
            before = incl - sum;
            long long total = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += ctl->warp_sum[w];
                total += ctl->warp_sum[w];
            }
            per = quotient(total + gridDim.x - 1, gridDim.x);
            run_lo = blockIdx.x * per;
            run_hi = min(total, run_lo + per);
        }
    }
    fence_async_smem();  // the lengths lie where TMA will write
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, ctl->tmem, 0);
    const long long run_first = run_lo < run_hi ? ctl->first_pos : run_hi;  // of the run's first tile

    if (run_first < run_hi) {
        Item it = ctl->first;
        int off = ctl->first_off;
        Waiter wait;

        if (warp == kLoadWarp) {
            // ---------------------------------------------------------------- TMA producer
            CopyPhases sent;
            const uint32_t slots = static_cast<uint32_t>(a.slots);
            const int per_tile = kKeys / a.box;
            named_bar_sync(4, kSoftmaxWarps * 32 + 32);  // the first query rows' loads are out
            for (long long pos = run_first; pos < run_hi && !wait.dead;) {
                const int n = static_cast<int>(min(static_cast<long long>(it.tiles - off), run_hi - pos));
                const int32_t *table = a.table + static_cast<int64_t>(it.seq) * a.max_pages;
                const auto page_row = [&](int key0) {  // row of this lane's box in the pool
                    const int key = key0 + lane * a.box;
                    if (lane >= per_tile || key >= it.vis) return -1;
                    int page = __ldcg(table + (key >> a.page_shift));
                    if (page < 0 || page >= a.n_pages) {
                        atomicOr(&g_paged_fault, kFaultInput);
                        page = 0;
                    }
                    return (page << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                };
                int row = page_row(off * kKeys);
                for (int i = off; i < off + n; ++i) {
                    const int row_next = i + 1 < off + n ? page_row((i + 1) * kKeys) : -1;
                    const bool mine = row >= 0;
                    const uint32_t boxes = __popc(__ballot_sync(kFullMask, mine));
                    // scales of the tile's keys
                    const uint32_t buf = sent.scales & 1;
                    if (sent.scales >= 2) wait(&ctl->scale_free[buf], last_parity(sent.scales >> 1));
                    if (wait.dead) break;
                    if (lane == 0) mbar_arrive_expect_tx(&ctl->scale_full[buf], boxes * a.box * 4);
                    __syncwarp();
                    if (mine) bulk_g2s_plain(tile_scale + buf * kKeys + lane * a.box, a.scales + row, a.box * 4, &ctl->scale_full[buf]);
                    ++sent.scales;
                    if (a.rope) {
                        if (sent.ropes >= 1) wait(&ctl->rope_free, last_parity(sent.ropes));
                        if (wait.dead) break;
                        if (lane == 0) mbar_arrive_expect_tx(&ctl->rope_full, boxes * a.box * a.rope);
                        __syncwarp();
                        if (mine)
                            tma_load_2d_plain(rope_k + lane * a.box * a.rope, &map_rope, a.rank, row, &ctl->rope_full);
                        ++sent.ropes;
                    }
                    for (int c = 0; c < pieces; ++c) {
                        const uint32_t slot = sent.slot;
                        if (sent.lap >= 1) wait(&ctl->freed[slot], last_parity(sent.lap));
                        if (wait.dead) break;
                        if (lane == 0) mbar_arrive_expect_tx(&ctl->full[slot], boxes * a.box * 128);
                        __syncwarp();
                        if (mine)
                            tma_load_2d_plain(ring + slot * kPiece + lane * a.box * 128, &map_lat, c * 128, row,
                                              &ctl->full[slot]);
                        sent.piece_announced(slots);
                    }
                    if (wait.dead) break;
                    row = row_next;
                }
                pos += n + kStart;
                off = 0;
                if (pos < run_hi && !wait.dead) {
                    next_item(a, it);
                    // The softmax warps are about two tiles behind: the next query rows come into L2.
                    const int64_t row0 = item_row0(a, it);
                    const int64_t size = Q3 ? 4 : 2, rows = item_rows(a, it);
                    prefetch_l2(static_cast<const uint8_t *>(a.q_lat) + row0 * a.rank * size, rows * a.rank * size, lane);
                    if (a.rope) prefetch_l2(static_cast<const uint8_t *>(a.q_pe) + row0 * a.rope * size, rows * a.rope * size, lane);
                }
            }
            if (wait.dead) {
                // Copies in flight: the last phase that was announced on every barrier, each wait bounded.
                for (uint32_t s = 0; s < slots; ++s)
                    if (sent.pieces_in(s)) (void)warp_wait_bounded(&ctl->full[s], last_parity(sent.pieces_in(s)));
                if (sent.ropes) (void)warp_wait_bounded(&ctl->rope_full, last_parity(sent.ropes));
                for (uint32_t b = 0; b < 2; ++b)
                    if (sent.scales_in(b)) (void)warp_wait_bounded(&ctl->scale_full[b], last_parity(sent.scales_in(b)));
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- tensor-core products
            // One thread issues everything.  The tensor cores hold about four products (200 cycles) of
            // work in hand, so a barrier is tested while the products before it are being issued and
            // its latency stays hidden.
            if (elect_one()) {
                // Products into one accumulator have one shape, so that they run in order: n = 128 for two query
                // terms, n = 64 for three.
                constexpr uint32_t idesc_s = f8_idesc(kKeys, Q3 ? kRows : 2 * kRows, kE4M3, kE4M3, false, false);
                constexpr uint32_t idesc_s3 = f8_idesc(kKeys, kRows, kE4M3, kE5M2, false, false);
                constexpr uint32_t idesc_hi = f8_idesc(128, kRows, kE4M3, kE4M3, true, true);
                constexpr uint32_t idesc_lo = f8_idesc(128, kRows, kE4M3, kE5M2, true, true);
                const uint32_t q_u = smem_u32(smem), p_u = smem_u32(weights);
                // descriptors; a step along an operand adds its bytes / 16
                const uint64_t d_ring = smem_desc(smem_u32(ring), 128), d_rope = smem_desc(smem_u32(rope_k), a.rope);
                const uint64_t d_q = smem_desc(q_u, 128), d_qr = smem_desc(q_u + 2 * a.rank * kRows, a.rope);
                const uint64_t d_p[3] = {smem_desc(p_u, 64), smem_desc(p_u + kKeys * kRows, 64),
                                         smem_desc(p_u + 2 * kKeys * kRows, 64)};
                const uint32_t q3_u = q_u + 2 * kRows * (a.rank + a.rope);
                const uint64_t d_q3 = smem_desc(q3_u, 128), d_qr3 = smem_desc(q3_u + a.rank * kRows, a.rope);
                // Pieces of the next tile's scores that may be awaited before this tile's pieces are free.
                const int lead = min(pieces, a.slots - pieces);
                ThreadWaiter wait;
                uint32_t tile_s = 0;             // tiles whose scores were issued
                uint32_t slot_s = 0, lap_s = 0;  // ring position of the scores
                uint32_t slot_o = 0;             // ring position of the outputs
                uint32_t item_count = 0;
                bool ready = false;  // the ring slot that the scores read next was seen full

                // One step of K: all query terms q (the second `lo` descriptor steps behind the first), q3.
                const auto score = [&](uint32_t d, uint64_t k, uint64_t q, uint32_t lo, uint64_t q3, bool acc) {
                    mma_f8(d, k, q, idesc_s, acc);
                    if (Q3) {
                        mma_f8(d + kRows, k, q + lo, idesc_s, acc);
                        mma_f8(d + kRows, k, q3, idesc_s3, true);
                    }
                };
                // Scores of one tile: pieces [c0, c1), the rope part before piece 0.
                const auto scores = [&](int c0, int c1) {
                    const uint32_t d = tmem + kScoreCol + (tile_s & 1) * (2 * kRows);
                    if (c0 == 0 && a.rope) {
                        wait(&ctl->rope_full, tile_s & 1);
                        tc_fence_after();
                        ready = mbar_test(&ctl->full[slot_s], lap_s & 1);
#pragma unroll 1
                        for (int k = 0; k < a.rope / 32; ++k)
                            score(d, d_rope + k * 2, d_qr + k * 2, kRows * a.rope / 16, d_qr3 + k * 2, k != 0);
                        if (!wait.dead) tc_commit(&ctl->rope_free);
                    }
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        if (!ready) wait(&ctl->full[slot_s], lap_s & 1);
                        tc_fence_after();
                        const uint64_t ka = d_ring + slot_s * (kPiece / 16), qa = d_q + c * (2 * kRows * 8), qa3 = d_q3 + c * (kRows * 8);
                        if (++slot_s == static_cast<uint32_t>(a.slots)) {
                            slot_s = 0;
                            ++lap_s;
                        }
                        ready = mbar_test(&ctl->full[slot_s], lap_s & 1);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            score(d, ka + k * 2, qa + k * 2, kLatLo / 16, qa3 + k * 2, a.rope || c != 0 || k != 0);
                    }
                    if (c1 == pieces) tc_commit(&ctl->score_full[tile_s++ & 1]);
                };

                int left = 0;       // tiles of the current segment that follow this one
                bool first = true;  // the tile starts a segment
                long long pos = run_first;
                wait(&ctl->q_ready, 0);
                tc_fence_after();
                scores(0, pieces);
                bool more = true;
#pragma unroll 1
                for (uint32_t i = 0; more; ++i) {
                    if (first) {
                        left = static_cast<int>(min(static_cast<long long>(it.tiles - off), run_hi - pos));
                        off = 0;
                        pos += left + kStart;
                        if (pos < run_hi) next_item(a, it);
                    }
                    --left;
                    const bool same = left > 0;
                    more = same || pos < run_hi;
                    if (more && same && lead > 0) scores(0, lead);
                    wait(&ctl->weights_ready, i & 1);
                    if (wait.dead) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < pieces; ++c) {
                        const uint64_t va = d_ring + slot_o * (kPiece / 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_f8(tmem + c * kRows, va + k * 256, d_p[0] + k * 128, idesc_hi, !first || k != 0);
                            mma_f8(tmem + c * kRows, va + k * 256, d_p[1] + k * 128, idesc_lo, true);
                            if (P3) mma_f8(tmem + c * kRows, va + k * 256, d_p[2] + k * 128, idesc_lo, true);
                        }
                        tc_commit(&ctl->freed[slot_o]);
                        if (++slot_o == static_cast<uint32_t>(a.slots)) slot_o = 0;
                    }
                    tc_commit(&ctl->out_done);
                    if (more) {
                        if (same) {
                            if (lead < pieces) scores(lead, pieces);
                        } else {
                            wait(&ctl->q_ready, ++item_count & 1);
                            tc_fence_after();
                            scores(0, pieces);
                        }
                    }
                    first = !same;
                }
                tc_commit(&ctl->drain);
            }
            __syncwarp();
            (void)warp_wait_bounded(&ctl->drain, 0);
        } else {
            // ---------------------------------------------------------------- softmax
            const int key = tid & (kKeys - 1), half = tid >> 7, wq = warp & 3;
            const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
            const int col = half * 32 + lane;  // the column whose statistics this lane holds
            uint32_t tile = 0, slot = 0;
            if (tid == 0) a.owner[blockIdx.x] = Owner{};
            // The segment whose accumulators are in TMEM: item `it`, tiles off .. off + n - 1.
            Item next = it;
            long long pos = run_first;
            int n = 0;
            bool have = false, more = true;  // a segment is complete; another one follows
            uint64_t sums[16];               // per pair of columns: sums of weights
            for (;;) {
                // The next item's queries are staged ahead of the accumulators' way out, so that the
                // tensor cores have its first scores ready by then.
                if (more) {
                    if (have) {
                        named_bar_sync(3, kSoftmaxWarps * 32);  // nobody reads the row scales any more
                        next = ctl->next;
                    }
                    stage_q<Q3>(a, ctl, smem, item_row0(a, next), item_rows(a, next), tid, !have);
                    fence_async_smem();
                    named_bar_sync(3, kSoftmaxWarps * 32);
                    if (lane == 0) mbar_arrive(&ctl->q_ready);
                }
                if (have) {
                    const int64_t row0 = item_row0(a, it);
                    const int rows = item_rows(a, it);
                    wait(&ctl->out_done, (tile - 1) & 1);
                    tc_fence_after();
                    // The weights' shared memory is free: the four warps' sums meet there, in a fixed order.
                    float *scratch = reinterpret_cast<float *>(weights);
                    float part[32];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 u = unpack2(sums[c]);
                        part[2 * c] = u.x;
                        part[2 * c + 1] = u.y;
                    }
                    scratch[wq * kRows + col] = column_sums(part, lane);
                    named_bar_sync(1 + half, 128);
                    const float sum = (scratch[col] + scratch[kRows + col]) +
                                      (scratch[2 * kRows + col] + scratch[3 * kRows + col]);
                    const bool whole = off == 0 && n == it.tiles;
                    const int here = 2 * static_cast<int>(blockIdx.x) + (pos == run_first ? 0 : 1);
                    const float scale_col = whole ? (sum == 0.f ? 0.f : __fdiv_rn(1.f, sum)) : 1.f;
                    float norm[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) norm[c] = __shfl_sync(kFullMask, scale_col, c);
                    if (!whole) {
                        if (wq == 0) a.stats[here * kRows + col] = make_float2(ctl->ref[col], sum);
                        if (off == 0 && tid == 0) {  // this CTA holds the item's start: it names its parts
                            Owner o = {};
                            o.row0 = row0;
                            o.rows = static_cast<unsigned char>(rows);
                            o.tail = static_cast<unsigned char>(here & 1);
                            o.last = static_cast<short>(quotient(pos + it.tiles - 1, per));
                            a.owner[blockIdx.x] = o;
                        }
                    }
#pragma unroll 1
                    for (int p = 0; p < pieces; ++p) {
                        float o[32];
                        tmem_ld32(tmem + lane_base + p * kRows + half * 32, o);
                        const int dim = p * 128 + key;
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] *= norm[c];
                        if (!whole || P3) {
                            float *dst = whole ? static_cast<float *>(a.out) + row0 * a.rank
                                               : a.part + static_cast<int64_t>(here) * kRows * a.rank;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (half * 32 + c < rows) dst[(half * 32 + c) * a.rank + dim] = o[c];
                        } else {
                            // lanes 2 k and 2 k + 1 hold neighbouring dims: each stores one pair of one column
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + row0 * a.rank + (dim & ~1);
                            const int odd = lane & 1;
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                const float got = __shfl_xor_sync(kFullMask, odd ? o[c] : o[c + 1], 1);
                                const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(got, o[c + 1])
                                                             : __floats2bfloat162_rn(o[c], got);
                                const int r = half * 32 + c + odd;
                                if (r < rows) *reinterpret_cast<__nv_bfloat162 *>(dst + r * a.rank) = v;
                            }
                        }
                    }
                    tc_fence_before();
                    named_bar_sync(3, kSoftmaxWarps * 32);  // the scratch is free again
                    pos += n + kStart;
                    off = 0;
                }
                if (!more) break;
                it = next;
                n = static_cast<int>(min(static_cast<long long>(it.tiles - off), run_hi - pos));
                have = true;
                more = pos + n + kStart < run_hi;
                if (tid == 0 && more) {
                    next_item(a, next);
                    ctl->next = next;
                }

                // keys that the column's token sees
                const int lim_min = max(0, min(it.vis, it.kv - it.t + it.tok + 1));
                if (wq == 0) ctl->ref[col] = ctl->peak[col] = kUnset;
                int watch = off + 2;  // tile that begins with a look at the weights of the one before
                uint64_t shift[16];  // per pair of columns: -(reference + slack)
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    shift[c] = 0;
                    sums[c] = 0;
                }
                for (int i = off; i < off + n; ++i, ++tile) {
                    const int k = i * kKeys + key;
                    wait(&ctl->scale_full[tile & 1], (tile >> 1) & 1);
                    float sj = tile_scale[(tile & 1) * kKeys + key];
                    __syncwarp();
                    if (lane == 0 && !wait.dead) mbar_arrive(&ctl->scale_free[tile & 1]);
                    const bool in = k < it.vis;
                    if (!in) sj = 1.f;  // no column sees it
                    const float f = sj * a.scale_log2;
                    // The weight of a row that is zero, or nearly, in every column must count in the sums
                    // and not lift the reference above the others', nor leave f32's range.
                    if (sj < kLeastScale) sj = kLeastScale;
                    const float add = __log2f(sj);
                    const uint64_t ff = pack2(f, f), aa = pack2(add, add);
                    // 256 is the weights' common factor; a NaN scale must not reach the columns that do
                    // not see its row
                    const float iv = sj == sj ? __fdiv_rn(256.f, sj) : 256.f;
                    const uint64_t inv = pack2(iv, iv);
                    const bool masked = (i + 1) * kKeys > lim_min;  // some column does not see some key
                    const uint32_t at_s = tmem + lane_base + kScoreCol + (tile & 1) * (2 * kRows) + half * 32;

                    // s = log2 of the weight over 2^8: score + log2 scale - reference - slack
                    float s[32];
                    wait(&ctl->score_full[tile & 1], (tile >> 1) & 1);
                    tc_fence_after();
                    // A look at this thread's own codes of the tile before, which every column saw.
                    bool down = false;
                    if (i == watch) {
                        watch = i + kLook;
                        if (i * kKeys <= lim_min) {
                            uint32_t near = 0;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint4 w = *reinterpret_cast<const uint4 *>(weights + swizzled(key, (half * 2 + q) * 16, 64));
                                near |= high_codes(w.x) << (4 * q) | high_codes(w.y) << (4 * q + 1) |
                                        high_codes(w.z) << (4 * q + 2) | high_codes(w.w) << (4 * q + 3);
                            }
                            near = __reduce_or_sync(kFullMask, near);
                            if (lane == 0) ctl->near[half * 4 + wq] = near;
                            named_bar_sync(1 + half, 128);
                            const uint4 w = *reinterpret_cast<const uint4 *>(&ctl->near[half * 4]);
                            down = (w.x | w.y | w.z | w.w) != kFullMask;
                            if (down) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) shift[c] = 0;
                            }
                        }
                    }
                    // Usually one turn, number 0.  When a column exceeds its reference by the slack, or was
                    // found far below it, and on the first tile, turn 1 takes the plain scores for the
                    // columns' maxima, to which the references move, and turn 2 the shifted scores again.
                    for (int turn = i == off || down ? 1 : 0;; ++turn) {
                        uint32_t r[32], r_lo[32];
                        tmem_ld32_nowait(at_s, r);
                        tmem_ld32_nowait(at_s + kRows, r_lo);
                        tc_wait_ld();
                        tmem_ld32_done(r);
                        tmem_ld32_done(r_lo);
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const ulonglong2 g = *reinterpret_cast<const ulonglong2 *>(&ctl->row_scale[half * 32 + 2 * c]);
                            const uint64_t r0 = add2(bits2(r[2 * c], r[2 * c + 1]), bits2(r_lo[2 * c], r_lo[2 * c + 1]));
                            const uint64_t r1 = add2(bits2(r[2 * c + 2], r[2 * c + 3]), bits2(r_lo[2 * c + 2], r_lo[2 * c + 3]));
                            const float2 v0 = unpack2(fma2(r0, mul2(ff, g.x), add2(aa, shift[c])));
                            const float2 v1 = unpack2(fma2(r1, mul2(ff, g.y), add2(aa, shift[c + 1])));
                            s[2 * c] = v0.x;
                            s[2 * c + 1] = v0.y;
                            s[2 * c + 2] = v1.x;
                            s[2 * c + 3] = v1.y;
                        }
                        if (masked) {
                            const int lim_col = max(0, min(it.vis, it.kv - it.t + it.tok + 1 +
                                                                       (a.head_blocks > 1 ? 0 : min(col / a.nh, a.group - 1))));
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (k >= __shfl_sync(kFullMask, lim_col, c)) s[c] = -INFINITY;
                        }
                        if (turn == 0) {
                            float m = s[0];
#pragma unroll
                            for (int c = 1; c < 32; ++c) m = fmaxf(m, s[c]);
                            if (!named_bar_any(1 + half, 128, m > kOver)) break;
#pragma unroll
                            for (int c = 0; c < 16; ++c) shift[c] = 0;
                            continue;
                        }
                        if (turn == 2) break;
                        atomicMax(&ctl->tops[col], order_bits(column_maxima(s, lane)));
                        named_bar_sync(1 + half, 128);
                        const float ref = ctl->ref[col], peak = ctl->peak[col], here = unorder_bits(ctl->tops[col]);
                        const float low = fmaxf(here, peak - kDepth);
                        const float to = down && low < ref - kKeep ? low : fmaxf(ref, here);
                        const float shrink = ex2(ref - to);
                        if (wq == 0) {
                            ctl->shrink[col] = shrink;
                            ctl->minus[col] = to == kUnset ? -kUnset : -(to + kSlack);
                        }
                        named_bar_sync(1 + half, 128);
                        if (wq == 0) {
                            ctl->tops[col] = 0;
                            ctl->ref[col] = to;
                            ctl->peak[col] = fmaxf(peak, to);
                        }
                        const uint64_t *by = reinterpret_cast<const uint64_t *>(&ctl->shrink[half * 32]);
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            shift[c] = *reinterpret_cast<const uint64_t *>(&ctl->minus[half * 32 + 2 * c]);
                        if (i > off && __any_sync(kFullMask, shrink != 1.f)) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) sums[c] = mul2(sums[c], by[c]);
                            if (__any_sync(kFullMask, shrink < kJump)) watch = i + 2;
                            wait(&ctl->out_done, (tile - 1) & 1);
                            tc_fence_after();
#pragma unroll 1
                            for (int p = 0; p < pieces; ++p) {
                                float o[32];
                                const uint32_t at = tmem + lane_base + p * kRows + half * 32;
                                tmem_ld32(at, o);
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    const float2 u = unpack2(mul2(pack2(o[2 * c], o[2 * c + 1]), by[c]));
                                    o[2 * c] = u.x;
                                    o[2 * c + 1] = u.y;
                                }
                                tmem_st32(at, o);
                            }
                            tc_wait_st();
                        }
                    }
                    uint32_t hi[8], mid[8], lo[8];  // lo: P3
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        uint32_t x[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float p0 = ex2(s[c + 2 * q]), p1 = ex2(s[c + 2 * q + 1]);
                            sums[c / 2 + q] = fma2(pack2(p0, p1), inv, sums[c / 2 + q]);
                            x[q] = f32x2_to_f16x2(p0, p1);
                        }
                        uint32_t h[2], m[2], l[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            h[q] = x[q] + 0x00400040u;  // to the nearest multiple of three fraction bits
                            const uint32_t rest = times256(sub_f16x2(x[q], h[q] & 0xff80ff80u));
                            m[q] = rest + 0x00800080u;
                            if (P3) l[q] = sub_f16x2(rest, m[q] & 0xff00ff00u) + 0x00800080u;
                            h[q] <<= 1;
                        }
                        hi[c / 4] = __byte_perm(h[0], h[1], 0x7531);
                        mid[c / 4] = e5m2_bits(m[0], m[1]);
                        if (P3) lo[c / 4] = e5m2_bits(l[0], l[1]);
                    }
                    if (tile >= 1) wait(&ctl->out_done, (tile - 1) & 1);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint8_t *at = weights + swizzled(key, (half * 2 + q) * 16, 64);
                        const auto put = [&](int term, const uint32_t(&v)[8]) {
                            *reinterpret_cast<uint4 *>(at + term * kKeys * kRows) =
                                make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                        };
                        put(0, hi);
                        put(1, mid);
                        if (P3) put(2, lo);
                    }
                    if (!in) {  // rows past the end: zero weights must meet finite codes
                        uint32_t sl = slot;
                        for (int p = 0; p < pieces; ++p) {
                            if ((p & 1) == half) {
                                uint4 *v = reinterpret_cast<uint4 *>(ring + sl * kPiece + key * 128);
#pragma unroll
                                for (int q = 0; q < 8; ++q) v[q] = make_uint4(0, 0, 0, 0);
                            }
                            if (++sl == static_cast<uint32_t>(a.slots)) sl = 0;
                        }
                    }
                    slot += pieces;
                    if (slot >= static_cast<uint32_t>(a.slots)) slot -= a.slots;
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->weights_ready);
                }
            }
        }
    } else if (tid == 0) {
        a.owner[blockIdx.x] = Owner{};
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the partial accumulators of the items that several CTAs shared.  CTAs (x, 0 .. gridDim.y - 1)
// serve the x-th such item, in units of 128 dims of a row (a lane four dims).  Up to kFewParts parts a
// warp serves a unit alone: no barrier, 64 units under way on an SM.  Above, a CTA serves it: warp w
// adds parts w, w + 8, ... and the eight sums are added in warp order.
constexpr int kCombineWarps = 8;
constexpr int kCombineThreads = kCombineWarps * 32;
constexpr int kFewParts = 32;
static_assert(kMaxGrid <= kCombineThreads, "a thread looks at one CTA's part");

__device__ __forceinline__ float4 load_part(const PagedArgs &a, int64_t slot, int r, int d) {
    return __ldcg(reinterpret_cast<const float4 *>(a.part + (slot * kRows + r) * a.rank + d));
}
__device__ __forceinline__ void fma4(float4 &acc, float4 v, float x) {
    acc.x = fmaf(v.x, x, acc.x);
    acc.y = fmaf(v.y, x, acc.y);
    acc.z = fmaf(v.z, x, acc.z);
    acc.w = fmaf(v.w, x, acc.w);
}

__device__ __forceinline__ void store_out(const PagedArgs &a, int64_t at, float4 o, float total) {
    const float n = total == 0.f ? 0.f : __fdiv_rn(1.f, total);
    o = make_float4(o.x * n, o.y * n, o.z * n, o.w * n);
    if (a.out_bf16) {
        __nv_bfloat162 v[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = *reinterpret_cast<uint2 *>(v);
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = o;
    }
}

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const PagedArgs a, int grid) {
    __shared__ int found;
    __shared__ Owner owner;
    __shared__ int counts[kCombineWarps];
    __shared__ float weight[kMaxGrid];
    __shared__ float red[2][kCombineWarps];
    __shared__ float4 sums[kCombineWarps][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    if (tid == 0) found = -1;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (tid < grid) raw = __ldcg(reinterpret_cast<const uint4 *>(a.owner + tid));
    const Owner own = *reinterpret_cast<const Owner *>(&raw);
    const bool flag = own.rows != 0;
    const unsigned ballot = __ballot_sync(kFullMask, flag);
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int rank_of = __popc(ballot & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) rank_of += counts[w];
    if (flag && rank_of == static_cast<int>(blockIdx.x)) {
        found = tid;
        owner = own;
    }
    __syncthreads();
    if (found < 0) return;
    const int cta = found, slot0 = 2 * cta + owner.tail;
    const long long row0 = owner.row0;
    const int parts = min(static_cast<int>(owner.last), grid - 1) - cta + 1, pieces = a.rank / 128;
    const int units = owner.rows * pieces;
    const auto slot_of = [&](int k) { return k == 0 ? slot0 : 2 * (cta + k); };
    if (parts <= kFewParts) {
        for (int unit = blockIdx.y * kCombineWarps + warp; unit < units; unit += gridDim.y * kCombineWarps) {
            const int r = unit / pieces, d = (unit - r * pieces) * 128 + lane * 4;
            float2 st = make_float2(kUnset, 0.f);
            if (lane < parts) st = __ldcg(a.stats + slot_of(lane) * kRows + r);
            const float w = ex2(st.x - warp_max(st.x));
            const float total = warp_sum(w * st.y);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k0 = 0; k0 < parts; k0 += 4) {  // past the last part: the last again, with weight 0
#pragma unroll
                for (int k = k0; k < k0 + 4; ++k) {
                    const float x = __shfl_sync(kFullMask, w, k);
                    fma4(acc, load_part(a, slot_of(min(k, parts - 1)), r, d), k < parts ? x : 0.f);
                }
            }
            store_out(a, (row0 + r) * a.rank + d, acc, total);
        }
        return;
    }
    for (int unit = blockIdx.y; unit < units; unit += gridDim.y) {
        const int r = unit / pieces, d = (unit - r * pieces) * 128 + lane * 4;
        float2 st = make_float2(kUnset, 0.f);
        if (tid < parts) st = __ldcg(a.stats + slot_of(tid) * kRows + r);
        // the first parts come in while the weights are formed
        float4 early[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) early[k] = load_part(a, slot_of(min(warp + k * kCombineWarps, parts - 1)), r, d);
        const float wm = warp_max(st.x);
        if (lane == 0) red[0][warp] = wm;
        __syncthreads();
        float top = red[0][0];
        for (int w = 1; w < kCombineWarps; ++w) top = fmaxf(top, red[0][w]);
        const float w = ex2(st.x - top);
        const float l = warp_sum(w * st.y);
        if (lane == 0) red[1][warp] = l;
        if (tid < parts) weight[tid] = w;
        __syncthreads();
        float total = 0.f;
        for (int k = 0; k < kCombineWarps; ++k) total += red[1][k];
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int part = warp + k * kCombineWarps;
            fma4(acc, early[k], part < parts ? weight[part] : 0.f);
        }
#pragma unroll 8
        for (int k = warp + 8 * kCombineWarps; k < parts; k += kCombineWarps)
            fma4(acc, load_part(a, slot_of(k), r, d), weight[k]);
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
            for (int k = 1; k < kCombineWarps; ++k) {
                const float4 v = sums[k][lane];
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
            }
            store_out(a, (row0 + r) * a.rank + d, acc, total);
        }
        __syncthreads();  // the shared arrays are free for the next unit
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// Rows of `width` bytes; a box of `rows` rows and `bytes` bytes, swizzled over its own row length.
bool encode_rows(CUtensorMap *map, const void *base, uint64_t width, uint64_t n, uint32_t bytes, uint32_t rows) {
    const EncodeTiledFn enc = encode_tiled();
    const cuuint64_t dims[2] = {width, n};
    const cuuint64_t strides[1] = {width};
    const cuuint32_t box[2] = {bytes, rows}, step[2] = {1, 1};
    const CUtensorMapSwizzle sw = bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_32B;
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

template <bool Q3, bool P3>
cudaError_t allow_smem(int bytes) {
    return cudaFuncSetAttribute(attn_paged_kernel<Q3, P3>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// SM count and opt-in shared memory of the current device, after allowing the kernel all of it
// (queried once per device).
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
        allow_smem<false, false>(smem) != cudaSuccess || allow_smem<false, true>(smem) != cudaSuccess ||
        allow_smem<true, false>(smem) != cudaSuccess || allow_smem<true, true>(smem) != cudaSuccess)
        return false;
    if (dev < kMaxDevices) {
        smem_cache[dev].store(smem, std::memory_order_relaxed);
        sm_cache[dev].store(sms, std::memory_order_release);
    }
    return true;
}

bool rank_ok(int rank) { return rank == 128 || rank == 256 || rank == 512; }
bool rope_ok(int rope) { return rope == 0 || rope == 32 || rope == 64 || rope == 128; }
bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Workspace: owners, statistics, partial accumulators.
constexpr int64_t kOwnerBytes = kMaxGrid * sizeof(Owner);
int64_t stat_bytes(int grid) { return static_cast<int64_t>(2) * grid * kRows * sizeof(float2); }
int64_t part_bytes(int grid, int rank) { return static_cast<int64_t>(2) * grid * kRows * rank * sizeof(float); }

}  // namespace
}  // namespace memq

// Internal: this translation unit's device fault word (not part of the public header).
int memq_internal_fault_paged(unsigned int *out, bool clear) {
    if (cudaMemcpyFromSymbol(out, memq::g_paged_fault, sizeof(unsigned int)) != cudaSuccess) return 1;
    if (!clear) return 0;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(memq::g_paged_fault, &zero, sizeof(zero)) == cudaSuccess ? 0 : 1;
}

extern "C" int64_t memq_mla_attn_paged_workspace(int kv_rank) {
    using namespace memq;
    if (!rank_ok(kv_rank)) return -1;
    int sms = 0, smem = 0;
    if (!device_info(sms, smem)) return -1;
    const int grid = std::min(sms, kMaxGrid);
    return kOwnerBytes + stat_bytes(grid) + part_bytes(grid, kv_rank);
}

extern "C" int memq_mla_attn_paged(int q_dtype, const void *q_lat, const void *q_pe, const uint8_t *cache,
                                   const float *scales, const int32_t *block_table, const int32_t *kv_len,
                                   const int32_t *cu_q, int out_dtype, void *out, void *workspace,
                                   int64_t workspace_bytes, int64_t n_tok, int n_seq, int nh, int kv_rank, int d_rope,
                                   int64_t n_pages, int page_size, int max_pages, float scale, void *stream) {
    using namespace memq;
    if ((q_dtype != MEMQ_F32 && q_dtype != MEMQ_BF16) || (out_dtype != MEMQ_F32 && out_dtype != MEMQ_BF16))
        return MEMQ_ERR_SHAPE;
    if (n_tok < 0 || n_tok > (1 << 24) || n_seq < 0 || n_seq > kMaxSeqs || nh < 1 || nh > 1024 || !rank_ok(kv_rank) ||
        !rope_ok(d_rope) || page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0 || n_pages < 0 ||
        n_pages > 0x7fffffffLL / page_size || max_pages < 0 || max_pages > kMaxCached / page_size ||
        !std::isfinite(scale * kLog2e))
        return MEMQ_ERR_SHAPE;
    if (n_tok == 0 || n_seq == 0) return MEMQ_OK;  // no query rows
    if (n_pages < 1 || max_pages < 1) return MEMQ_ERR_SHAPE;
    if (!q_lat || (d_rope > 0 && !q_pe) || !cache || !scales || !block_table || !kv_len || !cu_q || !out || !workspace)
        return MEMQ_ERR_NULL;
    const uintptr_t o_al = out_dtype == MEMQ_F32 ? 16 : 8;
    if (misaligned(q_lat, 16) || (d_rope > 0 && misaligned(q_pe, 16)) || misaligned(cache, 16) ||
        misaligned(scales, 16) || misaligned(block_table, 4) || misaligned(kv_len, 4) || misaligned(cu_q, 4) ||
        misaligned(out, o_al) || misaligned(workspace, 16))
        return MEMQ_ERR_ALIGN;
    int sms = 0, smem = 0;
    if (!device_info(sms, smem)) return MEMQ_ERR_LAUNCH;
    const int grid = std::min(sms, kMaxGrid);
    if (workspace_bytes < kOwnerBytes + stat_bytes(grid) + part_bytes(grid, kv_rank)) return MEMQ_ERR_SHAPE;

    PagedArgs a{};
    a.q_lat = q_lat;
    a.q_pe = q_pe;
    a.scales = scales;
    a.table = block_table;
    a.kv_len = kv_len;
    a.cu_q = cu_q;
    a.out = out;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.owner = reinterpret_cast<Owner *>(ws);
    a.stats = reinterpret_cast<float2 *>(ws + kOwnerBytes);
    a.part = reinterpret_cast<float *>(ws + kOwnerBytes + stat_bytes(grid));
    a.n_tok = static_cast<int>(n_tok);
    a.n_seq = n_seq;
    a.nh = nh;
    a.rank = kv_rank;
    a.rope = d_rope;
    a.n_pages = static_cast<int>(n_pages);
    a.page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
    a.box = std::min(page_size, kKeys);
    a.max_pages = max_pages;
    // Up to 64 heads: as many whole tokens as fit in the tile's 64 rows.  More: one token, the heads in
    // blocks of equal size.
    a.head_blocks = (nh + kRows - 1) / kRows;
    a.heads_per = (nh + a.head_blocks - 1) / a.head_blocks;
    a.group = a.head_blocks > 1 ? 1 : kRows / nh;
    a.out_bf16 = out_dtype == MEMQ_BF16;
    a.scale_log2 = scale * kLog2e;
    const bool q3 = q_dtype == MEMQ_F32, p3 = out_dtype == MEMQ_F32;
    const int fixed = smem_ring_off(q3, p3, kv_rank, d_rope) + smem_tail();
    a.slots = std::min(kMaxSlots, (smem - fixed) / kPiece);
    if (a.slots < kv_rank / 128) return MEMQ_ERR_LAUNCH;
    const uint64_t width = static_cast<uint64_t>(kv_rank + d_rope), pool = static_cast<uint64_t>(n_pages) * page_size;
    CUtensorMap lat, rope;
    if (!encode_rows(&lat, cache, width, pool, 128, a.box) ||
        !encode_rows(&rope, cache, width, pool, d_rope ? d_rope : 32, a.box))
        return MEMQ_ERR_LAUNCH;

    // Programmatic dependent launches: both kernels wait for their predecessors before they read.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(fixed) + static_cast<size_t>(a.slots) * kPiece;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const auto kernel = q3 ? (p3 ? attn_paged_kernel<true, true> : attn_paged_kernel<true, false>)
                           : (p3 ? attn_paged_kernel<false, true> : attn_paged_kernel<false, false>);
    if (cudaLaunchKernelEx(&cfg, kernel, lat, rope, a) != cudaSuccess) return MEMQ_ERR_LAUNCH;
    const int64_t items = n_tok * a.head_blocks;  // at least the number of items
    const unsigned x = static_cast<unsigned>(std::min<int64_t>(items, grid));
    // About eight CTAs an SM over all items, and no more than an item's rows have units of 128 dims.
    cfg.gridDim = dim3(x, std::max(1u, std::min(static_cast<unsigned>(kRows * kv_rank / 128), 8u * grid / x)));
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, combine_kernel, a, grid) == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}
