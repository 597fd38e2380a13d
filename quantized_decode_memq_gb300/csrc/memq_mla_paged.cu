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
// the operations at twice the 16-bit rate):
//   q = 2^e (hi + lo), both E4M3, e per row: 8 significant bits, which hold a bf16 value exactly
//       down to 2^-10 of the row's largest; below that an absolute 2^-18 of the largest;
//   p = hi (E4M3) + lo (E5M2), with p in (0, 2^8]: a relative 2^-7 at most (about 2^-10 rms), and
//       an absolute 2^-17, 2^-21 of the running maximum: E5M2 carries the long tail of small
//       weights that a second E4M3 term would flush.
// The key's scale is folded into its weight (p_j = 2^4 exp2(s_j + log2 scales_j - R)), so R, the
// running reference, bounds what the 8-bit terms must hold; the sum of weights is kept apart in f32.
// R moves, and the accumulators are rescaled, only when a tile's maximum exceeds it by 2^4.
//
// One CTA per SM.  The 128-key tiles of all (sequence, token group, head block) items form one list
// that is cut into equal runs, one per CTA; every CTA derives its run from the lengths on the device
// (nothing of the plan is on the host, so a captured graph serves other lengths).  An item that
// spans CTAs leaves f32 partial accumulators in the workspace, and combine_kernel adds them in CTA
// order: results do not depend on timing.
//
// Warps 0-7 are the softmax warps (thread = key x half of the columns), warp 8 issues the TMA copies
// of 128 x 128-byte pieces into a ring, warp 9 the tensor-core products.  S^T is double buffered:
// the scores of tile i + 1 are computed while the softmax of tile i runs.
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
constexpr int kThreads = (kSoftmaxWarps + 2) * 32;
constexpr int kMaxSeqs = 4096;
constexpr int kMaxGrid = 256;
constexpr float kUnset = -1e30f;  // the reference before the first visible key
constexpr float kSlack = 4.0f;    // log2 of how far weights may exceed the reference
constexpr float kBase = 4.0f;     // log2 of a weight at the reference
constexpr int kScoreCol = 256;    // TMEM: accumulators in columns 0..255, scores after them

struct Owner {
    long long row0;  // first output row of the item
    int rows;
    int slot;  // its first partial; the others are slots 2 c of the CTAs up to `last`
    int last;
    int pad;
};

struct PagedArgs {
    const void *q_lat, *q_pe;
    const float *scales;
    const int32_t *table, *kv_len, *cu_q;
    void *out;
    int *owner_flag;
    Owner *owner;
    float2 *stats;  // [slot][row] (reference, sum of weights)
    float *part;    // [slot][row][rank]
    int n_tok, n_seq, nh, rank, rope, n_pages, page_shift, box, max_pages;
    int group;  // tokens per item
    int heads_per, head_blocks;
    int slots;
    int q_bf16, out_bf16;
    float scale_log2;
};

struct Control {
    uint32_t tops[3][kRows];  // column maxima of three successive tiles (order_bits)
    float row_scale[kRows];
    uint64_t full[kMaxSlots], freed[kMaxSlots];
    uint64_t rope_full, rope_free, scale_full[2], scale_free[2], score_full[2];
    uint64_t weights_ready, out_done, q_ready, drain;
    uint32_t tmem;
    int first_seq, first_tok, first_block, first_off;
    long long total, warp_sum[kThreads / 32];
};
static_assert(sizeof(Control) <= 2048, "the control block has 2 KB of shared memory");

// Shared memory, from a 1024-byte boundary: Q terms (latent hi, lo; rope hi, lo), P terms, the rope
// piece, the ring, the scales of two tiles, the control block.
__host__ __device__ constexpr int smem_ring_off(int rank, int rope) {
    return rank * 128 + 128 * rope + 2 * kKeys * kRows + kKeys * rope;
}
__host__ __device__ constexpr int smem_tail() { return 2 * kKeys * 4 + 2048; }

struct Item {
    int seq, start, t, kv;  // sequence, its first token row, new tokens, cached rows
    int tok, block;         // first token of the group, head block
    int vis, tiles;         // keys that its last token sees, tiles
};

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
            if (++it.seq >= a.n_seq) {  // past the last sequence: an empty item, never reached
                it.t = 0;
                break;
            }
            seq_sizes(a, __ldcg(a.cu_q + it.seq), __ldcg(a.cu_q + it.seq + 1), __ldcg(a.kv_len + it.seq), it);
        } while (it.t == 0);
    }
    item_sizes(a, it);
}

// Waits for a barrier phase; after one wait expired, none is made any more (the kernel then runs to
// its end on whatever is there, and the fault word says so).
struct Waiter {
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        if (!dead && !warp_wait_bounded(bar, parity)) {
            dead = true;
            if ((threadIdx.x & 31) == 0) atomicOr(&g_paged_fault, kFaultWait);
        }
    }
};

// Four consecutive query elements.
__device__ __forceinline__ float4 load_q4(const void *p, int64_t i, bool bf16) {
    if (bf16) {
        const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i));
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    }
    return __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
}

__device__ __forceinline__ bool finite4(float4 v) {
    return isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w);
}

// hi and lo terms of four scaled query elements.
__device__ __forceinline__ void split_q4(float4 v, float inv, uint32_t &hi, uint32_t &lo) {
    const float x[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
    const uint32_t h0 = f32x2_to_e4m3x2(x[0], x[1]), h1 = f32x2_to_e4m3x2(x[2], x[3]);
    const uint32_t b0 = e4m3x2_to_f16x2(h0), b1 = e4m3x2_to_f16x2(h1);
    const float2 r0 = __half22float2(*reinterpret_cast<const __half2 *>(&b0));
    const float2 r1 = __half22float2(*reinterpret_cast<const __half2 *>(&b1));
    hi = h0 | (h1 << 16);
    lo = f32x2_to_e4m3x2(x[0] - r0.x, x[1] - r0.y) | (f32x2_to_e4m3x2(x[2] - r1.x, x[3] - r1.y) << 16);
}

// Byte offset of element `i` of row `r` in an operand of `row_bytes`-byte swizzled rows.
__device__ __forceinline__ int swizzled(int r, int i, int row_bytes) {
    const int x = row_bytes == 128 ? r & 7 : row_bytes == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
    return r * row_bytes + (i ^ (x << 4));
}

// The 64 query rows of an item -> their 8-bit terms and scales in shared memory (eight warps, eight
// rows each, four at a time).  Rows past `rows` are zeros.
__device__ __forceinline__ void stage_q(const PagedArgs &a, Control *ctl, uint8_t *smem, int64_t row0, int rows,
                                        int warp, int lane) {
    const int pieces = a.rank / 128;
    uint8_t *lat_lo = smem + a.rank * kRows;
    uint8_t *rope_hi = smem + 2 * a.rank * kRows, *rope_lo = rope_hi + kRows * a.rope;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float4 v[4][5];
        float amax[4];
        bool ok[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = warp * 8 + half * 4 + k;
            amax[k] = 0.f;
            ok[k] = true;
#pragma unroll
            for (int c = 0; c < 5; ++c) {
                v[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < rows) {
                    if (c < pieces) v[k][c] = load_q4(a.q_lat, (row0 + r) * a.rank + c * 128 + lane * 4, a.q_bf16);
                    if (c == 4 && lane * 4 < a.rope) v[k][c] = load_q4(a.q_pe, (row0 + r) * a.rope + lane * 4, a.q_bf16);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = warp * 8 + half * 4 + k;
#pragma unroll
            for (int c = 0; c < 5; ++c) {
                const float4 x = v[k][c];
                amax[k] = fmaxf(amax[k], fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
                ok[k] = ok[k] && finite4(x);
            }
            const float m = warp_max(amax[k]);
            const bool fin = __all_sync(kFullMask, ok[k]);
            // 2^e with m / 2^e in [128, 256); tiny rows keep a normal reciprocal
            const int e = max(static_cast<int>(__float_as_uint(m) >> 23), 32);
            const float inv = fin ? __uint_as_float(static_cast<uint32_t>(261 - e) << 23) : 0.f;
            if (lane == 0) ctl->row_scale[r] = fin ? __uint_as_float(static_cast<uint32_t>(e - 7) << 23) : NAN;
#pragma unroll
            for (int c = 0; c < 5; ++c) {
                uint32_t hi, lo;
                const float4 x = fin ? v[k][c] : make_float4(0.f, 0.f, 0.f, 0.f);
                split_q4(x, inv, hi, lo);
                if (c < pieces) {
                    const int at = c * kRows * 128 + swizzled(r, lane * 4, 128);
                    *reinterpret_cast<uint32_t *>(smem + at) = hi;
                    *reinterpret_cast<uint32_t *>(lat_lo + at) = lo;
                }
                if (c == 4 && lane * 4 < a.rope) {
                    const int at = swizzled(r, lane * 4, a.rope);
                    *reinterpret_cast<uint32_t *>(rope_hi + at) = hi;
                    *reinterpret_cast<uint32_t *>(rope_lo + at) = lo;
                }
            }
        }
    }
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

__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap map_lat, const __grid_constant__ CUtensorMap map_rope,
                      const PagedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pieces = a.rank / 128;
    uint8_t *weights = smem + a.rank * 128 + 128 * a.rope;
    uint8_t *rope_k = weights + 2 * kKeys * kRows;
    uint8_t *ring = smem + smem_ring_off(a.rank, a.rope);
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
    if (tid < 3 * kRows) ctl->tops[tid / kRows][tid % kRows] = 0;
    if (warp == 9) tmem_alloc(&ctl->tmem, 512);
    griddep_wait();

    // ------------------------------------------------------------------ this CTA's run of tiles
    int32_t *cu = reinterpret_cast<int32_t *>(ring), *kvl = cu + a.n_seq + 1;
    for (int i = tid; i <= a.n_seq; i += kThreads) cu[i] = __ldcg(a.cu_q + i);
    for (int i = tid; i < a.n_seq; i += kThreads) {
        const int kv = __ldcg(a.kv_len + i);
        kvl[i] = kv;
        if (kv < 0 || kv > (static_cast<long long>(a.max_pages) << a.page_shift)) atomicOr(&g_paged_fault, kFaultInput);
    }
    __syncthreads();
    // Thread i counts the tiles of the groups whose last token lies in its slice of the tokens.
    const int slice = (a.n_tok + kThreads - 1) / kThreads;
    const int tok_lo = min(a.n_tok, tid * slice), tok_hi = min(a.n_tok, tok_lo + slice);
    int seq0 = 0;
    {
        int hi = a.n_seq;  // first sequence that ends after tok_lo
        while (seq0 < hi) {
            const int mid = (seq0 + hi) >> 1;
            if (cu[mid + 1] <= tok_lo) seq0 = mid + 1; else hi = mid;
        }
    }
    long long run_lo = -1, run_hi = 0, per = 0;
    long long before = 0;
    for (int pass = 0; pass < 2; ++pass) {
        long long sum = before;  // pass 0: this slice's tiles; pass 1: find the run's first tile
        Item it{};
        it.seq = seq0;
        if (tok_lo < tok_hi && it.seq < a.n_seq) seq_sizes(a, cu[it.seq], cu[it.seq + 1], kvl[it.seq], it);
        for (int j = tok_lo; j < tok_hi && it.seq < a.n_seq; ++j) {
            while (j >= it.start + it.t && ++it.seq < a.n_seq)
                seq_sizes(a, cu[it.seq], cu[it.seq + 1], kvl[it.seq], it);
            if (it.seq >= a.n_seq) break;
            const int k = j - it.start;
            if (k < 0 || ((k + 1) % a.group != 0 && k + 1 != it.t)) continue;
            it.tok = k / a.group * a.group;
            item_sizes(a, it);
            const long long n = static_cast<long long>(it.tiles) * a.head_blocks;
            if (pass == 1 && sum <= run_lo && run_lo < sum + n) {
                ctl->first_seq = it.seq;
                ctl->first_tok = it.tok;
                ctl->first_block = static_cast<int>((run_lo - sum) / it.tiles);
                ctl->first_off = static_cast<int>((run_lo - sum) % it.tiles);
            }
            sum += n;
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
            before = incl - sum;
            long long total = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += ctl->warp_sum[w];
                total += ctl->warp_sum[w];
            }
            per = (total + gridDim.x - 1) / gridDim.x;
            run_lo = blockIdx.x * per;
            run_hi = min(total, run_lo + per);
        }
    }
    fence_async_smem();  // the lengths lie where TMA will write
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;

    if (run_lo < run_hi) {
        Item it{};
        it.seq = ctl->first_seq;
        it.tok = ctl->first_tok;
        it.block = ctl->first_block;
        seq_sizes(a, __ldcg(a.cu_q + it.seq), __ldcg(a.cu_q + it.seq + 1), __ldcg(a.kv_len + it.seq), it);
        item_sizes(a, it);
        int off = ctl->first_off;
        Waiter wait;

        if (warp == 8) {
            // ---------------------------------------------------------------- TMA producer
            uint32_t tile = 0, slot = 0, lap = 0;
            const int per_tile = kKeys / a.box;
            for (long long pos = run_lo; pos < run_hi;) {
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
                for (int i = off; i < off + n; ++i, ++tile) {
                    const int row_next = i + 1 < off + n ? page_row((i + 1) * kKeys) : -1;
                    const bool mine = row >= 0;
                    const uint32_t boxes = __popc(__ballot_sync(kFullMask, mine));
                    // scales of the tile's keys
                    uint64_t *bar = &ctl->scale_full[tile & 1];
                    if (tile >= 2) wait(&ctl->scale_free[tile & 1], ((tile >> 1) - 1) & 1);
                    if (!wait.dead) {
                        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * a.box * 4);
                        __syncwarp();
                        if (mine)
                            bulk_g2s_plain(tile_scale + (tile & 1) * kKeys + lane * a.box, a.scales + row, a.box * 4, bar);
                    }
                    if (a.rope) {
                        if (tile >= 1) wait(&ctl->rope_free, (tile - 1) & 1);
                        if (!wait.dead) {
                            if (lane == 0) mbar_arrive_expect_tx(&ctl->rope_full, boxes * a.box * a.rope);
                            __syncwarp();
                            if (mine)
                                tma_load_2d_plain(rope_k + lane * a.box * a.rope, &map_rope, a.rank, row, &ctl->rope_full);
                        }
                    }
                    for (int c = 0; c < pieces; ++c) {
                        if (lap >= 1) wait(&ctl->freed[slot], (lap - 1) & 1);
                        if (!wait.dead) {
                            if (lane == 0) mbar_arrive_expect_tx(&ctl->full[slot], boxes * a.box * 128);
                            __syncwarp();
                            if (mine)
                                tma_load_2d_plain(ring + slot * kPiece + lane * a.box * 128, &map_lat, c * 128, row,
                                                  &ctl->full[slot]);
                        }
                        if (++slot == static_cast<uint32_t>(a.slots)) {
                            slot = 0;
                            ++lap;
                        }
                    }
                    row = row_next;
                }
                pos += n;
                off = 0;
                if (pos < run_hi) next_item(a, it);
            }
            if (wait.dead) {
                // Copies in flight: every slot's last phase that was announced, each wait bounded.
                for (int s = 0; s < a.slots; ++s) {
                    const uint32_t uses = lap + (static_cast<uint32_t>(s) < slot ? 1 : 0);
                    if (uses) (void)warp_wait_bounded(&ctl->full[s], (uses - 1) & 1);
                }
                if (tile >= 1 && a.rope) (void)warp_wait_bounded(&ctl->rope_full, (tile - 1) & 1);
                if (tile >= 1) (void)warp_wait_bounded(&ctl->scale_full[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
            }
        } else if (warp == 9) {
            // ---------------------------------------------------------------- tensor-core products
            constexpr uint32_t idesc_s = f8_idesc(kKeys, kRows, kE4M3, kE4M3, false, false);
            constexpr uint32_t idesc_hi = f8_idesc(128, kRows, kE4M3, kE4M3, true, true);
            constexpr uint32_t idesc_lo = f8_idesc(128, kRows, kE4M3, kE5M2, true, true);
            const uint32_t q_hi = smem_u32(smem), q_lo = q_hi + a.rank * kRows;
            const uint32_t qr_hi = q_hi + 2 * a.rank * kRows, qr_lo = qr_hi + kRows * a.rope;
            const uint32_t p_hi = smem_u32(weights), p_lo = p_hi + kKeys * kRows;
            const uint32_t ring_u = smem_u32(ring), rope_u = smem_u32(rope_k);
            // Pieces of the next tile's scores that may be awaited before this tile's pieces are free.
            const int lead = min(pieces, a.slots - pieces);
            uint32_t tile_s = 0;              // tiles whose scores were issued
            uint32_t slot_s = 0, lap_s = 0;   // ring position of the scores
            uint32_t slot_o = 0;              // ring position of the outputs
            uint32_t item_count = 0;

            // Scores of one tile: pieces [c0, c1), the rope part before piece 0.
            const auto scores = [&](int c0, int c1) {
                const uint32_t d = tmem + kScoreCol + (tile_s & 1) * kRows;
                if (c0 == 0 && a.rope) {
                    wait(&ctl->rope_full, tile_s & 1);
                    tc_fence_after();
                    if (lane == 0) {
                        for (int k = 0; k < a.rope / 32; ++k) {
                            const uint64_t ka = smem_desc(rope_u + k * 32, a.rope);
                            mma_f8(d, ka, smem_desc(qr_hi + k * 32, a.rope), idesc_s, k != 0);
                            mma_f8(d, ka, smem_desc(qr_lo + k * 32, a.rope), idesc_s, true);
                        }
                        tc_commit(&ctl->rope_free);
                    }
                }
                for (int c = c0; c < c1; ++c) {
                    wait(&ctl->full[slot_s], lap_s & 1);
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t ka = smem_desc(ring_u + slot_s * kPiece, 128);
                        const uint64_t qa = smem_desc(q_hi + c * kRows * 128, 128);
                        const uint64_t qb = smem_desc(q_lo + c * kRows * 128, 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_f8(d, ka + k * 2, qa + k * 2, idesc_s, a.rope || c != 0 || k != 0);
                            mma_f8(d, ka + k * 2, qb + k * 2, idesc_s, true);
                        }
                    }
                    if (++slot_s == static_cast<uint32_t>(a.slots)) {
                        slot_s = 0;
                        ++lap_s;
                    }
                }
                if (c1 == pieces) {
                    if (lane == 0) tc_commit(&ctl->score_full[tile_s & 1]);
                    ++tile_s;
                }
                __syncwarp();
            };

            const uint32_t total = static_cast<uint32_t>(run_hi - run_lo);
            int left = 0;       // tiles of the current segment that follow this one
            bool first = true;  // the tile starts a segment
            long long pos = run_lo;
            wait(&ctl->q_ready, 0);
            tc_fence_after();
            scores(0, pieces);
            for (uint32_t i = 0; i < total; ++i) {
                if (first) {
                    left = static_cast<int>(min(static_cast<long long>(it.tiles - off), run_hi - pos));
                    off = 0;
                    pos += left;
                    next_item(a, it);
                }
                --left;
                const bool more = i + 1 < total, same = left > 0;
                if (more && same) scores(0, lead);
                wait(&ctl->weights_ready, i & 1);
                tc_fence_after();
                for (int c = 0; c < pieces; ++c) {
                    if (lane == 0) {
                        const uint32_t v = ring_u + slot_o * kPiece;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint64_t va = smem_desc(v + k * 4096, 128);
                            mma_f8(tmem + c * kRows, va, smem_desc(p_hi + k * 2048, 64), idesc_hi, !first || k != 0);
                            mma_f8(tmem + c * kRows, va, smem_desc(p_lo + k * 2048, 64), idesc_lo, true);
                        }
                        tc_commit(&ctl->freed[slot_o]);
                    }
                    if (++slot_o == static_cast<uint32_t>(a.slots)) slot_o = 0;
                }
                if (lane == 0) tc_commit(&ctl->out_done);
                __syncwarp();
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
            if (lane == 0) tc_commit(&ctl->drain);
            __syncwarp();
            (void)warp_wait_bounded(&ctl->drain, 0);
        } else {
            // ---------------------------------------------------------------- softmax
            const int key = tid & (kKeys - 1), half = tid >> 7, wq = warp & 3;
            const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
            const int col = half * 32 + lane;  // the column whose statistics this lane holds
            uint32_t tile = 0, slot = 0, top = 0;
            if (tid == 0) a.owner_flag[blockIdx.x] = 0;
            for (long long pos = run_lo; pos < run_hi;) {
                const int n = static_cast<int>(min(static_cast<long long>(it.tiles - off), run_hi - pos));
                // rows: consecutive (token, head) rows of q and out
                const int64_t row0 = (static_cast<int64_t>(it.start) + it.tok) * a.nh + it.block * a.heads_per;
                const int rows = a.head_blocks > 1 ? min(a.heads_per, a.nh - it.block * a.heads_per)
                                                   : min(a.group, it.t - it.tok) * a.nh;
                stage_q(a, ctl, smem, row0, rows, warp, lane);
                fence_async_smem();
                named_bar_sync(3, kSoftmaxWarps * 32);
                if (lane == 0) mbar_arrive(&ctl->q_ready);

                // keys that the column's token sees
                const int lim_col = max(0, min(it.vis, it.kv - it.t + it.tok + 1 +
                                                           (a.head_blocks > 1 ? 0 : min(col / a.nh, a.group - 1))));
                const int lim_min = max(0, min(it.vis, it.kv - it.t + it.tok + 1));
                float ref = kUnset;  // of column `col`
                float refs[32], sums[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    refs[c] = kUnset;
                    sums[c] = 0.f;
                }
                for (int i = off; i < off + n; ++i, ++tile) {
                    const int k = i * kKeys + key;
                    wait(&ctl->scale_full[tile & 1], (tile >> 1) & 1);
                    float sj = tile_scale[(tile & 1) * kKeys + key];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->scale_free[tile & 1]);
                    const bool in = k < it.vis;
                    if (!in || sj == 0.f) sj = 1.f;  // a zero row's codes are zeros
                    const float f = sj * a.scale_log2;
                    const float add = __log2f(sj), inv = sj == sj ? __fdiv_rn(1.f, sj) : 1.f;

                    wait(&ctl->score_full[tile & 1], (tile >> 1) & 1);
                    tc_fence_after();
                    float s[32];
                    tmem_ld32(tmem + lane_base + kScoreCol + (tile & 1) * kRows + half * 32, s);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 g = *reinterpret_cast<const float4 *>(&ctl->row_scale[half * 32 + c]);
                        s[c] = fmaf(s[c] * f, g.x, add);
                        s[c + 1] = fmaf(s[c + 1] * f, g.y, add);
                        s[c + 2] = fmaf(s[c + 2] * f, g.z, add);
                        s[c + 3] = fmaf(s[c + 3] * f, g.w, add);
                    }
                    if ((i + 1) * kKeys > lim_min) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (k >= __shfl_sync(kFullMask, lim_col, c)) s[c] = -INFINITY;
                    }
                    float mine = 0.f;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float m = warp_max(s[c]);
                        if (lane == c) mine = m;
                    }
                    // Maxima over the half's four warps.  Past this tile's barrier nobody reads the previous
                    // tile's entry any more, so it is cleared there for the tile after the next.
                    atomicMax(&ctl->tops[top][col], order_bits(mine));
                    named_bar_sync(1 + half, 128);
                    const float m = unorder_bits(ctl->tops[top][col]);
                    if (wq == 0) ctl->tops[top == 0 ? 2 : top - 1][col] = 0;
                    top = top == 2 ? 0 : top + 1;
                    const bool move = __any_sync(kFullMask, m > ref + kSlack);  // the same in the half's 4 warps
                    if (move) {
                        const float to = fmaxf(ref, m);
                        const float shrink = ex2(ref - to);
                        ref = to;
                        float by[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            refs[c] = __shfl_sync(kFullMask, ref, c);
                            by[c] = __shfl_sync(kFullMask, shrink, c);
                            sums[c] *= by[c];
                        }
                        if (i > off) {
                            wait(&ctl->out_done, (tile - 1) & 1);
                            tc_fence_after();
                            for (int p = 0; p < pieces; ++p) {
                                float o[32];
                                const uint32_t at = tmem + lane_base + p * kRows + half * 32;
                                tmem_ld32(at, o);
#pragma unroll
                                for (int c = 0; c < 32; ++c) o[c] *= by[c];
                                tmem_st32(at, o);
                            }
                            tc_wait_st();
                        }
                    }
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float p0 = ex2(s[c] - refs[c] + kBase), p1 = ex2(s[c + 1] - refs[c + 1] + kBase);
                        sums[c] = fmaf(p0, inv, sums[c]);
                        sums[c + 1] = fmaf(p1, inv, sums[c + 1]);
                        const uint32_t h = f32x2_to_f16x2(p0, p1);
                        const uint32_t q = f16x2_to_e4m3x2(h);
                        const uint32_t r = f16x2_to_e5m2x2(sub_f16x2(h, e4m3x2_to_f16x2(q)));
                        if (c & 2) {
                            hi[c / 4] |= q << 16;
                            lo[c / 4] |= r << 16;
                        } else {
                            hi[c / 4] = q;
                            lo[c / 4] = r;
                        }
                    }
                    if (tile >= 1) wait(&ctl->out_done, (tile - 1) & 1);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int at = swizzled(key, (half * 2 + q) * 16, 64);
                        *reinterpret_cast<uint4 *>(weights + at) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                        *reinterpret_cast<uint4 *>(weights + kKeys * kRows + at) =
                            make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
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

                // ------------------------------------------------------------ the segment's end
                wait(&ctl->out_done, (tile - 1) & 1);
                tc_fence_after();
                // The weights' shared memory is free: the four warps' sums meet there, in a fixed order.
                float *scratch = reinterpret_cast<float *>(weights);
                scratch[wq * kRows + col] = column_sums(sums, lane);
                named_bar_sync(1 + half, 128);
                const float sum = (scratch[col] + scratch[kRows + col]) +
                                  (scratch[2 * kRows + col] + scratch[3 * kRows + col]);
                const bool whole = off == 0 && n == it.tiles;
                const int here = 2 * static_cast<int>(blockIdx.x) + (pos == run_lo ? 0 : 1);
                const float scale_col = whole ? (sum == 0.f ? 0.f : __fdiv_rn(1.f, sum)) : 1.f;
#pragma unroll
                for (int c = 0; c < 32; ++c) refs[c] = __shfl_sync(kFullMask, scale_col, c);
                if (!whole) {
                    if (wq == 0) a.stats[here * kRows + col] = make_float2(ref, sum);
                    if (off == 0 && tid == 0) {  // this CTA holds the item's start: it names its parts
                        Owner &w = a.owner[blockIdx.x];
                        w.row0 = row0;
                        w.rows = rows;
                        w.slot = here;
                        w.last = static_cast<int>((pos + it.tiles - 1) / per);
                        a.owner_flag[blockIdx.x] = 1;
                    }
                }
                for (int p = 0; p < pieces; ++p) {
                    float o[32];
                    tmem_ld32(tmem + lane_base + p * kRows + half * 32, o);
                    const int dim = p * 128 + key;
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = refs[c] == 0.f ? 0.f : o[c] * refs[c];
                    if (!whole || !a.out_bf16) {
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
                named_bar_sync(3, kSoftmaxWarps * 32);  // the scratch and the row scales are free again
                pos += n;
                off = 0;
                if (pos < run_hi) next_item(a, it);
            }
        }
    } else if (tid == 0) {
        a.owner_flag[blockIdx.x] = 0;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the partial accumulators of the items that several CTAs shared.  CTA (x, y) serves rows
// y, y + gridDim.y, ... of the x-th such item; parts are added in CTA order.
constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const PagedArgs a, int grid) {
    __shared__ int found;
    __shared__ int counts[kCombineThreads / 32];
    __shared__ float weight[kMaxGrid];
    __shared__ float red[2][kCombineThreads / 32];
    __shared__ float4 other[128];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    if (tid == 0) found = -1;
    const bool flag = tid < grid && __ldcg(a.owner_flag + tid) != 0;
    const unsigned ballot = __ballot_sync(kFullMask, flag);
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int rank_of = __popc(ballot & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) rank_of += counts[w];
    if (flag && rank_of == static_cast<int>(blockIdx.x)) found = tid;
    __syncthreads();
    if (found < 0) return;
    const int cta = found;
    const Owner *op = a.owner + cta;
    const long long row0 = __ldcg(&op->row0);
    const int rows = __ldcg(&op->rows), slot0 = __ldcg(&op->slot), last = __ldcg(&op->last);
    const int parts = min(last, grid - 1) - cta + 1;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float2 st = make_float2(kUnset, 0.f);
        if (tid < parts) st = __ldcg(a.stats + (tid == 0 ? slot0 : 2 * (cta + tid)) * kRows + r);
        const float wm = warp_max(st.x);
        if (lane == 0) red[0][warp] = wm;
        __syncthreads();
        float top = red[0][0];
        for (int w = 1; w < kCombineThreads / 32; ++w) top = fmaxf(top, red[0][w]);
        const float w = ex2(st.x - top);
        const float l = warp_sum(w * st.y);
        if (lane == 0) red[1][warp] = l;
        __syncthreads();
        float total = 0.f;
        for (int k = 0; k < kCombineThreads / 32; ++k) total += red[1][k];
        if (tid < parts) weight[tid] = total == 0.f ? 0.f : __fdiv_rn(w, total);
        __syncthreads();
        // threads 0..127 take the even parts, 128..255 the odd ones; a thread holds four dims
        const int side = tid >> 7, d4 = tid & 127;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d4 * 4 < a.rank) {
#pragma unroll 4
            for (int k = side; k < parts; k += 2) {
                const int64_t s = k == 0 ? slot0 : 2 * (cta + k);
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part + (s * kRows + r) * a.rank) + d4);
                const float x = weight[k];
                if (x != 0.f) {  // an empty part's accumulator is not read into the sum
                    acc.x = fmaf(v.x, x, acc.x);
                    acc.y = fmaf(v.y, x, acc.y);
                    acc.z = fmaf(v.z, x, acc.z);
                    acc.w = fmaf(v.w, x, acc.w);
                }
            }
        }
        if (side == 1) other[d4] = acc;
        __syncthreads();
        if (side == 0 && d4 * 4 < a.rank) {
            const float4 b = other[d4];
            const int64_t at = (row0 + r) * a.rank + d4 * 4;
            const float4 o = make_float4(acc.x + b.x, acc.y + b.y, acc.z + b.z, acc.w + b.w);
            if (a.out_bf16) {
                __nv_bfloat162 v[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = *reinterpret_cast<uint2 *>(v);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = o;
            }
        }
        __syncthreads();
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
        cudaFuncSetAttribute(attn_paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
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

// Workspace: owner flags, owners, statistics, partial accumulators.
constexpr int64_t kFlagBytes = kMaxGrid * 4, kOwnerBytes = kMaxGrid * sizeof(Owner);
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
    return kFlagBytes + kOwnerBytes + stat_bytes(grid) + part_bytes(grid, kv_rank);
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
        n_pages > 0x7fffffffLL / page_size || max_pages < 0 || max_pages > 0x7fffffffLL / page_size ||
        !std::isfinite(scale))
        return MEMQ_ERR_SHAPE;
    if (n_tok == 0 || n_seq == 0) return MEMQ_OK;  // no query rows
    if (n_pages < 1 || max_pages < 1) return MEMQ_ERR_SHAPE;
    if (!q_lat || (d_rope > 0 && !q_pe) || !cache || !scales || !block_table || !kv_len || !cu_q || !out || !workspace)
        return MEMQ_ERR_NULL;
    const uintptr_t q_al = q_dtype == MEMQ_F32 ? 16 : 8, o_al = out_dtype == MEMQ_F32 ? 16 : 8;
    if (misaligned(q_lat, q_al) || (d_rope > 0 && misaligned(q_pe, q_al)) || misaligned(cache, 16) ||
        misaligned(scales, 16) || misaligned(block_table, 4) || misaligned(kv_len, 4) || misaligned(cu_q, 4) ||
        misaligned(out, o_al) || misaligned(workspace, 16))
        return MEMQ_ERR_ALIGN;
    int sms = 0, smem = 0;
    if (!device_info(sms, smem)) return MEMQ_ERR_LAUNCH;
    const int grid = std::min(sms, kMaxGrid);
    if (workspace_bytes < kFlagBytes + kOwnerBytes + stat_bytes(grid) + part_bytes(grid, kv_rank)) return MEMQ_ERR_SHAPE;

    PagedArgs a{};
    a.q_lat = q_lat;
    a.q_pe = q_pe;
    a.scales = scales;
    a.table = block_table;
    a.kv_len = kv_len;
    a.cu_q = cu_q;
    a.out = out;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.owner_flag = reinterpret_cast<int *>(ws);
    a.owner = reinterpret_cast<Owner *>(ws + kFlagBytes);
    a.stats = reinterpret_cast<float2 *>(ws + kFlagBytes + kOwnerBytes);
    a.part = reinterpret_cast<float *>(ws + kFlagBytes + kOwnerBytes + stat_bytes(grid));
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
    a.q_bf16 = q_dtype == MEMQ_BF16;
    a.out_bf16 = out_dtype == MEMQ_BF16;
    a.scale_log2 = scale * 1.4426950408889634f;
    const int fixed = smem_ring_off(kv_rank, d_rope) + smem_tail();
    a.slots = std::min(kMaxSlots, (smem - fixed) / kPiece);
    if (a.slots < kv_rank / 128 + 1) return MEMQ_ERR_LAUNCH;
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
    if (cudaLaunchKernelEx(&cfg, attn_paged_kernel, lat, rope, a) != cudaSuccess) return MEMQ_ERR_LAUNCH;
    const int64_t items = n_tok * a.head_blocks;  // at least the number of items
    const unsigned x = static_cast<unsigned>(std::min<int64_t>(items, grid));
    cfg.gridDim = dim3(x, std::max(1u, std::min(64u, 608u / x)));
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, combine_kernel, a, grid) == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}
