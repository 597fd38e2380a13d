// memq_attn_paged.cu -- memq_attn_paged: causal attention of a chunk of new tokens per sequence over a
// paged E4M3 cache of keys and values, heads in groups that share a kv head.
//
//   s_j = scale * ks_j * (q . k_j)          j <= position of the query's token
//   out = sum_j softmax(s)_j * vs_j * v_j   k_j, v_j codes, ks_j, vs_j the scales of their 16 tokens
//
// Codes are exact in f16 (cvt.rn.f16x2.e4m3x2), so both products are f16 products with f32 sums.  What is not
// a code is rounded to f16: a query row after a power of two that brings its largest element below 2^15 (of an
// f32 query the remainder, too, in a second product), and a weight, scaled by its values' scale,
//   p_j = 2^9 exp2(s_j + log2 vs_j - R)
// under a running reference R of the row that is never more than 6 (log2) behind the largest so far: eleven bits
// down to 2^-23 of the largest, steps of 2^-33 of it below; for f32 outputs the remainder is a second product.  The
// sum of weights is kept apart in f32, from p_j / vs_j.
//
// The single-token kernel: its time is the cache's bytes, so it is built around a stream.  A warp holds 16
// query rows (heads of a group, times tokens) as fragments of m16n8k16 products and runs through 32 keys a
// time; it works alone, with its own ring of TMA copies.  What of the list of all (sequence, kv head, 16
// rows, 32 keys) tiles a warp serves is one run of equal length, derived from the lengths on the device; the items
// that two or more warps share leave f32 pieces in the workspace, which a second kernel adds in order.
// The order of an inner product's terms is free, so lane (g, c) = (lane / 4, lane % 4) of a fragment takes 32 (or
// 16) consecutive bytes of key g, and of the values the 16 (8) columns from 16 g on: both are read from shared
// memory 16 bytes at once, and no code is moved between lanes.  The first tiles of a warp's next item are sent behind
// the last of this one, so the ring does not run dry between items.
// 64 sequences of up to 16384 rows, 64 query and 8 kv heads of 128: 213 to 221 us from run to run, 6.1 to 6.3 TB/s, 90 to
// 94% of the measured copy rate; one of 131071 rows: 47 us, 5.7 TB/s, and 7 for the pieces (8 items in 1216 runs).
// More than 16 rows of a kv head are items of their own, each of which reads the keys again (through L2): 4 tokens of 8
// heads over 32768 rows 35 us, where the cache's bytes take 9.9.  A short call is latency: of 14 us at
// 8192 rows the row kernel takes 10 (lengths, pages, scales and codes are read one behind another), the join 4.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "memq_attn.cuh"
#include "memq_attn_tiles.cuh"

namespace memq {
namespace {

constexpr int kRows = 16;   // query rows of a warp
constexpr int kKeys = 32;   // keys of a tile
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kWindow = 16;  // tiles whose pages and scales are looked up at once: two blocks a lane pair
constexpr int kStart = 2;    // tiles that starting an item counts as

template <int D>
struct Ring {
    static constexpr int kTile = 2 * kKeys * D;                  // bytes: keys, then values
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kWarpBytes = kStages * kTile;
    static constexpr int kBytes = kWarps * kWarpBytes;
};

__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + kKeys - 1) / kKeys); }

// 16 query rows of a (sequence, kv head) and their part of a run.
struct RowItem {
    int seq, head, row_tile, index;  // index: among all items
    AttnSeq s;
    int rows, row_tiles, units;  // of the sequence and head; tiles of an item and its start
    long long pos;               // of the item's first unit
    int off;                     // the first tile that the run serves
    bool live;
    int row0, n_rows, vis, end, t1;  // end: of the run's part; t1: of what is seen
    __device__ __forceinline__ void of_seq(const AttnArgs &a) {
        rows = s.t * a.group;
        row_tiles = (rows + kRows - 1) / kRows;
        units = tiles_of(s.kv) + kStart;
    }
    __device__ __forceinline__ void sizes(const AttnArgs &a, long long run_hi) {
        live = pos + kStart + off < run_hi;
        row0 = row_tile * kRows;
        n_rows = min(kRows, rows - row0);
        vis = max(0, s.kv - s.t + (row0 + n_rows - 1) / a.group + 1);
        end = static_cast<int>(min(static_cast<long long>(units - kStart), run_hi - pos - kStart));
        t1 = min(end, (vis + kKeys - 1) / kKeys);
    }
    __device__ __forceinline__ bool whole() const { return off == 0 && end == units - kStart; }
    __device__ __forceinline__ void advance(const AttnArgs &a, long long run_hi) {
        pos += units;
        off = 0;
        ++index;
        live = pos + kStart < run_hi;
        if (!live) return;
        if (++row_tile == row_tiles) {
            row_tile = 0;
            if (++head == a.n_kv) {
                head = 0;
                do {
                    if (++seq >= a.n_seq) {  // not with lengths that stand still
                        live = false;
                        return;
                    }
                    s = attn_seq(a, __ldcg(a.cu_q + seq), __ldcg(a.cu_q + seq + 1), __ldcg(a.kv_len + seq));
                    rows = s.t * a.group;
                } while (rows == 0 || rows < a.rows_from || rows > a.rows_to);
                of_seq(a);
            }
        }
        sizes(a, run_hi);
    }
};

struct Control {
    uint64_t full[kWarps][6];
    long long warp_sum[kWarps];
    int warp_items[kWarps];
    RowItem next[kWarps];  // of each warp
};

__host__ __device__ constexpr int smem_bytes(int ring) { return ring + 1024 + static_cast<int>(sizeof(Control)); }

template <int D, bool Q2, bool P2>
__global__ void __launch_bounds__(kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const AttnArgs a,
                     const int box) {
    constexpr int kSteps = D / 16;  // k16 steps of q . k; n8 columns of the values per thread group
    constexpr int kStages = Ring<D>::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFullMask, tid >> 5, 0);
    const int g = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + warp * Ring<D>::kWarpBytes;
    Control *ctl = reinterpret_cast<Control *>(smem + Ring<D>::kBytes);

    griddep_launch_dependents();
    if (tid == 0) {
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < kStages; ++i) mbar_init(&ctl->full[w][i], 1);
        mbar_init_fence();
    }
    // The tensor-core kernel lets this one start when all of its CTAs are past their own wait, so what came before is
    // there; nothing is taken from it or written where it writes.  This kernel's end still waits for it: the join
    // waits for this one alone.
    if (!a.behind_tiles) griddep_wait();

    // ------------------------------------------------------------------ the runs
    int4 *seqs = reinterpret_cast<int4 *>(smem);                            // (start, t, kv, items before)
    long long *first = reinterpret_cast<long long *>(smem + a.n_seq * 16);  // units before each sequence
    const int per_seq = (a.n_seq + kThreads - 1) / kThreads;
    bool descends = false;
    long long sum = 0;
    int items = 0;  // (at most 2^31: rows of q are)
    for (int i = 0; i < per_seq; ++i) {
        const int b = tid * per_seq + i;
        if (b >= a.n_seq) break;
        const int c0 = __ldcg(a.cu_q + b), c1 = __ldcg(a.cu_q + b + 1), kv = __ldcg(a.kv_len + b);
        if (c0 < 0 || c0 > c1 || c1 > a.n_tok || kv < 0 || kv > (static_cast<long long>(a.max_pages) << a.page_shift))
            atomicOr(&g_attn_fault, kAttnFaultInput);
        descends = descends || c0 > c1;
        const AttnSeq s = attn_seq(a, c0, c1, kv);
        const int rows = s.t * a.group;
        first[b] = sum;
        seqs[b] = make_int4(s.start, s.t, s.kv, items);
        if (rows >= a.rows_from && rows <= a.rows_to) {
            const int n = a.n_kv * ((rows + kRows - 1) / kRows);
            items += n;
            sum += static_cast<long long>(n) * (tiles_of(s.kv) + kStart);
        }
    }
    long long incl = sum;
    int items_incl = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(kFullMask, incl, o);
        const int up_items = __shfl_up_sync(kFullMask, items_incl, o);
        if (lane >= o) {
            incl += up;
            items_incl += up_items;
        }
    }
    if (lane == 31) {
        ctl->warp_sum[warp] = incl;
        ctl->warp_items[warp] = items_incl;
    }
    const bool nothing = __syncthreads_or(descends);
    long long before = incl - sum, total = 0;
    int items_before = items_incl - items, all_items = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            before += ctl->warp_sum[w];
            items_before += ctl->warp_items[w];
        }
        total += ctl->warp_sum[w];
        all_items += ctl->warp_items[w];
    }
    for (int i = 0; i < per_seq; ++i) {
        const int b = tid * per_seq + i;
        if (b >= a.n_seq) break;
        first[b] += before;
        seqs[b].w += items_before;
    }
    __syncthreads();
    const int run = blockIdx.x * kWarps + warp, runs = gridDim.x * kWarps;
    const long long per = max(static_cast<long long>(kStart + 1), (total + runs - 1) / runs);
    const long long run_lo = nothing ? total : run * per, run_hi = min(total, run_lo + per);
    RowItem it{};
    if (run_lo < run_hi) {
        int seq = 0, hi = a.n_seq;  // first[seq] <= run_lo < first[hi]
        while (hi - seq > 1) {
            const int mid = (seq + hi) >> 1;
            if (first[mid] <= run_lo) seq = mid; else hi = mid;
        }
        const int4 v = seqs[seq];
        it.seq = seq;
        it.s = AttnSeq{v.x, v.y, v.z};
        it.of_seq(a);
        const long long at = run_lo - first[seq];
        const int n = static_cast<int>(at / it.units), in_item = static_cast<int>(at - static_cast<long long>(n) * it.units);
        it.head = n / it.row_tiles;
        it.row_tile = n - it.head * it.row_tiles;
        it.index = v.w + n;
        it.off = max(0, in_item - kStart);
        it.pos = run_lo - in_item;
        it.sizes(a, run_hi);
    }
    fence_async_smem();
    __syncthreads();  // copies may go where the lengths lie
    // Owners are noted by run, or, where there are no more items than runs, by item: every item has one run that
    // serves its first tile.
    if (lane == 0 && (!a.by_item || nothing || run >= all_items)) a.owner[run].rows = 0;
    if (!it.live) {
        griddep_wait();
        return;
    }

    uint32_t sent = 0, taken = 0;  // tiles of the ring
    bool dead = false;
    // ---- pages and scales: lane l serves block l of a window of 32 blocks
    const auto page_of = [&](const RowItem &i, int tile) {  // -1: none; not checked yet
        const int key = tile * kKeys + lane * kAttnBlock;
        return tile < i.t1 && key < i.vis
                   ? __ldcg(a.table + static_cast<int64_t>(i.seq) * a.max_pages + (key >> a.page_shift))
                   : -1;
    };
    const auto row_of = [&](const RowItem &i, int page, int tile) {
        const int key = tile * kKeys + lane * kAttnBlock;
        return tile < i.t1 && key < i.vis ? attn_row(a, page, i.head, key) : -1;
    };
    const auto scale_at = [&](const float *scales, int row) { return row < 0 ? 1.f : __ldcg(scales + (row >> 4)); };
    const auto send = [&](int r0, int r1) {  // the copies of a tile's blocks
        if (lane == 0) {
            const uint32_t slot = sent % kStages;
            uint64_t *bar = &ctl->full[warp][slot];
            uint8_t *dst = ring + slot * Ring<D>::kTile;
            const int boxes = box < kKeys && r1 >= 0 ? 2 : 1;
            mbar_arrive_expect_tx(bar, 2 * boxes * box * D);
            tma_load_2d_plain(dst, &k_map, 0, r0, bar);
            tma_load_2d_plain(dst + kKeys * D, &v_map, 0, r0, bar);
            if (boxes == 2) {
                tma_load_2d_plain(dst + kAttnBlock * D, &k_map, 0, r1, bar);
                tma_load_2d_plain(dst + (kKeys + kAttnBlock) * D, &v_map, 0, r1, bar);
            }
        }
        ++sent;
    };
    int row_now = row_of(it, page_of(it, it.off), it.off);
    int early = 0;  // tiles of the item that were sent ahead of it
    while (it.live && !dead) {
        const int off = it.off, t1 = it.t1, vis = it.vis, row0 = it.row0, n_rows = it.n_rows;
        const int all_see = max(0, it.s.kv - it.s.t + row0 / a.group + 1);
        int win = off;
        int page_next = page_of(it, win + kWindow), page_later = page_of(it, win + 2 * kWindow);
        float ks_now = scale_at(a.k_scales, row_now), vs_now = scale_at(a.v_scales, row_now);
        int next_send = off + early;
        for (; next_send < t1 && sent - taken < kStages; ++next_send) {
            const int i = 2 * (next_send - win);
            send(__shfl_sync(kFullMask, row_now, i), __shfl_sync(kFullMask, row_now, i + 1));
        }
        // The item behind this one: its first tiles are sent as soon as this one's are.  It waits in shared memory.
        int row_then = -1, page_then = -1, sent_then = 0, most_then = 0;
        {
            RowItem next = it;
            next.advance(a, run_hi);
            if (next.live) {
                page_then = page_of(next, 0);
                most_then = min(next.t1, kWindow);
            }
            __syncwarp();
            if (lane == 0) ctl->next[warp] = next;
            __syncwarp();
        }

        // ---- the query rows
        uint32_t q_hi[kSteps][4], q_lo[Q2 ? kSteps : 1][4];
        float factor[2];  // of the scores, by row
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = g + 8 * k;
            float x[D / 4];
            const bool live = r < n_rows;
            const int rr = row0 + (live ? r : 0), tok = rr / a.group;
            const int64_t from = (static_cast<int64_t>(it.s.start) + tok) * a.q_stride +
                                 (it.head * a.group + rr - tok * a.group) * D + c * (D / 4);
            if (Q2) {
                const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + from);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const float4 v = live ? __ldcg(src + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[4 * i] = v.x;
                    x[4 * i + 1] = v.y;
                    x[4 * i + 2] = v.z;
                    x[4 * i + 3] = v.w;
                }
            } else {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + from);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 v = live ? __ldcg(src + i) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                    }
                }
            }
            uint32_t top = 0;  // as bits, infinities and NaN lie above all numbers
#pragma unroll
            for (int i = 0; i < D / 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
            top = max(top, __shfl_xor_sync(kFullMask, top, 1));
            top = max(top, __shfl_xor_sync(kFullMask, top, 2));
            // the largest comes to [2^14, 2^15); tiny rows keep a normal factor
            const int e = max(static_cast<int>(top >> 23), 32);
            const float inv = __uint_as_float(static_cast<uint32_t>(min(254, 127 + 14 - (e - 127))) << 23);
            const float back = __uint_as_float(static_cast<uint32_t>(max(1, 127 - 14 + (e - 127))) << 23);
            factor[k] = top < 0x7f800000u ? back * a.scale_log2 : NAN;
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float u = x[4 * j + 2 * i] * inv, v = x[4 * j + 2 * i + 1] * inv;
                    const uint32_t h = f32x2_to_f16x2(u, v);
                    q_hi[j][2 * i + k] = h;
                    if (Q2) q_lo[j][2 * i + k] = attn_rest(u, v, h);
                }
        }

        float o[kSteps * 2][4];  // column group j: columns of this thread 16 (2 c + i) + j
#pragma unroll
        for (int j = 0; j < kSteps * 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
        float ref[2] = {kAttnUnset, kAttnUnset}, total_w[2] = {0.f, 0.f};
        float lv_now = 0.f, inv_now = 1.f;
        int lim[2];  // keys that a row sees
#pragma unroll
        for (int k = 0; k < 2; ++k) lim[k] = min(vis, max(0, it.s.kv - it.s.t + (row0 + g + 8 * k) / a.group + 1));
        int row_next = row_of(it, page_next, win + kWindow);
        float ks_next = scale_at(a.k_scales, row_next), vs_next = scale_at(a.v_scales, row_next);
        if (most_then) row_then = row_of(ctl->next[warp], page_then, 0);
        const auto send_then = [&]() {
            const int i = 2 * sent_then++;
            send(__shfl_sync(kFullMask, row_then, i), __shfl_sync(kFullMask, row_then, i + 1));
        };
        while (next_send >= t1 && sent_then < most_then && sent - taken < kStages) send_then();

        for (int tile = off; tile < t1; ++tile) {
            if (tile - win == kWindow) {
                win = tile;
                row_now = row_next;
                ks_now = ks_next;
                vs_now = vs_next;
                row_next = row_of(it, page_later, win + kWindow);
                ks_next = scale_at(a.k_scales, row_next);
                vs_next = scale_at(a.v_scales, row_next);
                page_later = page_of(it, win + 2 * kWindow);
            }
            const uint32_t slot = taken % kStages;
            if (!warp_wait_bounded(&ctl->full[warp][slot], (taken / kStages) & 1)) {
                if (lane == 0) atomicOr(&g_attn_fault, kAttnFaultWait);
                dead = true;
                break;
            }
            ++taken;
            const uint8_t *kt = ring + slot * Ring<D>::kTile, *vt = kt + kKeys * D;
            const int key0 = tile * kKeys;
            const bool masked = key0 + kKeys > all_see;

            // ---- scores of 4 x 8 keys
            float sc[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int row = n * 8 + g;
                uint32_t w[D / 16];
                if (D == 128) {
                    const uint4 u = lds128(kt + row * 128 + ((2 * c ^ (row & 7)) << 4));
                    const uint4 v = lds128(kt + row * 128 + (((2 * c + 1) ^ (row & 7)) << 4));
                    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                    w[D / 16 - 4] = v.x; w[D / 16 - 3] = v.y; w[D / 16 - 2] = v.z; w[D / 16 - 1] = v.w;
                } else {
                    const uint4 u = lds128(kt + row * 64 + ((c ^ (row >> 1 & 3)) << 4));
                    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
                // f32 queries: the tensor cores' sums lose a bit with each step, so the remainders come first, while the sum
                // is small, and the row's halves are summed apart.
                if constexpr (Q2) {
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16x2x2(w[j], b0, b1);
                        mma_f16_16816(sc[n], q_lo[j][0], q_lo[j][1], q_lo[j][2], q_lo[j][3], b0, b1);
                    }
                }
                float upper[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16x2x2(w[j], b0, b1);
                    mma_f16_16816(Q2 && j >= kSteps / 2 ? upper : sc[n], q_hi[j][0], q_hi[j][1], q_hi[j][2], q_hi[j][3], b0, b1);
                }
                if constexpr (Q2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[n][i] += upper[i];
                }
            }
            // ---- their maxima, with the values' scales
            float lv[2], inv_vs[2];
            const int i0 = 2 * (tile - win);
            if (tile == win) {  // log2 and reciprocal of the window's value scales; exact for powers of two
                const float v = vs_now < kAttnLeastScale ? kAttnLeastScale : vs_now;
                lv_now = attn_log2(v);
                inv_now = __frcp_rn(v);
            }
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float ks = __shfl_sync(kFullMask, ks_now, i0 + b);
                lv[b] = __shfl_sync(kFullMask, lv_now, i0 + b);
                inv_vs[b] = __shfl_sync(kFullMask, inv_now, i0 + b);
                const float least = fmaxf(lv[b], kAttnLeastLog);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float f = factor[k] * ks;
                    float m = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &x = sc[2 * b + n][2 * k + i];
                            x *= f;
                            if (masked && key0 + b * 16 + n * 8 + 2 * c + i >= lim[k]) x = -INFINITY;
                            m = fmaxf(m, x);
                        }
                    top[k] = fmaxf(top[k], m + least);
                }
            }
            const bool move = top[0] > ref[0] + kAttnSlack || top[1] > ref[1] + kAttnSlack;
            if (__any_sync(kFullMask, move)) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float m = fmaxf(top[k], __shfl_xor_sync(kFullMask, top[k], 1));
                    m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 2));
                    const float to = fmaxf(ref[k], m), by = ex2(ref[k] - to);
                    ref[k] = to;
                    total_w[k] *= by;
#pragma unroll
                    for (int j = 0; j < kSteps * 2; ++j) {
                        o[j][2 * k] *= by;
                        o[j][2 * k + 1] *= by;
                    }
                }
            }
            // ---- weights
            uint32_t p_hi[2][4], p_lo[P2 ? 2 : 1][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float shift = lv[b] - ref[k] + kAttnTop;
                    const float back = inv_vs[b];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float p0 = ex2(sc[2 * b + n][2 * k] + shift), p1 = ex2(sc[2 * b + n][2 * k + 1] + shift);
                        total_w[k] = fmaf(p0 + p1, back, total_w[k]);
                        const uint32_t h = f32x2_to_f16x2(p0, p1);
                        p_hi[b][2 * n + k] = h;
                        if (P2) p_lo[P2 ? b : 0][2 * n + k] = attn_rest(p0, p1, h);
                    }
                }
            // ---- values
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t w[4][D / 32];  // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = b * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
                    if (D == 128) {
                        const uint4 u = lds128(vt + row * 128 + ((g ^ (row & 7)) << 4));
                        w[i][0] = u.x; w[i][1] = u.y; w[i][D / 32 - 2] = u.z; w[i][D / 32 - 1] = u.w;
                    } else {
                        const uint2 u = lds64(vt + row * 64 + (((g >> 1) ^ (row >> 1 & 3)) << 4) + (g & 1) * 8);
                        w[i][0] = u.x; w[i][1] = u.y;
                    }
                    if (masked && key0 + row >= vis) {  // zero weights must meet finite codes
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) w[i][j] = 0;
                    }
                }
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    uint32_t lo[4], hi[4];
                    e4m3x4_to_f16x2x2(__byte_perm(w[0][j], w[1][j], 0x5140), lo[0], lo[1]);
                    e4m3x4_to_f16x2x2(__byte_perm(w[0][j], w[1][j], 0x7362), lo[2], lo[3]);
                    e4m3x4_to_f16x2x2(__byte_perm(w[2][j], w[3][j], 0x5140), hi[0], hi[1]);
                    e4m3x4_to_f16x2x2(__byte_perm(w[2][j], w[3][j], 0x7362), hi[2], hi[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (P2) {
                            // f32 outputs: a block's products are summed apart, for the tensor cores truncate as they
                            // add to a long sum (64 x 16384 keys: thousands of steps)
                            float t[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16_16816(t, p_lo[b][0], p_lo[b][1], p_lo[b][2], p_lo[b][3], lo[i], hi[i]);
                            mma_f16_16816(t, p_hi[b][0], p_hi[b][1], p_hi[b][2], p_hi[b][3], lo[i], hi[i]);
#pragma unroll
                            for (int m = 0; m < 4; ++m) o[4 * j + i][m] += t[m];
                        } else {
                            mma_f16_16816(o[4 * j + i], p_hi[b][0], p_hi[b][1], p_hi[b][2], p_hi[b][3], lo[i], hi[i]);
                        }
                    }
                }
            }
            __syncwarp();  // all lanes have read the slot
            if (next_send < t1) {
                const int i = 2 * (next_send++ - win);
                const int from = i < 32 ? row_now : row_next;
                send(__shfl_sync(kFullMask, from, i & 31), __shfl_sync(kFullMask, from, (i + 1) & 31));
            } else if (sent_then < most_then) {
                send_then();
            }
        }
        if (dead) break;

        // ---- the way out: columns 16 (2 c + i) + j of rows g and g + 8 (D = 128)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            total_w[k] += __shfl_xor_sync(kFullMask, total_w[k], 1);
            total_w[k] += __shfl_xor_sync(kFullMask, total_w[k], 2);
        }
        const bool whole = it.whole();
        const int piece = 2 * run + (off == 0 ? 1 : 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = g + 8 * k;
            if (r >= n_rows) continue;
            constexpr int kCols = D / 8;  // columns of one n8 index
            if (whole) {
                const float n = total_w[k] == 0.f ? 0.f : __fdiv_rn(1.f, total_w[k]);
                const int64_t to = attn_out_at(a, it.s.start, it.head, row0 + r, D) + c * 2 * kCols;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (a.out_bf16) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to + i * kCols);
#pragma unroll
                        for (int j = 0; j < kCols / 8; ++j) {
                            __nv_bfloat162 v[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                v[m] = __floats2bfloat162_rn(o[8 * j + 2 * m][2 * k + i] * n, o[8 * j + 2 * m + 1][2 * k + i] * n);
                            dst[j] = *reinterpret_cast<uint4 *>(v);
                        }
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to + i * kCols);
#pragma unroll
                        for (int j = 0; j < kCols / 4; ++j)
                            dst[j] = make_float4(o[4 * j][2 * k + i] * n, o[4 * j + 1][2 * k + i] * n,
                                                 o[4 * j + 2][2 * k + i] * n, o[4 * j + 3][2 * k + i] * n);
                    }
                }
            } else {
                if (c == 0) a.stats[piece * kRows + r] = make_float2(ref[k], total_w[k]);
                float *to = a.part + (static_cast<int64_t>(piece) * kRows + r) * D + c * 2 * kCols;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < kCols / 4; ++j)
                        reinterpret_cast<float4 *>(to + i * kCols)[j] =
                            make_float4(o[4 * j][2 * k + i], o[4 * j + 1][2 * k + i], o[4 * j + 2][2 * k + i],
                                        o[4 * j + 3][2 * k + i]);
            }
        }
        if (off == 0 && lane == 0 && (!whole || a.by_item)) {
            AttnOwner own;
            own.start = it.s.start;
            own.row0 = row0;
            own.first = run;
            own.last = static_cast<int>((it.pos + it.units - 1) / per);
            own.head = it.head;
            own.rows = whole ? 0 : n_rows;
            if (!a.by_item || it.index < runs) a.owner[a.by_item ? it.index : run] = own;
        }
        it = ctl->next[warp];
        row_now = row_then;
        early = sent_then;
    }
    // (no owner's note stays what it was before the call)
    for (; dead && a.by_item && it.live; it.advance(a, run_hi))
        if (it.off == 0 && lane == 0 && it.index < runs) a.owner[it.index].rows = 0;
    if (dead) {  // copies in flight land before shared memory is given up, each wait bounded
        for (uint32_t i = taken; i != sent; ++i)
            (void)warp_wait_bounded(&ctl->full[warp][i % kStages], (i / kStages) & 1);
    }
    griddep_wait();
}

// Adds the pieces of the items that several runs shared, in the runs' order.  CTAs (x, 0 .. gridDim.y - 1) serve the
// x-th such item.  Up to kFewParts pieces a warp adds a row's alone, eight rows under way; above, the CTA's warps add
// every eighth and the eight sums are added in turn (one token over 131071 keys: 152 pieces an item; a warp alone
// took 55 us).  A join of few CTAs is latency, so its pieces are fetched EARLY, while their weights are formed, which takes
// 180 registers: 1 x 131071 56.6 -> 53.7 us, 1 x 8192 15.4 -> 13.8; one of many keeps 48 (2048 tokens over 2048 rows 117,
// early 142).
constexpr int kFewParts = 24;

struct JoinPart {
    const AttnOwner *owner;
    const float2 *stats;
    const float *part;
    int x, share;      // owners to look at, CTAs for each
    int runs, stride;  // runs, rows of a piece
};

template <int D, bool EARLY>
__global__ void __launch_bounds__(kThreads, EARLY ? 1 : 5) attn_join_kernel(const AttnArgs a, const JoinPart tiles, const JoinPart rows) {
    constexpr int E = D / 32;
    __shared__ float red[2][kWarps];
    __shared__ float sums[kWarps][D];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int of_tiles = tiles.x * tiles.share, cta = static_cast<int>(blockIdx.x);
    const JoinPart &p = cta < of_tiles ? tiles : rows;
    const int runs = p.runs, stride = p.stride, in_part = cta < of_tiles ? cta : cta - of_tiles;
    const int y = in_part % p.share;  // of the item's CTAs
    const int4 *at = reinterpret_cast<const int4 *>(p.owner + in_part / p.share);
    const int4 raw[2] = {__ldcg(at), __ldcg(at + 1)};
    const AttnOwner owner = *reinterpret_cast<const AttnOwner *>(raw);
    if (owner.rows == 0) return;
    if (!attn_owner_ok(owner, a.n_tok, a.n_kv, a.group, runs, stride)) {
        if (tid == 0) atomicOr(&g_attn_fault, kAttnFaultInput);
        return;
    }
    const int run = owner.first, parts = min(owner.last, runs - 1) - run + 1;
    const auto put = [&](int r, const float(&v)[E], float total) {
        const float n = total == 0.f ? 0.f : __fdiv_rn(1.f, total);
        const int64_t to = attn_out_at(a, owner.start, owner.head, owner.row0 + r, D) + lane * E;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            if (a.out_bf16)
                *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + to + i) =
                    __floats2bfloat162_rn(v[i] * n, v[i + 1] * n);
            else
                *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + to + i) = make_float2(v[i] * n, v[i + 1] * n);
        }
    };
    const auto slot_of = [&](int k, int r) { return static_cast<int64_t>(k == 0 ? 2 * run + 1 : 2 * (run + k)) * stride + r; };
    const auto fetch = [&](float(&v)[E], int64_t slot) {
        const float *src = p.part + slot * D + lane * E;
        if (E == 4) {
            const float4 u = __ldcg(reinterpret_cast<const float4 *>(src));
            v[0] = u.x;
            v[1] = u.y;
            v[E - 2] = u.z;
            v[E - 1] = u.w;
        } else {
            const float2 u = __ldcg(reinterpret_cast<const float2 *>(src));
            v[0] = u.x;
            v[1] = u.y;
        }
    };
    const auto add = [&](float(&acc)[E], const float(&v)[E], float by) {
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = fmaf(v[i], by, acc[i]);
    };
    if (parts <= kFewParts) {
        for (int r = y * kWarps + warp; r < owner.rows; r += p.share * kWarps) {
            float2 st = make_float2(kAttnUnset, 0.f);
            if (lane < parts) st = __ldcg(p.stats + slot_of(lane, r));
            float v[EARLY ? kFewParts : 1][E];  // past the last piece: the last again, with weight 0
            if constexpr (EARLY) {
#pragma unroll
                for (int k0 = 0; k0 < kFewParts; k0 += 8)
                    if (k0 < parts) {
#pragma unroll
                        for (int k = k0; k < k0 + 8; ++k) fetch(v[k], slot_of(min(k, parts - 1), r));
                    }
            }
            const float w = ex2(st.x - warp_max(st.x)), total = warp_sum(st.y * w);
            float acc[E];
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = 0.f;
#pragma unroll(EARLY ? kFewParts / 8 : 1)
            for (int k0 = 0; k0 < kFewParts && (EARLY || k0 < parts); k0 += 8) {
                if (EARLY && k0 >= parts) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!EARLY) fetch(v[0], slot_of(min(k0 + i, parts - 1), r));
                    const float by = __shfl_sync(kFullMask, w, (k0 + i) & 31);
                    add(acc, v[EARLY ? k0 + i : 0], k0 + i < parts ? by : 0.f);
                }
            }
            put(r, acc, total);
        }
        return;
    }
    for (int r = y; r < owner.rows; r += p.share) {
        float v[EARLY ? 16 : 1][E], top = kAttnUnset;
        const auto fetch16 = [&](int k0) {  // of this warp's: every eighth from k0 on
#pragma unroll
            for (int i = 0; i < 16; ++i) fetch(v[EARLY ? i : 0], slot_of(min(k0 + i * kWarps, parts - 1), r));
        };
        if (EARLY) fetch16(warp);
        for (int k = tid; k < parts; k += kThreads) top = fmaxf(top, __ldcg(p.stats + slot_of(k, r)).x);
        top = warp_max(top);
        if (lane == 0) red[0][warp] = top;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red[0][w]);
        float acc[E], total = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.f;
        // warp w adds pieces w, w + 8, ..: 32 of them a turn
        for (int k0 = warp; k0 < parts; k0 += 32 * kWarps) {
            const int k = k0 + lane * kWarps;
            float w = 0.f;
            if (k < parts) {
                const float2 st = __ldcg(p.stats + slot_of(k, r));
                w = ex2(st.x - top);
                total += st.y * w;
            }
            const int n = min(32, (parts - k0 + kWarps - 1) / kWarps);
            for (int i0 = 0; i0 < n; i0 += 16) {
                if (EARLY && (k0 != warp || i0 != 0)) fetch16(k0 + i0 * kWarps);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!EARLY) fetch(v[0], slot_of(min(k0 + (i0 + i) * kWarps, parts - 1), r));
                    const float by = __shfl_sync(kFullMask, w, (i0 + i) & 31);
                    add(acc, v[EARLY ? i : 0], i0 + i < n ? by : 0.f);
                }
            }
        }
        total = warp_sum(total);
        if (lane == 0) red[1][warp] = total;
#pragma unroll
        for (int i = 0; i < E; ++i) sums[warp][lane * E + i] = acc[i];
        __syncthreads();
        if (warp == 0) {
            total = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = 0.f;
            for (int w = 0; w < kWarps; ++w) {
                total += red[1][w];
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] += sums[w][lane * E + i];
            }
            put(r, acc, total);
        }
        __syncthreads();  // the shared arrays are free for the next row
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

// Rows of d codes; a box of `rows` whole rows, swizzled over a row.
bool encode_rows(CUtensorMap *map, const void *base, int d, uint64_t n, uint32_t rows) {
    const EncodeTiledFn enc = encode_tiled();
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), n};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), rows}, step[2] = {1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

template <int D, bool Q2, bool P2>
bool allow() {
    return cudaFuncSetAttribute(attn_rows_kernel<D, Q2, P2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_bytes(Ring<D>::kBytes)) == cudaSuccess &&
           cudaFuncSetAttribute(attn_tiles_kernel<D, Q2, P2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                TileShape<D, Q2, P2>::kBytes) == cudaSuccess;
}

// SM count of the current device, after allowing the kernels their shared memory (once per device).
bool device_info(int &sms) {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < kMaxDevices && (sms = cache[dev].load(std::memory_order_acquire)) > 0) return true;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || !allow<64, false, false>() ||
        !allow<64, false, true>() || !allow<64, true, false>() || !allow<64, true, true>() || !allow<128, false, false>() ||
        !allow<128, false, true>() || !allow<128, true, false>() || !allow<128, true, true>())
        return false;
    if (dev < kMaxDevices) cache[dev].store(sms, std::memory_order_release);
    return true;
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Workspace: owners, statistics and pieces of one kernel; both kernels' lie behind one another.
struct Workspace {
    int runs, rows;
    int64_t owners, stats, parts;
    Workspace(int runs_, int rows_, int d)
        : runs(runs_), rows(rows_), owners((static_cast<int64_t>(runs) * sizeof(AttnOwner) + 255) / 256 * 256),
          stats(static_cast<int64_t>(2) * runs * rows * sizeof(float2)),
          parts(static_cast<int64_t>(2) * runs * rows * d * sizeof(float)) {}
    int64_t bytes() const { return owners + stats + parts; }
    void place(AttnArgs &a, uint8_t *at) const {
        a.owner = reinterpret_cast<AttnOwner *>(at);
        a.stats = reinterpret_cast<float2 *>(at + owners);
        a.part = reinterpret_cast<float *>(at + owners + stats);
    }
};
int64_t workspace_need(int grid, int d) { return Workspace(grid * kWarps, kRows, d).bytes() + Workspace(grid, 256, d).bytes(); }
// Sequences of more query rows (heads of a group, times tokens) than this take the tensor-core kernel.  us with 16 /
// 32 / 64, 64 query and 8 kv heads of 128: 4 tokens (32 rows) over 32768 rows 41.9 / 35.2 / 35.2, 48 sequences of 4 over
// 4096 169 / 149 / 150; 8 tokens (64 rows) over 32768 43.1 / 42.8 / 50.9, 48 sequences of 8 172 / 172 / 271.
constexpr int kRowsKernelMost = 32;

}  // namespace
}  // namespace memq

// Internal: this translation unit's device fault word (not part of the public header).
int memq_internal_fault_attn(unsigned int *out, bool clear) {
    if (cudaMemcpyFromSymbol(out, memq::g_attn_fault, sizeof(unsigned int)) != cudaSuccess) return 1;
    if (!clear) return 0;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(memq::g_attn_fault, &zero, sizeof(zero)) == cudaSuccess ? 0 : 1;
}

extern "C" int64_t memq_attn_paged_workspace(int d) {
    using namespace memq;
    if (d != 64 && d != 128) return -1;
    int sms = 0;
    if (!device_info(sms)) return -1;
    return workspace_need(std::min(sms, kAttnMaxGrid), d);
}

extern "C" int memq_attn_paged(int q_dtype, const void *q, int64_t q_stride, const uint8_t *k_cache,
                               const float *k_scales, const uint8_t *v_cache, const float *v_scales,
                               const int32_t *block_table, const int32_t *kv_len, const int32_t *cu_q, int out_dtype,
                               void *out, void *workspace, int64_t workspace_bytes, int64_t n_tok, int n_seq, int nh,
                               int n_kv, int d, int64_t n_pages, int page_size, int max_pages, float scale, void *stream) {
    using namespace memq;
    if ((q_dtype != MEMQ_F32 && q_dtype != MEMQ_BF16) || (out_dtype != MEMQ_F32 && out_dtype != MEMQ_BF16))
        return MEMQ_ERR_SHAPE;
    if (n_tok < 0 || n_tok > (1 << 24) || n_seq < 0 || n_seq > kAttnMaxSeqs || nh < 1 || nh > 1024 || n_kv < 1 ||
        nh % n_kv != 0 || n_tok * nh > 0x7fffffffLL || (d != 64 && d != 128) || page_size < 16 || page_size > 1024 ||
        (page_size & (page_size - 1)) != 0 || n_pages < 0 || n_pages > 0x7fffffffLL / page_size / n_kv || max_pages < 0 ||
        max_pages > kAttnMaxCached / page_size || !std::isfinite(scale * kAttnLog2e) || q_stride < 0 ||
        q_stride > (int64_t{1} << 38))
        return MEMQ_ERR_SHAPE;
    if (n_tok == 0 || n_seq == 0) return MEMQ_OK;  // no query rows
    if (n_pages < 1 || max_pages < 1) return MEMQ_ERR_SHAPE;
    if (!q || !k_cache || !k_scales || !v_cache || !v_scales || !block_table || !kv_len || !cu_q || !out || !workspace)
        return MEMQ_ERR_NULL;
    const int64_t size = q_dtype == MEMQ_F32 ? 4 : 2;
    if (misaligned(q, 16) || (n_tok > 1 && (q_stride * size) % 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
        misaligned(k_scales, 4) || misaligned(v_scales, 4) || misaligned(block_table, 4) || misaligned(kv_len, 4) ||
        misaligned(cu_q, 4) || misaligned(out, 16) || misaligned(workspace, 16))
        return MEMQ_ERR_ALIGN;
    int sms = 0;
    if (!device_info(sms)) return MEMQ_ERR_LAUNCH;
    const int grid = std::min(sms, kAttnMaxGrid), runs = grid * kWarps;
    if (workspace_bytes < workspace_need(grid, d)) return MEMQ_ERR_SHAPE;

    AttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.table = block_table;
    a.kv_len = kv_len;
    a.cu_q = cu_q;
    a.out = out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.n_tok = static_cast<int>(n_tok);
    a.n_seq = n_seq;
    a.nh = nh;
    a.n_kv = n_kv;
    a.group = nh / n_kv;
    a.n_pages = static_cast<int>(n_pages);
    a.page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
    a.max_pages = max_pages;
    a.rows_from = 1;
    a.rows_to = 0x7fffffff;
    // at least as many items as there are; the workspace notes them by item where they are no more than the runs
    const auto items_of = [&](int rows) { return n_kv * (n_tok * a.group / rows + std::min<int64_t>(n_seq, n_tok)); };
    a.by_item = items_of(kRows) <= runs;
    a.out_bf16 = out_dtype == MEMQ_BF16;
    a.scale_log2 = scale * kAttnLog2e;
    const int box = std::min(page_size, kKeys);
    const uint64_t pool = static_cast<uint64_t>(n_pages) * page_size * n_kv;
    CUtensorMap k_map, v_map;
    if (!encode_rows(&k_map, k_cache, d, pool, box) || !encode_rows(&v_map, v_cache, d, pool, box)) return MEMQ_ERR_LAUNCH;

    cudaLaunchConfig_t cfg = {};
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool q2 = q_dtype == MEMQ_F32, p2 = out_dtype == MEMQ_F32;
    const Workspace of_rows(runs, kRows, d), of_tiles(grid, q2 || p2 ? 128 : 256, d);
    // One token a sequence, or rows that no sequence can have more of than a warp holds: the stream of keys is
    // all.  (More tokens than sequences may still lie in short ones: each kernel takes its own.  No more tokens than
    // sequences may be one sequence's, which the lengths on the device tell too late: a chunk of 200 over 4096 rows takes
    // 54 us alone and 129 in 256 slots of which the others are empty.)
    const bool rows_only = n_tok <= n_seq || n_tok * a.group <= kRowsKernelMost;
    JoinPart tiles{};
    if (!rows_only) {
        AttnArgs t = a;
        t.rows_from = kRowsKernelMost + 1;
        t.by_item = false;
        of_tiles.place(t, static_cast<uint8_t *>(workspace) + of_rows.bytes());
        a.rows_to = kRowsKernelMost;
        a.behind_tiles = true;
        using Tiles = void (*)(const AttnArgs);
        static constexpr Tiles kTiles[2][2][2] = {
            {{attn_tiles_kernel<64, false, false>, attn_tiles_kernel<64, false, true>},
             {attn_tiles_kernel<64, true, false>, attn_tiles_kernel<64, true, true>}},
            {{attn_tiles_kernel<128, false, false>, attn_tiles_kernel<128, false, true>},
             {attn_tiles_kernel<128, true, false>, attn_tiles_kernel<128, true, true>}}};
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(kTileThreads);
        static constexpr int kTileBytes[2][2][2] = {
            {{TileShape<64, false, false>::kBytes, TileShape<64, false, true>::kBytes},
             {TileShape<64, true, false>::kBytes, TileShape<64, true, true>::kBytes}},
            {{TileShape<128, false, false>::kBytes, TileShape<128, false, true>::kBytes},
             {TileShape<128, true, false>::kBytes, TileShape<128, true, true>::kBytes}}};
        cfg.dynamicSmemBytes = static_cast<size_t>(kTileBytes[d == 128][q2][p2]);
        if (cudaLaunchKernelEx(&cfg, kTiles[d == 128][q2][p2], t) != cudaSuccess) return MEMQ_ERR_LAUNCH;
        tiles = JoinPart{t.owner, t.stats, t.part, of_tiles.runs, 16, of_tiles.runs, of_tiles.rows};
    }
    of_rows.place(a, static_cast<uint8_t *>(workspace));
    using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const AttnArgs, const int);
    static constexpr Kernel kKernels[2][2][2] = {
        {{attn_rows_kernel<64, false, false>, attn_rows_kernel<64, false, true>},
         {attn_rows_kernel<64, true, false>, attn_rows_kernel<64, true, true>}},
        {{attn_rows_kernel<128, false, false>, attn_rows_kernel<128, false, true>},
         {attn_rows_kernel<128, true, false>, attn_rows_kernel<128, true, true>}}};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes(d == 128 ? Ring<128>::kBytes : Ring<64>::kBytes));
    if (cudaLaunchKernelEx(&cfg, kKernels[d == 128][q2][p2], k_map, v_map, a, box) != cudaSuccess) return MEMQ_ERR_LAUNCH;
    // about eight CTAs an SM over the row kernel's items, 16 rows or fewer a CTA of the other's
    const int x = a.by_item ? static_cast<int>(items_of(kRows)) : runs;
    const JoinPart rows{a.owner, a.stats, a.part, x, std::max(1, std::min(kRows, 8 * grid / x)), runs, kRows};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles.x * tiles.share + rows.x * rows.share));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 0;
    using Join = void (*)(const AttnArgs, const JoinPart, const JoinPart);
    static constexpr Join kJoins[2][2] = {{attn_join_kernel<64, false>, attn_join_kernel<64, true>},
                                          {attn_join_kernel<128, false>, attn_join_kernel<128, true>}};
    const bool early = cfg.gridDim.x <= static_cast<unsigned>(2 * grid);
    return cudaLaunchKernelEx(&cfg, kJoins[d == 128][early], a, tiles, rows) == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}
