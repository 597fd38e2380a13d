// memq_attn_tiles.cuh -- the tensor-core kernel of memq_attn_paged, for chunks of many query rows.
//
// A CTA serves 128 or 256 rows (heads of a group, times tokens) of one kv head, 128 keys a time:
//   S [128 rows x 128 keys] = Q [128 x d] . K^T     kind::f16, both from shared memory
//   O [128 rows x d]       += P [128 x 128] . V     P from TMEM, where it takes the place of its scores
// Both products are f16: the codes are widened to f16 in shared memory (64 KB of writes a tile, against 256 KB that the
// products read), the query rows and the weights rounded to it.  Two blocks of 128 rows take turns, and a block's
// scores are formed in halves of 64 keys with columns of their own: while the weights of one half are formed, the
// tensor cores run the products of the others.  (With one set of columns a block: 1170 us where this took 865.)
//
// Warps 0-3 and 4-7 form the weights of the two blocks, a thread a row, so that a row's maximum and sum need no
// exchange; warps 8-11 and 13-15 load codes of keys and of values, a tile ahead in registers, and widen them; one thread
// of warp 12 issues the products, and waits for itself (as a warp with votes: 1090).  An f32 query has two terms, two
// products, and its 128 rows the shared memory of 256.
//
// What bounds it, of 2048 tokens over 16384 rows with 64 query and 8 kv heads of 128 (841 to 851 us, 1.21 to 1.23 PFLOP/s,
// 64 to 65% of the measured bf16 peak): a half's weights take a warp some 1000 cycles besides 500 of waits and hand-over (two warps a
// scheduler: 64 exp2 each are 512), the tensor cores 640 a block and half (QK^T as m128n64 is bound by shared memory, 48
// cycles an instruction).  What bounds the rest has not been found: without exp2, widening, loads and 7 of 8 products it
// still takes 80% of the time.  f32 calls, two products of scores and two of outputs, 2048 tokens over 8192 rows: 886 us
// (bf16 435).
#pragma once

#include <type_traits>

#include "memq_attn.cuh"

namespace memq {

constexpr int kTileKeys = 128, kHalfKeys = 64;
constexpr int kTileThreads = 16 * 32;
// Registers a thread: 128 at launch; the two warpgroups that hold scores take 152, the others give theirs
// (168 and 88 spill in the others: 192 bytes of stack).
constexpr int kRegsWeights = 152, kRegsOthers = 104;
static_assert(2 * kRegsWeights + 2 * kRegsOthers <= 4 * 128, "a split beyond the launch's registers never comes");
constexpr int kWidenWarp = 8, kIssueWarp = 12;
constexpr int kTileStart = 3;  // tiles that starting an item counts as

struct TileItem {
    int seq, head, row_tile;
    AttnSeq s;
    int rows;           // of the sequence and kv head: t * group
    int row0, n_rows;   // of the item
    int vis, tiles;     // keys that its last row sees; tiles, one at least
};

struct TileControl {
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
    uint64_t scores[2][2], weights[2][2];  // by block of rows and half of the keys
    uint64_t q_ready, drain;
    uint32_t tmem;
    int first_off;
    long long first_pos;
    TileItem first;
    long long warp_sum[16];
    float4 scale[4][8];   // of a tile's blocks of keys: k's, log2 v's, 1 / v's, and log2 v's for the reference
    float factor[256];
};

template <int R>
__device__ __forceinline__ void set_registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

template <int D, bool Q2, bool P2>
struct TileShape {
    // Blocks of 128 rows.  f32 queries need the second one's shared memory, f32 outputs its columns: the tensor cores
    // truncate as they add to a long sum, so the weights' remainders and every other tile have sums of their own
    // (error of 300 rows over 4000 keys against 64 bits 6.3e-6 with one sum, 1.4e-6 that of f32 arithmetic).
    static constexpr int kBlocks = Q2 || P2 ? 1 : 2;
    static constexpr int kRows = kBlocks * 128;
    static constexpr int kQ = 2 * 128 * D * 2;                  // two blocks, or two terms of one
    static constexpr int kKv = kTileKeys * D * 2;
    static constexpr int kBytes = kQ + 4 * kKv + static_cast<int>(sizeof(TileControl));
};

__device__ __forceinline__ void tile_sizes(const AttnArgs &a, int rows_per, TileItem &it) {
    it.row0 = it.row_tile * rows_per;
    it.n_rows = min(rows_per, it.rows - it.row0);
    it.vis = max(0, it.s.kv - it.s.t + (it.row0 + it.n_rows - 1) / a.group + 1);
    it.tiles = max(1, (it.vis + kTileKeys - 1) / kTileKeys);
}

__device__ __forceinline__ bool tile_served(const AttnArgs &a, int rows) { return rows >= a.rows_from && rows <= a.rows_to; }

// Order: sequences, blocks of rows, kv heads.
__device__ __forceinline__ void next_tile_item(const AttnArgs &a, int rows_per, TileItem &it) {
    if (++it.head < a.n_kv) return;
    it.head = 0;
    ++it.row_tile;
    if (it.row_tile * rows_per >= it.rows) {
        it.row_tile = 0;
        do {
            if (++it.seq >= a.n_seq) {  // not with lengths that stand still: an item without rows and keys
                it.seq = a.n_seq;
                it.rows = 0;
                it.s = AttnSeq{0, 1, 0};  // (a token that sees none: with t = 0 it came out as one that sees a key)
                break;
            }
            it.s = attn_seq(a, __ldcg(a.cu_q + it.seq), __ldcg(a.cu_q + it.seq + 1), __ldcg(a.kv_len + it.seq));
            it.rows = it.s.t * a.group;
        } while (it.rows == 0 || !tile_served(a, it.rows));
    }
    tile_sizes(a, rows_per, it);
}

// The items of a run, as each warp walks them.
struct TileRun {
    const AttnArgs &a;
    int rows_per;
    long long hi;
    TileItem it;
    int off, end, t1, n;  // first tile, where the run's part ends, where what is seen ends, tiles to do
    long long pos;        // of the item's first unit
    bool live;
    __device__ __forceinline__ TileRun(const AttnArgs &args, int rows, long long run_hi)
        : a(args), rows_per(rows), hi(run_hi), live(false) {}
    __device__ __forceinline__ void start(const TileItem &first, int first_off, long long first_pos) {
        it = first;
        off = first_off;
        pos = first_pos;
        sizes();
    }
    __device__ __forceinline__ void sizes() {
        live = pos + kTileStart + off < hi;
        end = static_cast<int>(min(static_cast<long long>(it.tiles), hi - pos - kTileStart));
        t1 = min(end, (it.vis + kTileKeys - 1) / kTileKeys);
        n = max(0, t1 - off);
    }
    __device__ __forceinline__ bool more() const { return live; }
    __device__ __forceinline__ bool whole() const { return off == 0 && end == it.tiles; }
    __device__ __forceinline__ void next() {
        pos += it.tiles + kTileStart;
        off = 0;
        live = pos + kTileStart < hi;
        if (!live) return;
        next_tile_item(a, rows_per, it);
        sizes();
    }
};

// D[tmem] (+)= A[tmem] B[smem], K = 16; issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
// Instruction descriptor of kind::f16 with f16 operands and f32 sums, A K-major.
__host__ __device__ constexpr uint32_t f16_idesc(int n, bool b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// The values' operand: a row is one key and runs along d, in swizzled rows of 64 elements, the next 64 `next` bytes on.
__device__ __forceinline__ uint64_t values_desc(uint32_t addr, int next) {
    return (smem_desc(addr, 128) & ~(uint64_t{0x3fff} << 16)) | (static_cast<uint64_t>(next >> 4) << 16);
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
    return max3(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c));
}

// Eight columns of a warp's lanes times a number of each lane's.
__device__ __forceinline__ void tmem_scale8(uint32_t addr, float by) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        asm volatile("" : "+r"(r[i]));
        r[i] = __float_as_uint(__uint_as_float(r[i]) * by);
    }
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Waits for a barrier phase; after one wait expired, none is made any more, and the fault word says so.
struct AttnWaiter {
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        if (dead || __all_sync(kFullMask, mbar_test(bar, parity))) return;
        if (!warp_wait_bounded(bar, parity)) {
            dead = true;
            if ((threadIdx.x & 31) == 0) atomicOr(&g_attn_fault, kAttnFaultWait);
        }
    }
};

// The same for a single thread.
struct AttnThreadWaiter {
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        if (dead || mbar_test(bar, parity)) return;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (clock64() - t0 > kWaitCycles) {
                dead = true;
                atomicOr(&g_attn_fault, kAttnFaultWait);
                return;
            }
        }
    }
};

// Offset of the 16-byte piece `p` of row `r` in swizzled rows of 128 bytes.
__device__ __forceinline__ int piece_at(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }

// A row of a block -> its f16 terms in shared memory and its scores' factor.  16 lanes serve a row, 8 (4)
// elements each.
template <int D, bool Q2>
__device__ __forceinline__ void stage_queries(const AttnArgs &a, const TileItem &it, uint8_t *q, float *factors, int block,
                                              int warp, int lane) {
    constexpr int E = D / 16, kBatch = Q2 ? 4 : 8;  // rows whose loads are out at once
    using Load = typename std::conditional<Q2, float4[E / 4], typename std::conditional<E == 8, uint4[1], uint2[1]>::type>::type;
    const int part = lane & 15;
    const float sign = a.scale_log2 < 0.f ? -1.f : 1.f;
    // (token, head) of this lane's first row; the next is two rows on
    const int first = warp * 32 + (lane >> 4);
    int tok = (it.row0 + block * 128 + first) / a.group, head = it.row0 + block * 128 + first - tok * a.group;
    const int tok_step = 2 / a.group, head_step = 2 - tok_step * a.group;
#pragma unroll 1
    for (int i0 = 0; i0 < 16; i0 += kBatch) {
        Load raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const bool live = block * 128 + first + (i0 + i) * 2 < it.n_rows;
            const int64_t from = (static_cast<int64_t>(it.s.start) + tok) * a.q_stride + (it.head * a.group + head) * D + part * E;
            if constexpr (Q2) {
#pragma unroll
                for (int j = 0; j < E / 4; ++j) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (live) v = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + from) + j);
                    raw[i][j] = v;
                }
            } else if constexpr (E == 8) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (live) v = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + from));
                raw[i][0] = v;
            } else {
                uint2 v = make_uint2(0, 0);
                if (live) v = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + from));
                raw[i][0] = v;
            }
            tok += tok_step;
            head += head_step;
            if (head >= a.group) {
                head -= a.group;
                ++tok;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = first + (i0 + i) * 2;
            float x[E];
            const uint32_t *words = reinterpret_cast<const uint32_t *>(&raw[i]);
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                if constexpr (Q2) {
                    x[2 * j] = __uint_as_float(words[2 * j]);
                    x[2 * j + 1] = __uint_as_float(words[2 * j + 1]);
                } else {
                    x[2 * j] = __uint_as_float(words[j] << 16);
                    x[2 * j + 1] = __uint_as_float(words[j] & 0xffff0000u);
                }
            }
            uint32_t top = 0;  // as bits, infinities and NaN lie above all numbers
#pragma unroll
            for (int j = 0; j < E; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));
            const int e = max(static_cast<int>(top >> 23), 32);
            const float inv = sign * __uint_as_float(static_cast<uint32_t>(min(254, 268 - e)) << 23);
            const float back = __uint_as_float(static_cast<uint32_t>(max(1, e - 14)) << 23);
            if (part == 0) factors[block * 128 + r] = top < 0x7f800000u ? back * fabsf(a.scale_log2) : NAN;
            uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float u = x[2 * j] * inv, v = x[2 * j + 1] * inv;
                hi[j] = f32x2_to_f16x2(u, v);
                if (Q2) lo[j] = attn_rest(u, v, hi[j]);
            }
            uint8_t *base = q + (Q2 ? 0 : block) * (128 * D * 2);
            const int byte = part * E * 2, half = byte >> 7, p = (byte & 127) >> 4;
            uint8_t *at = base + half * 16384 + piece_at(r, p) + (byte & 15);
            if (E == 8) {
                *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[E / 2 - 2], hi[E / 2 - 1]);
                if (Q2)
                    *reinterpret_cast<uint4 *>(at + 128 * D * 2) = make_uint4(lo[0], lo[1], lo[E / 2 - 2], lo[E / 2 - 1]);
            } else {
                *reinterpret_cast<uint2 *>(at) = make_uint2(hi[0], hi[1]);
                if (Q2) *reinterpret_cast<uint2 *>(at + 128 * D * 2) = make_uint2(lo[0], lo[1]);
            }
        }
    }
}

template <int D, bool Q2, bool P2>
__global__ void __launch_bounds__(kTileThreads, 1) attn_tiles_kernel(const AttnArgs a) {
    using Shape = TileShape<D, Q2, P2>;
    constexpr int kBlocks = Shape::kBlocks, kRowsPer = Shape::kRows;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFullMask, tid >> 5, 0);
    uint8_t *q_smem = smem, *k_smem = smem + Shape::kQ, *v_smem = k_smem + 2 * Shape::kKv;
    TileControl *ctl = reinterpret_cast<TileControl *>(v_smem + 2 * Shape::kKv);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->k_full[i], 4);
            mbar_init(&ctl->k_free[i], 1);
            mbar_init(&ctl->v_full[i], 3);
            mbar_init(&ctl->v_free[i], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&ctl->scores[i][h], 1);
                mbar_init(&ctl->weights[i][h], 4);
            }
        }
        mbar_init(&ctl->q_ready, kBlocks * 4);
        mbar_init(&ctl->drain, 1);
        mbar_init_fence();
        ctl->first = TileItem{};  // no item, should the lengths change before a thread finds the first
        ctl->first_off = 0;
        ctl->first_pos = 1ll << 62;
    }
    if (warp == kIssueWarp) tmem_alloc(&ctl->tmem, 512);
    griddep_wait();
    griddep_launch_dependents();  // behind the wait: the row kernel may start on what this one may

    // ------------------------------------------------------------------ this CTA's run of tiles
    // Blocks of rows before each sequence; then a thread counts the tiles of a slice of the blocks.
    int4 *seqs = reinterpret_cast<int4 *>(smem);  // (start, t, kv, blocks before), of at most 2^27 blocks
    const auto prefix = [&](long long v, long long &total) {  // exclusive, over the CTA
        long long incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(kFullMask, incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();
        if (lane == 31) ctl->warp_sum[warp] = incl;
        __syncthreads();
        const long long s = lane < kTileThreads / 32 ? ctl->warp_sum[lane] : 0;
        long long run = s;
#pragma unroll
        for (int o = 1; o < kTileThreads / 32; o <<= 1) {
            const long long up = __shfl_up_sync(kFullMask, run, o);
            if (lane >= o) run += up;
        }
        total = __shfl_sync(kFullMask, run, kTileThreads / 32 - 1);
        return __shfl_sync(kFullMask, run - s, warp) + incl - v;
    };
    const int per_seq = (a.n_seq + kTileThreads - 1) / kTileThreads;
    bool descends = false;
    long long blocks = 0, total_blocks = 0, total = 0;
    for (int i = 0; i < per_seq; ++i) {
        const int b = tid * per_seq + i;
        if (b >= a.n_seq) break;
        const int c0 = __ldcg(a.cu_q + b), c1 = __ldcg(a.cu_q + b + 1), kv = __ldcg(a.kv_len + b);
        if (c0 < 0 || c0 > c1 || c1 > a.n_tok || kv < 0 || kv > (static_cast<long long>(a.max_pages) << a.page_shift))
            atomicOr(&g_attn_fault, kAttnFaultInput);
        descends = descends || c0 > c1;
        const AttnSeq s = attn_seq(a, c0, c1, kv);
        const int rows = s.t * a.group;
        seqs[b] = make_int4(s.start, s.t, s.kv, static_cast<int>(blocks));
        if (tile_served(a, rows)) blocks += (rows + kRowsPer - 1) / kRowsPer;
    }
    const bool nothing = __syncthreads_or(descends);
    long long before = prefix(blocks, total_blocks);
    for (int i = 0; i < per_seq; ++i) {
        const int b = tid * per_seq + i;
        if (b < a.n_seq) seqs[b].w += static_cast<int>(before);
    }
    if (nothing) total_blocks = 0;
    __syncthreads();
    const long long slice = (total_blocks + kTileThreads - 1) / kTileThreads;
    const int lo_block = static_cast<int>(min(total_blocks, tid * slice)),
              hi_block = static_cast<int>(min(total_blocks, lo_block + slice));
    long long own = 0, per = 0, run_lo = 0, run_hi = 0;
    before = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1 && (run_lo < before || run_lo >= before + own)) break;
        long long sum = before;
        TileItem it{};
        if (lo_block < hi_block) {
            int lo = 0, hi = a.n_seq;  // the last sequence whose first block is at or before lo_block
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (seqs[mid].w <= lo_block) lo = mid; else hi = mid;
            }
            const int4 v = seqs[lo];
            it.seq = lo;
            it.s = AttnSeq{v.x, v.y, v.z};
            it.rows = it.s.t * a.group;
            it.row_tile = lo_block - v.w;
            tile_sizes(a, kRowsPer, it);
        }
        for (int b = lo_block; b < hi_block; ++b) {
            const int units = it.tiles + kTileStart;
            const long long n = static_cast<long long>(units) * a.n_kv;
            if (pass == 1 && sum <= run_lo && run_lo < sum + n) {
                const long long at = run_lo - sum;
                it.head = static_cast<int>(at / units);
                const int in_item = static_cast<int>(at - static_cast<long long>(it.head) * units);
                ctl->first = it;
                ctl->first_off = max(0, in_item - kTileStart);
                ctl->first_pos = run_lo - in_item;  // of the item's first unit
            }
            sum += n;
            if (b + 1 < hi_block) {
                it.head = a.n_kv - 1;
                next_tile_item(a, kRowsPer, it);
            }
        }
        if (pass == 0) {
            own = sum;
            before = prefix(own, total);
            per = max(static_cast<long long>(kTileStart + 1), (total + gridDim.x - 1) / gridDim.x);
            run_lo = blockIdx.x * per;
            run_hi = min(total, run_lo + per);
        }
    }
    if (tid == 0) a.owner[blockIdx.x].rows = 0;
    fence_async_smem();  // the lengths lie where codes will
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, ctl->tmem, 0);
    // columns of a block's scores and outputs
    const auto s_col = [&](int b) { return tmem + static_cast<uint32_t>(b) * 128; };
    const auto o_col = [&](int b) { return tmem + 256 + static_cast<uint32_t>(b) * 128; };

    AttnWaiter wait;
    const auto my_run = [&]() {
        TileRun run{a, kRowsPer, run_hi};
        if (run_lo < run_hi) run.start(ctl->first, ctl->first_off, ctl->first_pos);
        return run;
    };
    if (warp < 8)  // whole warpgroups, one instruction each
        set_registers_up<kRegsWeights>();
    else
        set_registers_down<kRegsOthers>();
    if (warp < 8) {
        // ------------------------------------------------------------ weights and the way out
        TileRun run = my_run();
        const int b = warp >> 2, wq = warp & 3, r = b * 128 + wq * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t at_s = s_col(b) + lanes, at_o = o_col(b) + lanes, at_odd = o_col(1) + lanes, at_rest = s_col(1) + lanes;
        uint32_t tile = 0, turns = 0, all_items = 0;
        for (; b < kBlocks && run.more() && !wait.dead; run.next()) {
            const TileItem &it = run.it;
            const int n = run.n;
            const bool mine = b == 0 || it.n_rows > 128;
            float ref = kAttnUnset, total_w = 0.f;
            if (n > 0) {
                if (mine) stage_queries<D, Q2>(a, it, q_smem, ctl->factor, b, wq, lane);
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->q_ready);
                if (!mine) wait(&ctl->q_ready, all_items & 1);  // never two arrivals in one phase
                ++all_items;
            }
            if (mine && n > 0) {
                const int see0 = it.s.kv - it.s.t + 1;
                const int lim = min(it.vis, max(0, see0 + (it.row0 + r) / a.group));
                const float factor = lim > 0 ? ctl->factor[r] : 1.f;  // of no keys there is no NaN, whatever the query is
                const int all_see = max(0, see0 + (it.row0 + b * 128) / a.group);
                // Half a tile a time: a half's scores have their own columns, so that the products of the next half
                // run meanwhile.
                for (int u = 0; u < 2 * n; ++u) {
                    const int half = u & 1, key0 = (run.off + (u >> 1)) * kTileKeys + half * kHalfKeys;
                    const float4 *scale = ctl->scale[(tile + (u >> 1)) & 3] + half * 4;
                    const uint32_t at = at_s + half * kHalfKeys;
                    wait(&ctl->scores[b][half], (turns + (u >> 1)) & 1);
                    if (wait.dead) break;
                    tc_fence_after();
                    const bool masked = key0 + kHalfKeys > all_see;
                    uint32_t raw[2][32];
                    tmem_ld32_nowait(at, raw[0]);
                    tmem_ld32_nowait(at + 32, raw[1]);
                    tc_wait_ld();
                    tmem_ld32_done(raw[0]);
                    tmem_ld32_done(raw[1]);
                    if (masked) {  // -infinity is a weight of 0 under any factor but 0, which there is none of
                        const int left = lim - key0;  // keys of the half that the row sees
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i >= left) raw[c][i] = 0xff800000u;
                    }
                    float f[4], top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[i] = factor * scale[i].x;
                        if (f[i] == 0.f) f[i] = 0x1p-120f;
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t(&x)[32] = raw[c];
                            const int k = 16 * h;
                            const float m0 = max3(max3(x[k], x[k + 1], x[k + 2]), max3(x[k + 3], x[k + 4], x[k + 5]),
                                                  max3(x[k + 6], x[k + 7], x[k + 8]));
                            const float m1 = max3(max3(x[k + 9], x[k + 10], x[k + 11]), max3(x[k + 12], x[k + 13], x[k + 14]),
                                                  __uint_as_float(x[k + 15]));
                            top = fmaxf(top, fmaf(fmaxf(m0, m1), f[2 * c + h], scale[2 * c + h].w));
                        }
                    if (__any_sync(kFullMask, top > ref + kAttnSlack)) {
                        const float to = fmaxf(ref, top), by = ex2(ref - to);
                        ref = to;
                        total_w *= by;
                        if (u > 0) {  // behind the last half's products: the scores after these come behind them
                            wait(&ctl->scores[b][half ^ 1], (turns + ((u + 1) >> 1)) & 1);
                            if (wait.dead) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) tmem_scale8(at_o + c * 8, by);
                            if (P2) {
#pragma unroll 1
                                for (int c = 0; c < D / 8; ++c) {
                                    tmem_scale8(at_rest + c * 8, by);
                                    if (u >= 3) tmem_scale8(at_odd + c * 8, by);  // (its first products are of the third half)
                                }
                            }
                        }
                    }
                    float sums[4];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t w[16], rest[P2 ? 16 : 1];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 sc = scale[2 * c + h];
                            const float shift = sc.y - ref + kAttnTop;
                            const uint64_t f2 = pack2(f[2 * c + h], f[2 * c + h]), shift2 = pack2(shift, shift);
                            uint64_t sum[2] = {0, 0};
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int k = h * 16 + 2 * i;
                                const float2 x = unpack2(fma2(bits2(raw[c][k], raw[c][k + 1]), f2, shift2));
                                const float p0 = ex2(x.x), p1 = ex2(x.y);
                                sum[i & 1] = add2(sum[i & 1], pack2(p0, p1));
                                w[h * 8 + i] = f32x2_to_f16x2(p0, p1);
                                if (P2) rest[P2 ? h * 8 + i : 0] = attn_rest(p0, p1, w[h * 8 + i]);
                            }
                            const float2 t = unpack2(add2(sum[0], sum[1]));
                            sums[2 * c + h] = (t.x + t.y) * sc.z;
                        }
                        tmem_st16(at + c * 16, w);
                        if (P2) tmem_st16(at + 32 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(rest));
                    }
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->weights[b][half]);
                    total_w += (sums[0] + sums[1]) + (sums[2] + sums[3]);
                }
                // the last products: the turns behind the last scores
                wait(&ctl->scores[b][0], (turns + n) & 1);
                wait(&ctl->scores[b][1], (turns + n) & 1);
                turns += n + 1;
                tc_fence_after();
            }
            tile += n;
            if (mine && !wait.dead) {
                const bool whole = run.whole();
                const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (run.off == 0 ? 1 : 0);
                const bool live = r < it.n_rows;
                const int64_t to = whole ? attn_out_at(a, it.s.start, it.head, it.row0 + (live ? r : 0), D)
                                         : (piece * kRowsPer + r) * D;
                const float norm = !whole ? 1.f : total_w == 0.f ? 0.f : __fdiv_rn(1.f, total_w);
                if (!whole && live) a.stats[piece * kRowsPer + r] = make_float2(ref, total_w);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    if (n > 0) {
                        tmem_ld32(at_o + c * 32, o);
                        if (P2) {
                            float more[32];
                            tmem_ld32(at_rest + c * 32, more);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] += more[i];
                            if (n > 1) {
                                tmem_ld32(at_odd + c * 32, more);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] += more[i];
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0.f;
                    }
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= norm;
                    if (whole && a.out_bf16) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to + c * 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            __nv_bfloat162 v[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) v[m] = __floats2bfloat162_rn(o[8 * i + 2 * m], o[8 * i + 2 * m + 1]);
                            dst[i] = *reinterpret_cast<uint4 *>(v);
                        }
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>((whole ? static_cast<float *>(a.out) : a.part) + to + c * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (!whole && run.off == 0 && warp == 0 && lane == 0) {
                    AttnOwner owner;
                    owner.start = it.s.start;
                    owner.row0 = it.row0;
                    owner.first = blockIdx.x;
                    owner.last = static_cast<int>((run.pos + it.tiles + kTileStart - 1) / per);
                    owner.head = it.head;
                    owner.rows = it.n_rows;
                    a.owner[blockIdx.x] = owner;
                }
            }
        }
    } else if (warp != kIssueWarp) {
        // ------------------------------------------------------------ codes -> f16
        // The lower four warps widen keys, three of the upper values.  16 codes are a thread's load.
        constexpr int kChunks = D / 16;
        TileRun run = my_run();
        const bool keys = warp < kIssueWarp;
        const int ct = keys ? tid - kWidenWarp * 32 : tid - (kIssueWarp + 1) * 32;
        const int chunk = ct % kChunks, r0 = ct / kChunks, step = (keys ? 128 : 96) / kChunks;
        constexpr int kLoads = (kTileKeys * kChunks + 95) / 96;
        const uint8_t *cache = keys ? a.k_cache : a.v_cache;
        uint8_t *to_smem = keys ? k_smem : v_smem;
        uint64_t *full = keys ? ctl->k_full : ctl->v_full, *freed = keys ? ctl->k_free : ctl->v_free;
        const bool scaling = warp == kWidenWarp && lane < 8;
        uint32_t tile = 0;
        for (; run.more() && !wait.dead; run.next()) {
            const TileItem &it = run.it;
            if (run.n == 0) continue;
            const int32_t *table = a.table + static_cast<int64_t>(it.seq) * a.max_pages;
            // Lane l (of 8) serves the tile's block l: its page, three tiles ahead of the codes' use; its first row in
            // the pool, two; its scales, one.
            const auto page_at = [&](int j) {  // not checked yet
                const int key = j * kTileKeys + (lane & 7) * kAttnBlock;
                return j < run.t1 && key < it.vis ? __ldcg(table + (key >> a.page_shift)) : -1;
            };
            const auto base_at = [&](int page, int j) -> int {
                const int key = j * kTileKeys + (lane & 7) * kAttnBlock;
                return j < run.t1 && key < it.vis ? attn_row(a, page, it.head, key) : -1;
            };
            const auto scale_at = [&](const float *scales, int base) {
                return scaling && base >= 0 ? __ldcg(scales + (base >> 4)) : 1.f;
            };
            const auto load = [&](uint4(&to)[kLoads], int base, int j) {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int r = r0 + i * step;
                    const int from = __shfl_sync(kFullMask, base, (r >> 4) & 7);
                    to[i] = r < kTileKeys && from >= 0 && j * kTileKeys + r < it.vis
                                ? __ldcg(reinterpret_cast<const uint4 *>(cache + (static_cast<int64_t>(from) + (r & 15)) * D) + chunk)
                                : make_uint4(0, 0, 0, 0);
                }
            };
            int base_next = base_at(page_at(run.off), run.off);
            float ks = scale_at(a.k_scales, base_next), vs = scale_at(a.v_scales, base_next);
            uint4 code[kLoads];
            load(code, base_next, run.off);
            base_next = base_at(page_at(run.off + 1), run.off + 1);
            int page_later = page_at(run.off + 2);
            for (int j = run.off; j < run.t1; ++j, ++tile) {
                const uint32_t buf = tile & 1;
                const float ks_next = scale_at(a.k_scales, base_next), vs_next = scale_at(a.v_scales, base_next);
                if (tile >= 2) wait(&freed[buf], ((tile >> 1) - 1) & 1);
                if (wait.dead) break;
                if (scaling) {
                    const float v = vs < kAttnLeastScale ? kAttnLeastScale : vs, l = attn_log2(v);
                    ctl->scale[tile & 3][lane] = make_float4(ks, l, __frcp_rn(v), fmaxf(l, kAttnLeastLog));
                }
                // 16 codes fill two pieces of a swizzled row; half of the lanes store them in the other order, off the
                // banks of the others
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int r = r0 + i * step;
                    uint8_t *half = to_smem + buf * Shape::kKv + (chunk >> 2) * 16384;
                    uint4 x, y;
                    e4m3x4_to_f16x2x2(code[i].x, x.x, x.y);
                    e4m3x4_to_f16x2x2(code[i].y, x.z, x.w);
                    e4m3x4_to_f16x2x2(code[i].z, y.x, y.y);
                    e4m3x4_to_f16x2x2(code[i].w, y.z, y.w);
                    const int p = (chunk & 3) * 2, swap = kChunks == 8 ? chunk >> 2 : r & 1;
                    if (r < kTileKeys) {
                        *reinterpret_cast<uint4 *>(half + piece_at(r, p + swap)) = swap ? y : x;
                        *reinterpret_cast<uint4 *>(half + piece_at(r, p + 1 - swap)) = swap ? x : y;
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[buf]);
                load(code, base_next, j + 1);
                base_next = base_at(page_later, j + 2);
                page_later = page_at(j + 3);
                ks = ks_next;
                vs = vs_next;
            }
        }
    } else {
        // ------------------------------------------------------------ products
        constexpr uint32_t kQk = f16_idesc(kHalfKeys, false), kPv = f16_idesc(D, true);
        const uint32_t q_at = smem_u32(q_smem), k_at = smem_u32(k_smem), v_at = smem_u32(v_smem);
        const auto scores = [&](int b, int half, uint32_t buf) {
#pragma unroll
            for (int term = Q2 ? 1 : 0; term >= 0; --term)  // the remainders first, while the sums are small
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t at = (i >> 2) * 16384 + (i & 3) * 32;
                    mma_f16_ss(s_col(b) + half * kHalfKeys, smem_desc(q_at + (Q2 ? term : b) * (128 * D * 2) + at, 128),
                               smem_desc(k_at + buf * Shape::kKv + half * (kHalfKeys * 128) + at, 128), kQk,
                               (Q2 && term == 0) || i > 0);
                }
        };
        const auto outputs = [&](int b, int u, uint32_t buf) {
            const int half = u & 1;
            const uint32_t to = P2 ? o_col((u >> 1) & 1) : o_col(b);
            const bool acc = P2 ? u >= 4 || half : u > 0;
#pragma unroll
            for (int i = 0; i < kHalfKeys / 16; ++i) {
                const uint64_t v = values_desc(v_at + buf * Shape::kKv + half * (kHalfKeys * 128) + i * 2048, 16384);
                const uint32_t p = s_col(b) + half * kHalfKeys + i * 8;
                mma_f16_ts(to, p, v, kPv, acc || i > 0);
                if (P2) mma_f16_ts(s_col(1), p + 32, v, kPv, u > 0 || i > 0);
            }
        };
        if (elect_one()) {
            // One thread from here on, whose waits need no votes (a whole warp that elects one for each product took 1093 us
            // where this took 949, 2048 tokens over 16384 rows).
            AttnThreadWaiter ready;
            TileRun run = my_run();
            uint32_t tile = 0, turns[2] = {0, 0}, all_items = 0;
            for (; run.more() && !ready.dead; run.next()) {
                const int n = run.n, live_blocks = run.it.n_rows > 128 ? 2 : 1;
                if (n == 0) continue;
                ready(&ctl->q_ready, all_items & 1);
                ++all_items;
                ready(&ctl->k_full[tile & 1], (tile >> 1) & 1);
                if (ready.dead) break;
                tc_fence_after();
                for (int half = 0; half < 2; ++half)
                    for (int b = 0; b < live_blocks; ++b) {
                        scores(b, half, tile & 1);
                        tc_commit(&ctl->scores[b][half]);
                    }
                tc_commit(&ctl->k_free[tile & 1]);
                for (int u = 0; u < 2 * n && !ready.dead; ++u) {
                    const int half = u & 1, j = u >> 1;
                    const uint32_t buf = (tile + j) & 1, next = tile + j + 1;
                    const bool more = j + 1 < n;
                    if (half == 0) {
                        ready(&ctl->v_full[buf], ((tile + j) >> 1) & 1);
                        if (more) ready(&ctl->k_full[next & 1], (next >> 1) & 1);
                    }
                    for (int b = 0; b < live_blocks; ++b) {
                        ready(&ctl->weights[b][half], (turns[b] + j) & 1);
                        if (ready.dead) break;
                        tc_fence_after();
                        outputs(b, u, buf);
                        if (more) scores(b, half, next & 1);
                        tc_commit(&ctl->scores[b][half]);  // behind the last scores: of the products alone
                    }
                    if (half == 1 && !ready.dead) {
                        tc_commit(&ctl->v_free[buf]);
                        if (more) tc_commit(&ctl->k_free[next & 1]);
                    }
                }
                tile += n;
                for (int b = 0; b < live_blocks; ++b) turns[b] += n;
            }
            if (ready.dead) {  // products in flight end before TMEM is given up, the wait bounded
                tc_commit(&ctl->drain);
                ready.dead = false;
                ready(&ctl->drain, 0);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace memq
