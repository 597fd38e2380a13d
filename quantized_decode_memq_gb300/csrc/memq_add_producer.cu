// memq_add_producer.cu -- memq_add_rmsnorm_q8_1: the residual stream's addition in front of the
// RMSNorm -> q8_1 producer, in one launch.
//
//   h = x + res;   z = (h * rr) * w;   d = max |z| / 127 and qs = round(z / d) per 32 elements
//
// It reads x, res and writes h, qs, d: 13.1 bytes an element instead of the 17.1 of an addition
// followed by memq_rmsnorm_q8_1 (12 + 5.1), and is bound by memory on many rows (4096 x 8192: 83.6 us,
// 5.3 TB/s, 77% of a copy's rate) and by latency on few (1 x 5120: 3.2 us a launch, back to back).
//
// z, qs and d are bit for bit what memq_rmsnorm_q8_1 gives for h.  The only order that matters is that
// of the sum of squares: a thread of that kernel adds the float4 slices tid, tid + threads, ... of the
// row in f32, then f64 sums run over the lanes and the warps.  Here up to four threads share what one
// does there: all load, add and quantise S slices each, so that few loads and few roundings follow one
// another (latency is what a single row costs), and one of the four sums their slices up, in order,
// from shared memory.
//
// On few or wide rows a cluster shares a row: the row's warps are dealt out to up to eight CTAs, which exchange
// the warps' sums through distributed shared memory.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "memq.h"
#include "memq_dev.cuh"

namespace memq {
namespace {

constexpr int kMaxCluster = 8;

__device__ __forceinline__ void store_dsmem(double *p, int cta, double v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(cta));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(v) : "memory");
}
// A CTA's shared memory may be written from outside only once it runs, which co-scheduling alone does
// not say: every CTA of the cluster arrives at its entry, and waits for the others ahead of its first
// remote store.  No data passes here, so the arrival orders nothing.
__device__ __forceinline__ void cluster_started_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// round(z / dd), ties away from zero, with a multiplication for most divisions: inv is the correctly
// rounded 1 / dd and |z / dd| <= 127, so z * inv is within 2.3e-5 of the correctly rounded quotient,
// and both round to the same integer unless z * inv lies that near to a half; there, and where 1 / dd
// leaves the normal range, the quotient itself is taken.
__device__ __forceinline__ uint32_t code_of(float z, float dd, float inv) {
    const float t = __fmul_rn(z, inv);
    float r = rintf(t);
    if (!(fabsf(t - r) < 0.5f - 3.0e-5f) || !(dd > 7.9e-31f))
        r = dd != 0.0f ? roundf(__fdiv_rn(z, dd)) : 0.0f;
    return static_cast<uint32_t>(static_cast<uint8_t>(static_cast<int8_t>(r)));
}

// CTA `part` of a row's `ctas`.  `nwarps` summing warps serve the row, `per_cta` of them this CTA, whose
// threads are R times as many; thread (k, t) holds the slices of summing thread t from number k on in
// steps of R.
template <int S, int R, bool LATE>
__global__ void __launch_bounds__(R == 1 ? 256 : 1024, R == 1 ? (S <= 2 ? 8 : 4) : S <= 2 ? 2 : 1)
    add_rmsnorm_q8_1_kernel(const float *x, const float *res, float *h, const float *__restrict__ w, float *z,
                            int8_t *qs, float *d, int ncols, float eps, int nwarps, int per_cta, int ctas) {
    extern __shared__ __align__(16) float4 held[];  // [S R][summing threads of this CTA]
    __shared__ double red[32];
    __shared__ float r_shared;
    if (ctas > 1) cluster_started_arrive();
    griddep_launch_dependents();
    griddep_wait();

    const int part = ctas == 1 ? 0 : static_cast<int>(blockIdx.x) % ctas;
    const int64_t row = ctas == 1 ? blockIdx.x : blockIdx.x / ctas;
    const int lane = threadIdx.x & 31;
    const int sums = per_cta * 32, k = static_cast<int>(threadIdx.x) / sums, t = static_cast<int>(threadIdx.x) - k * sums;
    const int warp = part * per_cta + (t >> 5);  // summing warp
    const int nthr = nwarps * 32, f0 = warp * 32 + lane + k * nthr, step = R * nthr;
    const int nf4 = warp < nwarps ? ncols >> 2 : 0;  // the last CTA may have a warp too many
    const float4 *x4 = reinterpret_cast<const float4 *>(x + row * ncols);
    const float4 *r4 = reinterpret_cast<const float4 *>(res + row * ncols);
    const float4 *w4 = reinterpret_cast<const float4 *>(w);
    float4 *h4 = reinterpret_cast<float4 *>(h + row * ncols);

    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v[S], wk[S];
    {
        float4 b[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int f = f0 + i * step;
            v[i] = f < nf4 ? __ldcg(x4 + f) : zero;
            b[i] = f < nf4 ? __ldcg(r4 + f) : zero;
        }
        if (R == 1) {
#pragma unroll
            for (int i = 0; i < S; ++i) wk[i] = f0 + i * step < nf4 ? __ldg(w4 + f0 + i * step) : zero;
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            v[i] = make_float4(__fadd_rn(v[i].x, b[i].x), __fadd_rn(v[i].y, b[i].y), __fadd_rn(v[i].z, b[i].z),
                               __fadd_rn(v[i].w, b[i].w));
            if (R > 1) held[(k + i * R) * sums + t] = v[i];
            if (f0 + i * step < nf4) h4[f0 + i * step] = v[i];
        }
    }
    // Where threads share, w is loaded here: the first loads then have its registers, and it arrives while
    // one of four threads sums (us, here / with the first loads: 2048 rows of 17408 107 / 129, 4096 of 8192
    // 85.2 / 87.3; without sharing, 1000 of 4096 14.2 / 13.4).  LATE: after the sum.
    if (R > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (!LATE) wk[i] = f0 + i * step < nf4 ? __ldg(w4 + f0 + i * step) : zero;
    }
    if (ctas > 1) cluster_started_wait();  // long over by the time that the row's loads are back
    if (k == 0) {
        float ss = 0.0f;  // a slice past the row's end adds zeros
#pragma unroll
        for (int i = 0; i < S * R; ++i) {
            const float4 q = R > 1 ? held[i * sums + t] : v[i];
            ss = fmaf(q.x, q.x, ss);
            ss = fmaf(q.y, q.y, ss);
            ss = fmaf(q.z, q.z, ss);
            ss = fmaf(q.w, q.w, ss);
        }
        const double total = warp_sum(static_cast<double>(ss));
        if (ctas > 1) {
            if (lane < ctas && warp < nwarps) store_dsmem(&red[warp], lane, total);
        } else if (lane == 0) {
            red[warp] = total;
        }
    }
    if (ctas > 1)
        cluster_sync();  // nobody reaches into another CTA past this point
    else
        __syncthreads();
    if (threadIdx.x < 32) {
        const double total = warp_sum(lane < nwarps ? red[lane] : 0.0);
        if (lane == 0)
            r_shared = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(
                __fdiv_rn(static_cast<float>(total), static_cast<float>(ncols)), eps)));
    }
    __syncthreads();
    const float r = r_shared;

    float4 *z4 = z ? reinterpret_cast<float4 *>(z + row * ncols) : nullptr;
    uint32_t *q4 = reinterpret_cast<uint32_t *>(qs + row * ncols);
    float *drow = d + row * (ncols >> 5);
    // A 32-element block is eight adjacent lanes, wholly inside the row or outside it.
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int f = f0 + i * step;
        if (LATE) wk[i] = f < nf4 ? __ldg(w4 + f) : zero;
        const float4 zz = make_float4(__fmul_rn(__fmul_rn(v[i].x, r), wk[i].x), __fmul_rn(__fmul_rn(v[i].y, r), wk[i].y),
                                      __fmul_rn(__fmul_rn(v[i].z, r), wk[i].z), __fmul_rn(__fmul_rn(v[i].w, r), wk[i].w));
        float am = fmaxf(fmaxf(fabsf(zz.x), fabsf(zz.y)), fmaxf(fabsf(zz.z), fabsf(zz.w)));
        am = fmaxf(am, __shfl_xor_sync(kFullMask, am, 1));
        am = fmaxf(am, __shfl_xor_sync(kFullMask, am, 2));
        am = fmaxf(am, __shfl_xor_sync(kFullMask, am, 4));
        const float dd = __fdiv_rn(am, 127.0f), inv = __frcp_rn(dd);
        if (f < nf4) {
            q4[f] = code_of(zz.x, dd, inv) | code_of(zz.y, dd, inv) << 8 | code_of(zz.z, dd, inv) << 16 |
                    code_of(zz.w, dd, inv) << 24;
            if (z4) z4[f] = zz;
            if ((lane & 7) == 0) drow[f >> 3] = dd;
        }
    }
}

template <int S, int R, bool LATE = false>
cudaError_t launch(const float *x, const float *res, const float *w, float *h, float *z, int8_t *qs, float *d, int ncols,
                   int rows, float eps, int nwarps, int per_cta, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(per_cta) * 32 * R);
    cfg.dynamicSmemBytes = R > 1 ? static_cast<size_t>(per_cta) * 32 * S * R * sizeof(float4) : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, add_rmsnorm_q8_1_kernel<S, R, LATE>, x, res, h, w, z, qs, d, ncols, eps, nwarps, per_cta,
                              ctas);
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

constexpr int kMaxDevices = 64;

// SM count of the current device (queried once a device).
int sm_count() {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev < kMaxDevices && (sms = cache[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    if (dev < kMaxDevices) cache[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

}  // namespace
}  // namespace memq

extern "C" int memq_add_rmsnorm_q8_1(const float *x, const float *res, const float *w, float *h, float *z, int8_t *qs,
                                     float *d, int64_t ncols, int64_t rows, float eps, void *stream) {
    using namespace memq;
    if (ncols < 32 || ncols > MEMQ_MAX_NCOLS || (ncols % 32) != 0) return MEMQ_ERR_SHAPE;
    if (rows < 0 || rows > 0x7fffffffLL) return MEMQ_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MEMQ_ERR_SHAPE;
    if (rows == 0) return MEMQ_OK;  // empty input: nothing to read or write, pointers unused
    if (!x || !res || !w || !h || !qs || !d) return MEMQ_ERR_NULL;
    if (misaligned(x, 16) || misaligned(res, 16) || misaligned(w, 16) || misaligned(h, 16) ||
        (z && misaligned(z, 16)) || misaligned(qs, 4) || misaligned(d, 4))
        return MEMQ_ERR_ALIGN;
    const int sms = sm_count();
    if (sms <= 0) return MEMQ_ERR_LAUNCH;

    // The producer's threads: the fewest float4 slices each (a power of two) that take at most 256
    // threads, up to 512 once they are 16.
    const int nf4 = static_cast<int>(ncols / 4);
    int v = 1;
    while (v < 16 && (nf4 + v - 1) / v > 256) v *= 2;
    const int nwarps = ((nf4 + v - 1) / v + 31) / 32;
    // A cluster of eight shares a row that is wider than 8192 (us, 8 CTAs a row against 2: 8 rows of
    // 17408 4.3 / 5.3, 64 6.9 / 7.2, 512 31.4 / 45.5), and one wider than 4096 while there are SMs for it
    // (8 / 1: 1 row of 5120 3.2 / 3.5, 19 of 5120 3.3 / 3.6, 19 of 8192 3.8 / 4.6, where an SM has one CTA; past
    // two each the cluster loses: 40 of 8192 4.7 / 4.9, 76 5.0 / 4.6, 152 8.2 / 4.7).
    const bool split = v == 16 || (v == 8 && rows * kMaxCluster <= sms);
    const int per_cta = split ? (nwarps + kMaxCluster - 1) / kMaxCluster : nwarps;
    const int ctas = (nwarps + per_cta - 1) / per_cta;
    if (rows * ctas > 0x7fffffffLL) return MEMQ_ERR_SHAPE;
    const int nc = static_cast<int>(ncols), nr = static_cast<int>(rows);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    // Up to 4096 columns, threads share a summing thread's slices only while two CTAs an SM serve all rows:
    // more rows have the loads in flight without it (us, shared / not: 160 x 4096 4.6 / 6.0, 304 x 4096 4.7 /
    // 4.5, 305 x 4096 6.8 / 6.4, 500 x 4096 8.1 / 6.5; 250 x 2048 5.0 / 5.5, 912 x 2048 8.0 / 7.5).
    const bool few = rows <= 2 * sms;
    // Up to 8192 columns, w is loaded after the sum once many rows follow one another on an SM: other rows
    // hide its latency, and the first loads go out ahead of it (us, after the sum / before: 1000 x 7168
    // 23.6 / 23.1, 2000 x 5120 29.1 / 30.3, 8192 x 5120 95.0 / 101.7, 4096 x 8192 83.6 / 84.8).
    const bool many = rows >= 10 * sms;
    switch (v) {
        case 1: e = launch<1, 1>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st); break;
        case 2:
            e = few ? launch<1, 2>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st)
                    : launch<2, 1>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st);
            break;
        case 4:
            e = few ? launch<1, 4>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st)
                    : launch<4, 1>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st);
            break;
        case 8:
            e = many ? launch<2, 4, true>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st)
                     : launch<2, 4>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st);
            break;
        default: e = launch<4, 4>(x, res, w, h, z, qs, d, nc, nr, eps, nwarps, per_cta, ctas, st); break;
    }
    return e == cudaSuccess ? MEMQ_OK : MEMQ_ERR_LAUNCH;
}
