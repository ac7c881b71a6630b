// group.hip -- the two ends of a mixture-of-experts layer: the ragged layout
// from the router's choice (qgemm_group_plan) and the weighted sum back to
// tokens (qgemm_group_combine).
#include "kernels_common.h"
#include "qgemm_internal.h"

namespace qg {
namespace {

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of S = T * topk ids with E + 1 keys (key E: an
// id outside [0, E)). A wave takes a contiguous run of the choices, 64 at a
// time: lanes with equal keys find each other with one ballot per key bit,
// the lane's rank among them is a population count, so a run's choices are
// counted and later placed in order with no atomics. The counters of a wave
// live in LDS, [wave][E + 1]; a scan over (key, workgroup, wave) turns them
// into first positions.
//   one workgroup (S up to kPlanOneMax): count, scan, place in one launch;
//   more: a count launch leaves [workgroup][E + 1] totals in the workspace,
//   and in the second launch every workgroup adds up what it needs of them.
// Bound by latency, not by bytes (12 bytes a choice): few launches, and a
// wave's run short.
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 16;
constexpr int kPlanThreads = 64 * kPlanWaves;

// Orders a wave's own LDS accesses for the compiler (the hardware keeps them
// in order).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <class I>
__device__ __forceinline__ int plan_key(const I *__restrict__ ids, int i, int E) {
    const I v = ids[i];
    return v >= 0 && v < (I)E ? (int)v : E;
}

// Lanes of `live` whose key equals this lane's (bits: of the largest key).
__device__ __forceinline__ unsigned long long same_key(int key, unsigned long long live, int bits) {
    unsigned long long m = live;
    for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? set : ~set;
    }
    return m;
}

// Counts the run [lo, hi) of a wave into cnt[0 .. E].
template <class I>
__device__ __forceinline__ void plan_count(const I *__restrict__ ids, int lo, int hi, int E, int bits, int *cnt) {
    const int lane = threadIdx.x & 63;
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int i = i0 + lane;
        const int key = i < hi ? plan_key(ids, i, E) : E;
        const unsigned long long m = same_key(key, __ballot(i < hi), bits);
        // the lowest of the equal lanes adds them all
        if (i < hi && __ffsll((long long)m) - 1 == lane) cnt[key] += __popcll(m);
        wave_sync();
    }
}

// Places the run: pos[0 .. E] holds the next free position of every key.
template <class I>
__device__ __forceinline__ void plan_place(const I *__restrict__ ids, int lo, int hi, int E, int bits, int topk,
                                           int *pos, int32_t *__restrict__ rows, int32_t *__restrict__ slots) {
    const int lane = threadIdx.x & 63;
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int i = i0 + lane;
        const bool on = i < hi;
        const int key = on ? plan_key(ids, i, E) : E;
        const unsigned long long m = same_key(key, __ballot(on), bits);
        const int rank = __popcll(m & ((1ull << lane) - 1));
        int p = 0;
        if (on) p = pos[key] + rank;
        // every lane has read its position before the lowest equal lane moves
        // it on (one wave's LDS operations complete in order)
        wave_sync();
        if (on && __ffsll((long long)m) - 1 == lane) pos[key] += __popcll(m);
        wave_sync();
        if (on) {
            rows[p] = i / topk;
            slots[i] = key < E ? p : -1;
        }
    }
}

// Run of wave w of workgroup g: whole 64s of the S choices.
__device__ __forceinline__ void plan_run(int S, int G, int g, int w, int *lo, int *hi) {
    const int chunks = (S + 63) / 64, W = G * kPlanWaves, x = g * kPlanWaves + w;
    const int per = chunks / W, more = chunks % W;
    const int c0 = x * per + min(x, more), c1 = c0 + per + (x < more ? 1 : 0);
    *lo = min(c0 * 64, S);
    *hi = min(c1 * 64, S);
}

// The counters cnt[wave][E + 1] of this workgroup, and totals `before` of
// earlier workgroups and `all` of everything per key (LDS), become first
// positions; offsets are written by the workgroup that is told to.
__device__ __forceinline__ void plan_scan(int E, int *cnt, const int *before, int *all, int *wsum,
                                          int32_t *offsets) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // exclusive scan of all[0 .. E] over the keys: thread k takes key k (and
    // key 1024, if there is one, goes last: its start is the sum of the rest)
    const int mine = tid <= E ? all[tid] : 0;
    int inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(inc, d);
        if (lane >= d) inc += x;
    }
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    int base = 0, total = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        if (w < wave) base += wsum[w];
        total += wsum[w];
    }
    for (int key = tid; key <= E; key += kPlanThreads) {
        const int first = key == tid ? base + inc - mine : total;
        if (offsets) offsets[key] = first;
        int p = first + before[key];
        for (int w = 0; w < kPlanWaves; ++w) {
            const int n = cnt[w * (E + 1) + key];
            cnt[w * (E + 1) + key] = p;
            p += n;
        }
    }
    __syncthreads();
}

template <class I>
__global__ __launch_bounds__(kPlanThreads) void plan_one_kernel(int S, int topk, int E, int bits,
                                                                const I *__restrict__ ids,
                                                                int32_t *__restrict__ offsets,
                                                                int32_t *__restrict__ rows,
                                                                int32_t *__restrict__ slots) {
    extern __shared__ int lds[];             // cnt [waves][E + 1], before [E + 1], all [E + 1]
    __shared__ int wsum[kPlanWaves];
    int *cnt = lds, *before = lds + kPlanWaves * (E + 1), *all = before + (E + 1);
    const int wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < (kPlanWaves + 1) * (E + 1); i += kPlanThreads) lds[i] = 0;
    __syncthreads();
    int lo, hi;
    plan_run(S, 1, 0, wave, &lo, &hi);
    plan_count(ids, lo, hi, E, bits, cnt + wave * (E + 1));
    __syncthreads();
    for (int key = threadIdx.x; key <= E; key += kPlanThreads) {
        int n = 0;
        for (int w = 0; w < kPlanWaves; ++w) n += cnt[w * (E + 1) + key];
        all[key] = n;
    }
    __syncthreads();
    plan_scan(E, cnt, before, all, wsum, offsets);
    plan_place(ids, lo, hi, E, bits, topk, cnt + wave * (E + 1), rows, slots);
}

template <class I>
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(int S, int E, int bits, const I *__restrict__ ids,
                                                                  int32_t *__restrict__ totals) {
    extern __shared__ int lds[];
    const int wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kPlanWaves * (E + 1); i += kPlanThreads) lds[i] = 0;
    __syncthreads();
    int lo, hi;
    plan_run(S, gridDim.x, blockIdx.x, wave, &lo, &hi);
    plan_count(ids, lo, hi, E, bits, lds + wave * (E + 1));
    __syncthreads();
    for (int key = threadIdx.x; key <= E; key += kPlanThreads) {
        int n = 0;
        for (int w = 0; w < kPlanWaves; ++w) n += lds[w * (E + 1) + key];
        totals[(size_t)blockIdx.x * (E + 1) + key] = n;
    }
}

template <class I>
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(int S, int topk, int E, int bits,
                                                                  const I *__restrict__ ids,
                                                                  const int32_t *__restrict__ totals,
                                                                  int32_t *__restrict__ offsets,
                                                                  int32_t *__restrict__ rows,
                                                                  int32_t *__restrict__ slots) {
    extern __shared__ int lds[];
    __shared__ int wsum[kPlanWaves];
    int *cnt = lds, *before = lds + kPlanWaves * (E + 1), *all = before + (E + 1);
    const int wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < (kPlanWaves + 2) * (E + 1); i += kPlanThreads) lds[i] = 0;
    __syncthreads();
    // the totals of every workgroup, read in a row and added up per key
    // (whole numbers: the order does not matter)
    const int n = (int)gridDim.x * (E + 1), mine = (int)blockIdx.x * (E + 1);
    const int step = kPlanThreads % (E + 1);
    int key = threadIdx.x % (E + 1);
    for (int i = threadIdx.x; i < n; i += 8 * kPlanThreads) {
        int t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = i + u * kPlanThreads < n ? totals[i + u * kPlanThreads] : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (t[u]) {
                atomicAdd(all + key, t[u]);
                if (i + u * kPlanThreads < mine) atomicAdd(before + key, t[u]);
            }
            key += step;
            if (key > E) key -= E + 1;
        }
    }
    int lo, hi;
    plan_run(S, gridDim.x, blockIdx.x, wave, &lo, &hi);
    plan_count(ids, lo, hi, E, bits, cnt + wave * (E + 1));
    __syncthreads();
    plan_scan(E, cnt, before, all, wsum, blockIdx.x == 0 ? offsets : nullptr);
    plan_place(ids, lo, hi, E, bits, topk, cnt + wave * (E + 1), rows, slots);
}

template <class I>
hipError_t plan(int S, int topk, int E, const I *ids, int32_t *offsets, int32_t *rows, int32_t *slots,
                int32_t *totals, hipStream_t s) {
    int bits = 1;
    while ((1 << bits) <= E) ++bits;
    const size_t lds = (size_t)(kPlanWaves + 2) * (E + 1) * sizeof(int);   // 74 KB at 1024 experts
    const int G = plan_groups(S);
    if (G == 1) {
        hipLaunchKernelGGL(plan_one_kernel<I>, dim3(1), dim3(kPlanThreads), lds, s, S, topk, E, bits, ids, offsets,
                           rows, slots);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(plan_count_kernel<I>, dim3(G), dim3(kPlanThreads), lds, s, S, E, bits, ids, totals);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(plan_place_kernel<I>, dim3(G), dim3(kPlanThreads), lds, s, S, topk, E, bits, ids, totals,
                       offsets, rows, slots);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: C[t][n] = sum_j weights[t][j] * Y[slots[t][j]][n], j ascending,
// fp32 fused multiply-adds, one rounding. A thread owns VEC neighbouring
// columns of one token: every row of Y is read once in whole vectors, C is
// written once, and no atomics are needed. Bound by memory: 4099 tokens of 4
// fp16 rows of 4096 columns (168 MB) 34 us from memory (4.9 TB/s; a tenth of
// the choices elsewhere and two sets in turn, partly from the last-level cache,
// 28); 16 tokens of 8 rows 3.8 us, of which most is the launch. Where N is not a
// multiple of 8 a thread owns one column and the loads are what bounds it: 4100
// columns 105 us, 1.6 TB/s.
// Block x covers one of `cols` column strips of one of `per` tokens, block y
// the next `per`: the threads of a launch along x must stay below 2^32.
// ---------------------------------------------------------------------------
constexpr unsigned kCombineX = 1u << 22;      // workgroups of 256 threads along x, at most

template <class TY, class TC, int VEC>
__global__ __launch_bounds__(256) void combine_kernel(int T, int topk, int N, int S, const TY *__restrict__ Y,
                                                      const int32_t *__restrict__ slots,
                                                      const float *__restrict__ weights, TC *__restrict__ C,
                                                      unsigned cols, unsigned per) {
    typedef TY yv __attribute__((ext_vector_type(VEC)));
    typedef TC cv __attribute__((ext_vector_type(VEC)));
    const size_t t = (size_t)blockIdx.y * per + blockIdx.x / cols;
    const int n = ((int)(blockIdx.x % cols) * 256 + (int)threadIdx.x) * VEC;
    if (n >= N || t >= (size_t)T) return;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    const int32_t *sl = slots + t * topk;
    const float *wt = weights + t * topk;
    for (int j = 0; j < topk; ++j) {
        const int s = sl[j];
        if (s < 0 || s >= S) continue;            // uniform
        const float w = wt[j];
        const yv y = *reinterpret_cast<const yv *>(Y + (size_t)s * N + n);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, (float)y[i], acc[i]);
    }
    cv o;
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = (TC)acc[i];
    *reinterpret_cast<cv *>(C + t * N + n) = o;
}

template <class TY, class TC, int VEC>
hipError_t combine_vec(int T, int topk, int N, int S, const void *Y, const int32_t *slots, const float *weights,
                       void *C, hipStream_t s) {
    const unsigned cols = (unsigned)div_up(N, 256 * VEC), most = kCombineX / cols;
    const unsigned per = (unsigned)T < most ? (unsigned)T : most;
    hipLaunchKernelGGL((combine_kernel<TY, TC, VEC>), dim3(per * cols, ((unsigned)T + per - 1) / per), dim3(256), 0, s,
                       T, topk, N, S, static_cast<const TY *>(Y), slots, weights, static_cast<TC *>(C), cols, per);
    return hipGetLastError();
}

// Whole vectors only where every row of Y and C starts on a vector.
template <class TY, class TC>
hipError_t combine(int T, int topk, int N, int S, const void *Y, const int32_t *slots, const float *weights,
                   void *C, hipStream_t s) {
    return N % 8 == 0 ? combine_vec<TY, TC, 8>(T, topk, N, S, Y, slots, weights, C, s)
                      : combine_vec<TY, TC, 1>(T, topk, N, S, Y, slots, weights, C, s);
}

}  // namespace

hipError_t launch_group_plan(int S, int topk, int E, const void *ids, bool ids64, int32_t *offsets, int32_t *rows,
                             int32_t *slots, int32_t *totals, hipStream_t s) {
    return ids64 ? plan(S, topk, E, static_cast<const int64_t *>(ids), offsets, rows, slots, totals, s)
                 : plan(S, topk, E, static_cast<const int32_t *>(ids), offsets, rows, slots, totals, s);
}

hipError_t launch_group_combine(int T, int topk, int N, int S, const void *Y, bool y16, const int32_t *slots,
                                const float *weights, void *C, bool c16, hipStream_t s) {
    if (y16)
        return c16 ? combine<_Float16, _Float16>(T, topk, N, S, Y, slots, weights, C, s)
                   : combine<_Float16, float>(T, topk, N, S, Y, slots, weights, C, s);
    return c16 ? combine<float, _Float16>(T, topk, N, S, Y, slots, weights, C, s)
               : combine<float, float>(T, topk, N, S, Y, slots, weights, C, s);
}

}  // namespace qg
