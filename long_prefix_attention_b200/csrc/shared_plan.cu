// shared_plan.cu -- the plan of a shared-prefix attention call, made on the
// GPU from the step's lengths.
//
// One block: running maxima make the offsets monotone whatever they hold,
// then sums over the rows, the runs of rows that share prefix tiles and the
// tiles give the tile list, the cost and the partial rows before each tile.  Bound by
// latency: some ten sums over the block, one after the other (10 us for 16 to 64
// rows, 14 for 600, 56 for 4096); a step's layers share one plan.  A step of few
// rows and tokens takes 128 threads, whose sums are shorter, longer ones 1024 (in a
// captured graph, 128 against 1024: 16 rows 8.5 and 10.7 us, 100 8.5 and 11.0, 128 11.0
// and 11.2, 129 12.2 and 11.2, 400 20.9 and 12.7).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"
#include "shared.cuh"

namespace asmk {
namespace shared {


constexpr int kSmallPlan = 128;   // threads of a small step's plan

struct PlanArgs {
    const int *q_off, *seq_len, *group_off, *prefix_len;
    int R, NG, T, Hq, Hkv, S, max_pages, max_prefix_pages, workers;
    char *plan;
};

// N threads.
template <int N, typename Op>
__device__ __forceinline__ long long plan_scan(long long v, long long *warp_v, long long zero, long long &tot, Op op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, m);
        if (lane >= m) v = op(o, v);
    }
    __syncthreads();
    if (lane == 31) warp_v[warp] = v;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < N / 32 ? warp_v[lane] : zero;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, w, m);
            if (lane >= m) w = op(o, w);
        }
        if (lane < N / 32) warp_v[lane] = w;
    }
    __syncthreads();
    tot = warp_v[N / 32 - 1];
    return warp > 0 ? op(warp_v[warp - 1], v) : op(zero, v);
}

// First index i < n with ends[i] > x (n if there is none); ends ascending.
__device__ __forceinline__ int first_above(const int *ends, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// off[0..n] = running maxima of src, kept within [0, hi].
template <int N>
__device__ void monotone(const int *src, int *off, int n, int hi, long long *warp_v) {
    const int per = (n + 1 + N - 1) / N, i0 = threadIdx.x * per;
    long long m = 0, tot;
    for (int i = i0; i < i0 + per && i <= n; ++i) m = max(m, (long long)min(max(src[i], 0), hi));
    const long long inc = plan_scan<N>(m, warp_v, 0, tot, [](long long a, long long b) { return max(a, b); });
    // the maximum before this thread's entries: the inclusive one of its left neighbour
    __shared__ int left[N];
    left[threadIdx.x] = (int)inc;
    __syncthreads();
    int run = threadIdx.x > 0 ? left[threadIdx.x - 1] : 0;
    for (int i = i0; i < i0 + per && i <= n; ++i) {
        run = max(run, min(max(src[i], 0), hi));
        off[i] = run;
    }
    __syncthreads();
}

template <int N>
__global__ void __launch_bounds__(N)
shared_plan_kernel(const PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ long long warp_v[32];
    const int R = a.R, NG = a.NG, tid = threadIdx.x, G = a.Hq / a.Hkv;
    // offsets; tiles up to and with each row's and each run's; a row's run, a run's first and last row
    int *qo = sm, *go = qo + R + 1, *row_end = go + NG + 1, *run_end = row_end + R, *run_of = run_end + R,
        *run_lo = run_of + R, *run_hi = run_lo + R;
    const PlanLayout lay = plan_layout(R, NG, a.T, G);
    Header *hdr = reinterpret_cast<Header *>(a.plan);
    int *first = reinterpret_cast<int *>(a.plan + lay.first);
    Tile *tiles = reinterpret_cast<Tile *>(a.plan + lay.tiles);
    int2 *tok = reinterpret_cast<int2 *>(a.plan + lay.tok);
    const auto add = [](long long x, long long y) { return x + y; };
    const int dual = kDualRows / G;  // tokens of a 256-row tile
    const int single = kTileRows / G;

    monotone<N>(a.q_off, qo, R, a.T, warp_v);
    if (NG > 0) monotone<N>(a.group_off, go, NG, R, warp_v);
    // tiles of n tokens: one of up to 128 query rows, else 256-row ones
    auto n_tiles = [&](int n) { return n <= 0 ? 0 : n <= single ? 1 : (n + dual - 1) / dual; };
    // group of a row, -1 for none
    auto group_of = [&](int r) {
        if (NG == 0 || r < go[0] || r >= go[NG]) return -1;
        return first_above(go + 1, NG, r);
    };
    auto prefix_keys = [&](int g) {
        return (int)min((long long)max(a.prefix_len[g], 0), (long long)a.max_prefix_pages * a.S);
    };
    auto tall_row = [&](int r) { return qo[r + 1] - qo[r] > single; };
    // a run: neighbouring rows of one group, none of them tall
    auto starts_run = [&](int r, int g) {
        return g >= 0 && !tall_row(r) && (r == go[g] || tall_row(r - 1));
    };
    const int per = (R + N - 1) / N, r0 = tid * per, r1 = min(r0 + per, R);
    long long tot, n_runs, n_prefix;
    {
        long long s = 0;
        for (int r = r0; r < r1; ++r) s += starts_run(r, group_of(r));
        long long e = plan_scan<N>(s, warp_v, 0, n_runs, add) - s;
        for (int r = r0; r < r1; ++r) {
            const int g = group_of(r);
            if (starts_run(r, g)) run_lo[e++] = r;
            const bool in = g >= 0 && !tall_row(r);
            run_of[r] = in ? (int)e - 1 : -1;
            if (in && (r + 1 == go[g + 1] || tall_row(r + 1))) run_hi[e - 1] = r + 1;
        }
    }
    __syncthreads();
    // prefix tiles come first: theirs are the long key lists
    {
        long long s = 0;
        for (int i = r0; i < min(r0 + per, (int)n_runs); ++i) s += n_tiles(qo[run_hi[i]] - qo[run_lo[i]]);
        long long e = plan_scan<N>(s, warp_v, 0, n_prefix, add) - s;
        for (int i = r0; i < min(r0 + per, (int)n_runs); ++i) {
            e += n_tiles(qo[run_hi[i]] - qo[run_lo[i]]);
            run_end[i] = (int)e;
        }
    }
    {
        long long s = 0;
        for (int r = r0; r < r1; ++r) s += n_tiles(qo[r + 1] - qo[r]);
        long long e = n_prefix + plan_scan<N>(s, warp_v, 0, tot, add) - s;
        for (int r = r0; r < r1; ++r) {
            e += n_tiles(qo[r + 1] - qo[r]);
            row_end[r] = (int)e;
        }
    }
    __syncthreads();
    const int ntiles = (int)(n_prefix + tot);
    // ---- the tiles, and the cost before each (chunks of one tile a thread)
    long long before = 0;
    int tall = 0;
    for (int c = 0; c < ntiles; c += N) {
        const int i = c + tid;
        Tile t{};
        if (i < ntiles) {
            if (i < n_prefix) {
                const int q = first_above(run_end, (int)n_runs, i), g = group_of(run_lo[q]);
                const int t0 = qo[run_lo[q]], n = qo[run_hi[q]] - t0, len = n <= single ? n : dual;
                const int j = i - (q > 0 ? run_end[q - 1] : 0);
                t.tok0 = t0 + j * len;
                t.ntok = min(len, n - j * len);
                t.group = g;
                t.pre_keys = prefix_keys(g);
            } else {
                const int r = first_above(row_end, R, i), g = group_of(r);
                const int t0 = qo[r], n = qo[r + 1] - t0, len = n <= single ? n : dual;
                const int j = i - (r > 0 ? row_end[r - 1] : (int)n_prefix);
                const int seq = (int)min((long long)max(a.seq_len[r], 0), (long long)a.max_pages * a.S);
                t.tok0 = t0 + j * len;
                t.ntok = min(len, n - j * len);
                t.row = r;
                t.base = seq - n + j * len;
                t.keys = min(max(t.base + t.ntok, 0), seq);
                const int pre = g >= 0 ? prefix_keys(g) : 0;
                if (n > single && g >= 0) {
                    t.group = g;
                    t.pre_keys = pre;
                }
                t.direct = pre == 0 || n > single;
            }
            t.units = (t.pre_keys + kUnitKeys - 1) / kUnitKeys + (t.keys + kUnitKeys - 1) / kUnitKeys;
        }
        const long long cost = cost_of(t.ntok * G, t.units);
        const long long inc = plan_scan<N>(cost, warp_v, 0, tot, add);
        t.cost0 = before + inc - cost;
        before += tot;
        tall |= t.ntok * G > kTileRows;
        if (i < ntiles) tiles[i] = t;
    }
    const long long W = before * a.Hkv;
    long long range = (W + a.workers - 1) / a.workers;
    const int dearest = cost_unit(__syncthreads_or(tall) ? kDualRows : kTileRows);
    range = range < dearest ? dearest : range;
    const bool too_long = range > INT32_MAX;      // hours of work: no plan (the attention refuses a header without its magic)
    // ---- partial rows before each tile
    before = 0;
    for (int c = 0; c < ntiles; c += N) {
        const int i = c + tid;
        long long rows = 0;
        int cap = 0;
        if (i < ntiles && tiles[i].units > 0) {
            cap = (int)(cost_of(tiles[i].ntok * G, tiles[i].units) / range) + 2;
            rows = (long long)cap * a.Hkv * tiles[i].ntok * G;
        }
        const long long inc = plan_scan<N>(rows, warp_v, 0, tot, add);
        if (i < ntiles) {
            tiles[i].cap = cap;
            tiles[i].row0 = before + inc - rows;
            // the workers whose ranges begin in this tile
            const long long c0 = tiles[i].cost0 * a.Hkv, c1 = c0 + cost_of(tiles[i].ntok * G, tiles[i].units) * a.Hkv;
            for (long long w = (c0 + range - 1) / range; !too_long && w * range < c1; ++w) first[w] = i;
        }
        before += tot;
    }
    // ---- the tiles of every token
    for (int t = tid; t < a.T; t += N) {
        int2 v = make_int2(-1, -1);
        if (t >= qo[0] && t < qo[R]) {
            const int r = first_above(qo + 1, R, t);
            const int n = qo[r + 1] - qo[r];
            v.x = (r > 0 ? row_end[r - 1] : (int)n_prefix) + (n <= single ? 0 : (t - qo[r]) / dual);
            const int q = run_of[r];
            if (q >= 0) {
                const int t0 = qo[run_lo[q]], gn = qo[run_hi[q]] - t0;
                v.y = (q > 0 ? run_end[q - 1] : 0) + (gn <= single ? 0 : (t - t0) / dual);
            }
        }
        tok[t] = v;
    }
    if (tid == 0) {
        Header h{};
        h.magic = too_long ? 0 : kMagic;
        h.R = R; h.NG = NG; h.T = a.T; h.Hq = a.Hq; h.Hkv = a.Hkv;
        h.page_size = a.S; h.max_pages = a.max_pages; h.max_prefix_pages = a.max_prefix_pages;
        h.workers = a.workers; h.ntiles = ntiles; h.range = (int)range; h.W = W; h.inv_range = 1.0 / (double)range;
        *hdr = h;
    }
}

template <int N>
cudaError_t launch_plan(const PlanArgs &a, cudaStream_t st) {
    const size_t smem = sizeof(int) * (6 * (size_t)a.R + (size_t)a.NG + 2);
    if (smem > 40 * 1024) {  // beside the static arrays
        cudaError_t e = cudaFuncSetAttribute(shared_plan_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (7 * kMaxRows + 2) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    shared_plan_kernel<N><<<1, N, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace shared
}  // namespace asmk

size_t asm_shared_plan_bytes(int R, int NG, int T, int Hq, int Hkv) {
    return asmk::shared::plan_layout(R, NG, T, Hq / Hkv).total;
}

cudaError_t asm_shared_plan_launch(const int32_t *q_off, const int32_t *seq_len, const int32_t *group_off,
                                   const int32_t *prefix_len, int R, int NG, int T, int Hq, int Hkv, int page_size,
                                   int max_pages, int max_prefix_pages, void *plan, int num_sms, cudaStream_t st) {
    using namespace asmk::shared;
    PlanArgs a{};
    a.q_off = q_off; a.seq_len = seq_len; a.group_off = group_off; a.prefix_len = prefix_len;
    a.R = R; a.NG = NG; a.T = T; a.Hq = Hq; a.Hkv = Hkv;
    a.S = page_size; a.max_pages = max_pages; a.max_prefix_pages = max_prefix_pages;
    a.workers = num_sms < kMaxWorkers ? num_sms : kMaxWorkers;
    a.plan = static_cast<char *>(plan);
    if (R <= kSmallPlan && T <= 2 * kSmallPlan) return launch_plan<kSmallPlan>(a, st);
    return launch_plan<1024>(a, st);
}
