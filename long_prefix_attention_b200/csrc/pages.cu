// pages.cu -- page tables and slot maps of one step, built from the rows' lengths.
//
// A row of kv tokens holds ceil(kv / S) pages of S tokens.  n new tokens need
//   need = ceil((kv + n) / S) - ceil(kv / S)
// further pages, taken from the head of a ring of free pages in row order; a
// row is granted all of its pages or none (need == 0, or the running sum of
// the needs, this row included, does not exceed the free count).  Rows that
// end give their pages back behind the ring's tail.  Everything a token or a
// moved page has to know follows from exclusive sums over the rows, so there
// is one launch and no communication between blocks: every block forms the
// sums of all rows again in shared memory (at most 4096 rows, 32 KB of lengths from
// L2) and then takes its share of the tokens and of the moved pages, each of
// which finds its row by bisection.  Nothing read is written in the same
// call (the ring's taken and returned places are disjoint), so a call can be
// repeated on the same inputs.  Bound by latency: two dependent trips to
// memory, the lengths and a token's page (16 rows 5.0 us in a captured graph,
// 1500 rows 9.4), and for many rows by the sums (see the rule at the launch).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"

namespace asmk {
namespace pages {

constexpr int kThreads = 512;
constexpr int kMaxRows = 4096;

struct Args {
    const int *kv_len, *new_len, *pos_base, *pool_state;
    int *pool, *table, *seq_len, *q_off, *row, *pos, *slot, *pool_out;
    int R, F, shift, max_pages, T;
};

// Place i of a ring of F from its place `head` on: head < F, i <= F.
__device__ __forceinline__ int ring(int head, long long i, int F) {
    const long long p = head + i;
    return (int)(p >= F ? p - F : p);
}

// Inclusive sum over the block's threads in order; `tot` gets the total.
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sums, long long &tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, m);
        if (lane >= m) v += o;
    }
    __syncthreads();  // the sums of the previous call have been read
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    long long before = 0;
    tot = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long s = warp_sums[w];
        if (w < warp) before += s;
        tot += s;
    }
    return before + v;
}

// First index r < R with ends[r] > t (R if there is none).
__device__ __forceinline__ int find_row(const int *ends, int R, int t) {
    int lo = 0, hi = R;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// PER: rows per thread at most.
template <int PER>
__global__ void __launch_bounds__(kThreads)
page_step_kernel(const Args a) {
    extern __shared__ int sm[];
    __shared__ long long warp_sums[kThreads / 32];
    __shared__ int s_refused;
    const int R = a.R, tid = threadIdx.x;
    int *tok_end = sm, *give_end = sm + R, *back_end = sm + 2 * R;
    int *kv_ok = sm + 3 * R;  // the row's cached tokens; complemented where it was refused
    const int S1 = (1 << a.shift) - 1;
    const long long cap = (long long)a.max_pages << a.shift;
    if (tid == 0) s_refused = 0;

    const int head0 = a.pool_state[0], cnt0 = a.pool_state[1];
    const int count = min(max(cnt0, 0), a.F);
    const int head = (int)((unsigned)max(head0, 0) % (unsigned)a.F);

    // rows [r0, r0 + PER) of this thread
    const int r0 = tid * PER;
    int kv[PER], nw[PER];
    long long sum = 0, tot;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = r0 + i;
        const bool in = r < R;
        const int k = in ? a.kv_len[r] : 0;
        kv[i] = (int)min((long long)max(k, 0), cap);
        nw[i] = in ? a.new_len[r] : 0;
        sum += max(nw[i], 0);
    }
    // ends of the rows' tokens in the batch
    long long end = block_scan(sum, warp_sums, tot) - sum;
    long long need[PER];
    unsigned fits = 0;
    sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        end += max(nw[i], 0);
        if (r0 + i < R) tok_end[r0 + i] = (int)min(end, (long long)a.T);
        const long long want = (long long)kv[i] + max(nw[i], 0);
        const bool f = nw[i] >= 0 && end <= a.T && want <= cap;
        fits |= (unsigned)f << i;
        need[i] = f ? ((want + S1) >> a.shift) - (((long long)kv[i] + S1) >> a.shift) : 0;
        sum += need[i];
    }
    // grants, in row order
    long long asked = block_scan(sum, warp_sums, tot) - sum;
    long long gives = 0, backs = 0;
    unsigned ok = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        asked += need[i];
        const bool o = ((fits >> i) & 1u) && (need[i] == 0 || asked <= count);
        ok |= (unsigned)o << i;
        if (o) gives += need[i];
        if (nw[i] < 0) backs += ((long long)kv[i] + S1) >> a.shift;
    }
    long long n_give, n_back;
    long long ge = block_scan(gives, warp_sums, n_give) - gives;
    long long be = block_scan(backs, warp_sums, n_back) - backs;
    n_back = min(n_back, (long long)(a.F - count));  // a ring cannot hold more than it has places
    int refused = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = r0 + i;
        if (r >= R) continue;
        const bool o = (ok >> i) & 1u;
        if (o) ge += need[i];
        if (nw[i] < 0) be += ((long long)kv[i] + S1) >> a.shift;
        give_end[r] = (int)ge;                            // <= count
        back_end[r] = (int)min(be, (long long)INT32_MAX);
        kv_ok[r] = o ? kv[i] : ~kv[i];
        if (!o && nw[i] > 0) ++refused;
        if (blockIdx.x == 0) a.seq_len[r] = nw[i] < 0 ? 0 : (o ? kv[i] + nw[i] : kv[i]);
    }
    if (refused) atomicAdd(&s_refused, refused);
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int r = tid; r <= R; r += kThreads) a.q_off[r] = r == 0 ? 0 : tok_end[r - 1];
        if (tid == 0) {
            a.pool_out[0] = ring(head, n_give, a.F);
            a.pool_out[1] = (int)(count - n_give + n_back);
            a.pool_out[2] = s_refused;
        }
    }

    // the page with index j of row r, whose first `held` pages were there before
    auto page_of = [&](int r, int j, int held, int gstart) {
        if (j < held) return a.table[(size_t)r * a.max_pages + j];
        return a.pool[ring(head, gstart + (j - held), a.F)];
    };
    const int step = gridDim.x * kThreads;
    for (int t = blockIdx.x * kThreads + tid; t < a.T; t += step) {
        const int r = find_row(tok_end, R, t);
        int pos = 0, slot = -1;
        if (r < R) {
            const int c = kv_ok[r], k = c < 0 ? ~c : c;
            const int x = k + t - (r > 0 ? tok_end[r - 1] : 0);
            pos = x + (a.pos_base ? a.pos_base[r] : 0);
            if (c >= 0) {
                const int id = page_of(r, x >> a.shift, (int)(((long long)k + S1) >> a.shift), r > 0 ? give_end[r - 1] : 0);
                const long long s = ((long long)id << a.shift) + (x & S1);
                if (id >= 0 && s <= INT32_MAX) slot = (int)s;
            }
        }
        a.row[t] = r < R ? r : -1;
        a.pos[t] = pos;
        a.slot[t] = slot;
    }
    // granted pages into the table, returned pages behind the ring's tail
    for (long long i = (long long)blockIdx.x * kThreads + tid; i < n_give; i += step) {
        const int r = find_row(give_end, R, (int)i), gs = r > 0 ? give_end[r - 1] : 0;
        const int c = kv_ok[r], held = (int)(((long long)(c < 0 ? ~c : c) + S1) >> a.shift);
        a.table[(size_t)r * a.max_pages + held + ((int)i - gs)] = a.pool[ring(head, i, a.F)];
    }
    for (long long i = (long long)blockIdx.x * kThreads + tid; i < n_back; i += step) {
        const int r = find_row(back_end, R, (int)i), j = (int)i - (r > 0 ? back_end[r - 1] : 0);
        a.pool[ring(head, count + i, a.F)] = a.table[(size_t)r * a.max_pages + j];
    }
}

template <int PER>
cudaError_t launch(const Args &a, int blocks, cudaStream_t st) {
    const size_t smem = sizeof(int) * 4 * (size_t)a.R;
    if (smem > 40 * 1024) {  // beside the static arrays
        cudaError_t e = cudaFuncSetAttribute(page_step_kernel<PER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             4 * kMaxRows * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    page_step_kernel<PER><<<blocks, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace pages
}  // namespace asmk

cudaError_t asm_page_step_launch(const int32_t *kv_len, const int32_t *new_len, const int32_t *pos_base, int R,
                                 int page_size, int max_pages, int32_t *table, int32_t *pool,
                                 const int32_t *pool_state, int F, int T, int32_t *seq_len, int32_t *q_off,
                                 int32_t *row, int32_t *pos, int32_t *slot, int32_t *pool_out, int num_sms,
                                 cudaStream_t st) {
    using namespace asmk::pages;
    Args a{};
    a.kv_len = kv_len; a.new_len = new_len; a.pos_base = pos_base; a.pool_state = pool_state;
    a.pool = pool; a.table = table; a.seq_len = seq_len; a.q_off = q_off;
    a.row = row; a.pos = pos; a.slot = slot; a.pool_out = pool_out;
    a.R = R; a.F = F; a.max_pages = max_pages; a.T = T;
    a.shift = 0;
    while ((1 << a.shift) < page_size) ++a.shift;
    // one token a thread, up to a block per SM; the moved pages are at most about as many
    int blocks = (T + kThreads - 1) / kThreads;
    const int by_rows = (R + 127) / 128;
    blocks = blocks > by_rows ? blocks : by_rows;
    blocks = blocks < num_sms ? blocks : num_sms;
    blocks = blocks < 1 ? 1 : blocks;
    // Rows per thread: a thread's rows follow one another in four 64-bit sums, so as few as
    // there are threads for: 512 rows 5.7 us with one, 5.9 with two, 8.0 with eight;
    // 1024 rows 6.3 with two, 8.3 with eight (what 1025 rows and more take: 8.2, 2000 8.9).
    if (R <= kThreads) return launch<1>(a, blocks, st);
    if (R <= 2 * kThreads) return launch<2>(a, blocks, st);
    return launch<kMaxRows / kThreads>(a, blocks, st);
}
