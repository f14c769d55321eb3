// shared_attn.cu -- attention of a ragged batch over shared prefixes and the
// rows' own pages: the CUDA-core kernel (fp32 storage) and the merge of the
// partial states.
//
// For token t of row r and query head h (KV head g = h / G), over the keys j
// of the row's prefix group and the local keys up to the token itself:
//   m = max_j s <q, k_j>,  l = sum_j e^(s <q, k_j> - m),
//   o = sum_j e^(s <q, k_j> - m) v_j,   out = o / l,   lse = m + ln l,
// one pass over the keys with running (m, l, o) (in base 2); states of
// disjoint key sets join by rescaling both to the larger maximum.
//
// A prefix tile holds query rows of all the rows of its group, so a prefix is
// read once for up to 256 query rows.  Each CTA takes one worker's range of
// the plan's unit sequence.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"
#include "shared.cuh"

namespace asmk {
namespace shared {

// ------------------------------------------------------- CUDA-core kernel --
//
// Half a unit, 64 keys, at a time in shared memory, the next half on its way
// (cp.async, two buffers).  Tiles of up to 16 query rows (decode): four
// threads share a 4 x 4 block of scores (a quarter of the products each), the
// 16 threads of a row find its weights, and each half-warp adds 4 keys to a
// whole 16 x D output, summed over the half-warps at the end; so K and V leave
// shared memory once per half (64 rows of 2048 local keys: 139 us, a row-wise
// split that waits for its loads 190).  Longer tiles take 32, 48 or 64 rows at a
// time, 2, 3 or 4 rows x 4 keys of scores a thread (always 64: 279 us against 251
// for 20 rows of a group behind 20000 keys, 49 against 43 for 44 query rows behind
// 4000); 17 to 64 rows through the short path in turns of 16 measured slower (44
// rows: 64 us).  Neither form reaches the FMA rate: a thread loads 4 + MR words of 16
// bytes from shared memory for 16 MR FMAs of the scores, and waits at barriers.
// 44 query rows behind two 4000-key prefixes: 43 us, the FMA pipe 12% busy, the SMs
// half of the time, since 172 units of 128 keys meet 148 SMs; 1447 tokens of four
// chunks behind 4000 keys 937 us, 36% of the FMA rate.

__device__ __forceinline__ float dot4(const float4 &x, const float4 &y, float t) {
    t = fmaf(x.x, y.x, t);
    t = fmaf(x.y, y.y, t);
    t = fmaf(x.z, y.z, t);
    return fmaf(x.w, y.w, t);
}
__device__ __forceinline__ void axpy4(float w, const float4 &v, float4 &o) {
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
}
__device__ __forceinline__ void scale4(float f, float4 &o) {
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
}

constexpr int kThreads = 256;
constexpr int kKB = 64;   // keys per step
constexpr int kFew = 16;  // query rows of a short tile

template <int D>
struct Smem {
    static constexpr int LD = D + 4, LQ = D + 16, LP = kKB + 4;
    float q[64 * LQ], k[2][kKB * LD], v[2][kKB * LD];
    float p[64 * LP];     // scores, then weights; few rows: weights by key, [kKB][kFew + 4]
    float al[kFew];       // few rows: this step's factor on a row's output
    float2 ml[kFew];      // few rows: a row's (max, sum)
};
static_assert(kKB * (kFew + 4) + kFew * (kKB + 4) <= 64 * (kKB + 4), "scores and weights of few rows");

// Where the keys of the half unit `hu` of a segment lie.
struct Half {
    int kb, k1;           // first key; end of its list
    const int *list;
    bool pre;
};
__device__ __forceinline__ Half half_of(const AttnArgs &a, const Seg &s, int hu) {
    const int pu = (s.t.pre_keys + kUnitKeys - 1) / kUnitKeys;  // prefix units
    Half f;
    f.pre = hu < 2 * pu;
    f.kb = (f.pre ? hu : hu - 2 * pu) * kKB;
    f.k1 = f.pre ? s.t.pre_keys : s.t.keys;
    f.list = f.pre ? a.prefix_table + (size_t)s.t.group * a.max_prefix_pages
                   : a.table + (size_t)s.t.row * a.max_pages;
    return f;
}

// Start the copies of a half; places behind the list's end and of bad pages
// become zeros.
template <int D>
__device__ __forceinline__ void start_keys(const AttnArgs &a, int g, const Half &f, float *k, float *v) {
    constexpr int LD = Smem<D>::LD, C = D / 4, N = kKB * C / kThreads;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / C, c = (e - r * C) * 4, key = f.kb + r;
        int id = key < f.k1 ? f.list[key >> a.shift] : -1;
        if (key < f.k1 && (id < 0 || id >= a.n_pages)) {
            id = -1;
            atomicExch(a.ws_err, (int)ASM_ERR_INVALID_ARG);
        }
        const long long off = id < 0 ? 0 : ((((long long)id * a.Hkv + g) << a.shift) + (key & (a.S - 1))) * D + c;
        const uint32_t bytes = id < 0 ? 0u : 16u;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(smem_addr(k + r * LD + c)), "l"(static_cast<const float *>(a.k_pages) + off), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(smem_addr(v + r * LD + c)), "l"(static_cast<const float *>(a.v_pages) + off), "r"(bytes)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void wait_keys() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <int D>
__device__ __forceinline__ void load_queries(const AttnArgs &a, const Seg &s, int rb, int n, int rows, float *q) {
    for (int i = threadIdx.x; i < n * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i - r * (D / 4)) * 4, rr = rb + r;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (rr < rows)
            load_vec<float, 4>(static_cast<const float *>(a.q) +
                                   ((size_t)(s.t.tok0 + rr / a.G) * a.Hq + s.g * a.G + rr % a.G) * D + c, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= a.sl2;
        store_vec<float, 4>(q + r * Smem<D>::LQ + c, x);
    }
}

// One row's 4 columns of a finished segment: the output itself, or a partial state.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs &a, const Seg &s, int rows, int rr, int col, float4 o, float m,
                                          float l, bool stats) {
    if (s.direct) {
        const size_t th = (size_t)(s.t.tok0 + rr / a.G) * a.Hq + s.g * a.G + rr % a.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + th * D + col) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (a.lse && stats) a.lse[th] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
    } else {
        *reinterpret_cast<float4 *>(a.ws_o + partial_at(s.prow, rows, rr, col, D)) = o;
        if (stats) a.ws_ml[s.prow + rr] = make_float2(m, l);
    }
}

template <int D>
__device__ void run_few(const AttnArgs &a, const Seg &s, Smem<D> &sm) {
    constexpr int LD = Smem<D>::LD, LQ = Smem<D>::LQ, LS = kKB + 4, LW = kFew + 4, NC = D / 64;
    const int tid = threadIdx.x, tx = tid & 15, hw = tid >> 4;
    const int rows = s.t.ntok * a.G;
    float *sc = sm.p, *wt = sm.p + kFew * LS;        // [kFew][LS] scores, [kKB][LW] weights
    // scores: places 4 (ds + 4 t) .. of rows r4 + 4 i and keys k16 + 16 j
    const int ds = tid & 3, r4 = (tid >> 2) & 3, k16 = tid >> 4;
    const int own = min(s.t.keys, s.t.base + hw / a.G + 1);   // weights: row hw
    const int own_first = min(s.t.keys, s.t.base + 1);
    float m = kNegInf, l = 0.f;
    float4 o[kFew][NC];
#pragma unroll
    for (int r = 0; r < kFew; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();                                  // the segment before is done with the buffers
    start_keys<D>(a, s.g, half_of(a, s, 2 * s.k), sm.k[0], sm.v[0]);
    load_queries<D>(a, s, 0, kFew, rows, sm.q);
    int buf = 0;
    for (int hu = 2 * s.k; hu < 2 * (s.k + s.n); ++hu) {
        const Half f = half_of(a, s, hu);
        wait_keys();
        __syncthreads();                              // this half is here, the other buffer free
        if (hu + 1 < 2 * (s.k + s.n)) start_keys<D>(a, s.g, half_of(a, s, hu + 1), sm.k[buf ^ 1], sm.v[buf ^ 1]);
        if (f.kb < f.k1) {
            {
                float t[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = 0.f;
#pragma unroll 4
                for (int d = 4 * ds; d < D; d += 16) {
                    float4 kx[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        kx[j] = *reinterpret_cast<const float4 *>(sm.k[buf] + (k16 + 16 * j) * LD + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 qx = *reinterpret_cast<const float4 *>(sm.q + (r4 + 4 * i) * LQ + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[i][j] = dot4(qx, kx[j], t[i][j]);
                    }
                }
                // the four threads' sums: two rows, then one row each
                const bool hi = ds & 2, odd = ds & 1;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float send = hi ? t[i][j] : t[i + 2][j], keep = hi ? t[i + 2][j] : t[i][j];
                        t[i][j] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float send = odd ? t[0][j] : t[1][j], keep = odd ? t[1][j] : t[0][j];
                    sc[(r4 + 4 * ds) * LS + k16 + 16 * j] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
                }
            }
            __syncthreads();
            {
                const int lim = f.pre ? f.k1 : own;
                float x[4], mx = kNegInf;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = f.kb + tx + 16 * j < lim ? sc[hw * LS + tx + 16 * j] : kNegInf;
                    mx = fmaxf(mx, x[j]);
                }
#pragma unroll
                for (int i = 8; i >= 1; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
                const float mn = fmaxf(m, mx), ref = mn == kNegInf ? 0.f : mn, al = exp2f(m - ref);
                m = mn;
                float ps = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(x[j] - ref);
                    ps += p;
                    wt[(tx + 16 * j) * LW + hw] = p;
                }
#pragma unroll
                for (int i = 8; i >= 1; i >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, i);
                l = l * al + ps;
                if (tx == 0) sm.al[hw] = al;
            }
            __syncthreads();
            // the weight of 0 of a key that a row does not see must not meet its value
            const bool masked = !f.pre && f.kb + kKB > own_first;
#pragma unroll
            for (int r = 0; r < kFew; ++r) {
                const float al = sm.al[r];
#pragma unroll
                for (int c = 0; c < NC; ++c) scale4(al, o[r][c]);
            }
#pragma unroll 2
            for (int i = 0; i < kKB / 16; ++i) {
                const int kk = hw * (kKB / 16) + i;
                const int hidden = masked ? (f.kb + kk - s.t.base) * a.G : 0;   // rows that do not see this key
                float4 vx[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    vx[c] = *reinterpret_cast<const float4 *>(sm.v[buf] + kk * LD + 64 * c + 4 * tx);
#pragma unroll
                for (int r = 0; r < kFew; r += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(wt + kk * LW + r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = e == 0 ? w4.x : e == 1 ? w4.y : e == 2 ? w4.z : w4.w;
                        if (r + e < hidden) continue;
#pragma unroll
                        for (int c = 0; c < NC; ++c) axpy4(w, vx[c], o[r + e][c]);
                    }
                }
            }
        }
        buf ^= 1;
    }
    // the half-warps' outputs meet in the key and value buffers
    static_assert(16 * kFew * D <= 4 * kKB * Smem<D>::LD, "outputs of the half-warps fit the buffers");
    float *all = sm.k[0];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFew; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            *reinterpret_cast<float4 *>(all + (hw * kFew + r) * D + 64 * c + 4 * tx) = o[r][c];
    if (tx == 0) sm.ml[hw] = make_float2(m, l);
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < 16; ++w) {
            const float4 x = *reinterpret_cast<const float4 *>(all + (w * kFew + r) * D + col);
            t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
        }
        const float2 ml = sm.ml[r];
        store_row<D>(a, s, rows, r, col, t, ml.x, ml.y, col == 0);
    }
}

// Rows rb .. rb + 16 MR of a tile: a thread has rows rb + ty + 16 i.
template <int D, int MR>
__device__ void run_rows(const AttnArgs &a, const Seg &s, Smem<D> &sm, int rb) {
    constexpr int LD = Smem<D>::LD, LQ = Smem<D>::LQ, LP = Smem<D>::LP, BR = 16 * MR, NC = D / 64;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int rows = s.t.ntok * a.G;
    __syncthreads();  // the previous rows are done with the buffers
    start_keys<D>(a, s.g, half_of(a, s, 2 * s.k), sm.k[0], sm.v[0]);
    load_queries<D>(a, s, rb, BR, rows, sm.q);
    float m[MR], l[MR];
    float4 o[MR][NC];
    int own[MR];  // local keys the row sees
#pragma unroll
    for (int i = 0; i < MR; ++i) {
        m[i] = kNegInf;
        l[i] = 0.f;
        const int rr = rb + ty + 16 * i;
        own[i] = min(s.t.keys, s.t.base + rr / a.G + 1);
#pragma unroll
        for (int c = 0; c < NC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int buf = 1;
    for (int hu = 2 * s.k; hu < 2 * (s.k + s.n); ++hu) {   // halves of units
        buf ^= 1;
        const Half f = half_of(a, s, hu);
        const bool pre = f.pre;
        const int kb = f.kb, k1 = f.k1;
        wait_keys();
        __syncthreads();  // this half is here, the other buffer free
        if (hu + 1 < 2 * (s.k + s.n)) start_keys<D>(a, s.g, half_of(a, s, hu + 1), sm.k[buf ^ 1], sm.v[buf ^ 1]);
        if (kb >= k1) continue;
        const float *kt = sm.k[buf], *vt = sm.v[buf];
        float sc[MR][4];
#pragma unroll
        for (int i = 0; i < MR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 kx[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) kx[j] = *reinterpret_cast<const float4 *>(kt + (tx + 16 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < MR; ++i) {
                const float4 qx = *reinterpret_cast<const float4 *>(sm.q + (ty + 16 * i) * LQ + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[i][j] = dot4(qx, kx[j], sc[i][j]);
            }
        }
        bool masked = false;
#pragma unroll
        for (int i = 0; i < MR; ++i) {
            float mx = kNegInf;
            const int lim = pre ? k1 : own[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (kb + tx + 16 * j >= lim) sc[i][j] = kNegInf;
                mx = fmaxf(mx, sc[i][j]);
            }
            masked |= kb + kKB > lim;
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[i], mx);
            const float ref = mn == kNegInf ? 0.f : mn;  // nothing seen yet: every weight is 0
            const float al = exp2f(m[i] - ref);
            m[i] = mn;
            float ps = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(sc[i][j] - ref);
                ps += p;
                sm.p[(ty + 16 * i) * LP + tx + 16 * j] = p;
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
            l[i] = l[i] * al + ps;
#pragma unroll
            for (int c = 0; c < NC; ++c) scale4(al, o[i][c]);
        }
        __syncwarp();
        const int kn = min(kKB, k1 - kb);
        for (int k = 0; k < kn; k += 4) {
            float4 px[MR];
#pragma unroll
            for (int i = 0; i < MR; ++i) px[i] = *reinterpret_cast<const float4 *>(sm.p + (ty + 16 * i) * LP + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 vx = *reinterpret_cast<const float4 *>(vt + (k + e) * LD + 64 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < MR; ++i) {
                        const float p = e == 0 ? px[i].x : e == 1 ? px[i].y : e == 2 ? px[i].z : px[i].w;
                        // the weight of 0 of a key that the row does not see must not meet its value
                        if (masked && kb + k + e >= (pre ? k1 : own[i])) continue;
                        axpy4(p, vx, o[i][c]);
                    }
                }
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < MR; ++i) {
        const int rr = rb + ty + 16 * i;
        if (rr >= rows) continue;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            store_row<D>(a, s, rows, rr, 64 * c + 4 * tx, o[i][c], m[i], l[i], c == 0 && tx == 0);
    }
}

template <int D>
__device__ void run_many(const AttnArgs &a, const Seg &s, Smem<D> &sm) {
    const int rows = s.t.ntok * a.G;
    for (int rb = 0; rb < rows; rb += 64) {
        if (rows - rb <= 32) run_rows<D, 2>(a, s, sm, rb);
        else if (rows - rb <= 48) run_rows<D, 3>(a, s, sm, rb);
        else run_rows<D, 4>(a, s, sm, rb);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
shared_attn_kernel(const AttnArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
    pdl_wait();
    pdl_launch_dependents();
    const Header h = *a.hdr;
    if (!plan_ok(a, h)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.ws_err, (int)ASM_ERR_INVALID_ARG);
        return;
    }
    Walk walk(a, h, blockIdx.x);  // one block per worker
    Seg s;
    while (walk.step(s)) {
        if (s.t.ntok * a.G <= kFew) run_few<D>(a, s, sm);
        else run_many<D>(a, s, sm);
    }
}

// ------------------------------------------------------------------ merge --
//
// NW warps per (token, KV head), G query rows at once: the rows of one token
// lie side by side in the partial states (16 bytes of each).  Lane l owns row
// l % G and the 4-column groups l / G + k 32 / G; each warp takes every NW-th
// state, four in flight, with running statistics, and the warps meet in shared
// memory.  Tokens whose only state was written as output already are skipped;
// tokens without any key get (0, -inf).  Bound by latency (offsets, tile,
// statistics and states are read one after the other; 7.5 us for 16 decode rows
// of 32 heads) for a few tokens, by memory for many.

constexpr int kMergeThreads = 256;

template <typename T, int D, int G, int NW>
__global__ void __launch_bounds__(kMergeThreads)
shared_merge_kernel(const AttnArgs a) {
    constexpr int C4 = D / 4, E = C4 * G < 32 ? 1 : C4 * G / 32;  // 4-column groups of a row, and per lane
    constexpr int PPB = kMergeThreads / 32 / NW;         // pairs per block
    __shared__ float4 so[NW > 1 ? kMergeThreads / 32 : 1][NW > 1 ? E : 1][32];
    __shared__ float2 sml[NW > 1 ? kMergeThreads / 32 : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % NW;
    const int hh = lane % G, cg = lane / G;
    const bool mine = C4 * G >= 32 || cg < C4;           // a row of 64 columns alone leaves half of the warp
    pdl_wait();
    pdl_launch_dependents();
    const Header h = *a.hdr;
    if (!plan_ok(a, h)) return;
    const long long pairs = (long long)a.T * a.Hkv;
    for (long long base = (long long)blockIdx.x * PPB; base < pairs; base += (long long)gridDim.x * PPB) {
        const long long pr = base + warp / NW;
        bool live = pr < pairs;
        const int t = live ? (int)(pr / a.Hkv) : 0, g = live ? (int)(pr - (long long)t * a.Hkv) : 0;
        const int2 tt = live ? a.tok[t] : make_int2(-1, -1);
        live = live && tt.x >= 0;               // tokens outside every row are left as they are
        // states of the two tiles: count, statistics and outputs of this lane's row, and their strides
        int n[2] = {0, 0};
        const float2 *ml[2] = {a.ws_ml, a.ws_ml};
        const float4 *po[2] = {reinterpret_cast<const float4 *>(a.ws_o), reinterpret_cast<const float4 *>(a.ws_o)};
        int rows[2] = {0, 0};
        if (live) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = x == 0 ? tt.x : tt.y;
                if (i < 0) continue;
                const Tile tl = a.tiles[i];
                rows[x] = tl.ntok * G;
                n[x] = segments(tl.cost0 * a.Hkv + g * cost_of(rows[x], tl.units), rows[x], tl.units, h);
                if (x == 0 && n[x] == 1 && tl.direct) live = false;  // already written
                const long long first = tl.row0 + (long long)g * tl.cap * rows[x];
                const int at = (t - tl.tok0) * G + hh;
                ml[x] += first + at;
                po[x] += first * C4 + (long long)cg * rows[x] + at;
            }
        }
        const int tot = live ? n[0] + n[1] : 0;
        float m = kNegInf, l = 0.f;
        float4 o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int e0 = sub; e0 < tot; e0 += 4 * NW) {
            float2 st[4];
            float4 v[4][E];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = e0 + j * NW;
                if (e >= tot) {
                    st[j] = make_float2(kNegInf, 0.f);
                    continue;
                }
                const int x = e < n[0] ? 0 : 1, ee = x ? e - n[0] : e;
                st[j] = __ldcg(ml[x] + (long long)ee * rows[x]);
                const float4 *p = po[x] + (long long)ee * rows[x] * C4;
#pragma unroll
                for (int k = 0; k < E; ++k)
                    v[j][k] = mine ? __ldcg(p + (long long)k * (32 / G) * rows[x]) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mn = m;
#pragma unroll
            for (int j = 0; j < 4; ++j) mn = fmaxf(mn, st[j].x);
            const float ref = mn == kNegInf ? 0.f : mn, al = exp2f(m - ref);
            m = mn;
            l *= al;
#pragma unroll
            for (int k = 0; k < E; ++k) { o[k].x *= al; o[k].y *= al; o[k].z *= al; o[k].w *= al; }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (st[j].y == 0.f) continue;   // an empty state's row may hold anything
                const float w = exp2f(st[j].x - ref);
                l = fmaf(w, st[j].y, l);
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    o[k].x = fmaf(w, v[j][k].x, o[k].x);
                    o[k].y = fmaf(w, v[j][k].y, o[k].y);
                    o[k].z = fmaf(w, v[j][k].z, o[k].z);
                    o[k].w = fmaf(w, v[j][k].w, o[k].w);
                }
            }
        }
        if (NW > 1) {
            __syncthreads();
            sml[warp][lane] = make_float2(m, l);
#pragma unroll
            for (int k = 0; k < E; ++k) so[warp][k][lane] = o[k];
            __syncthreads();
            if (sub == 0) {
                float mm = m;
                for (int w = 1; w < NW; ++w) mm = fmaxf(mm, sml[warp + w][lane].x);
                const float ref = mm == kNegInf ? 0.f : mm, al = exp2f(m - ref);
                l *= al;
#pragma unroll
                for (int k = 0; k < E; ++k) { o[k].x *= al; o[k].y *= al; o[k].z *= al; o[k].w *= al; }
                for (int w = 1; w < NW; ++w) {
                    const float2 s2 = sml[warp + w][lane];
                    const float x = exp2f(s2.x - ref);
                    l = fmaf(x, s2.y, l);
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const float4 y = so[warp + w][k][lane];
                        o[k].x = fmaf(x, y.x, o[k].x);
                        o[k].y = fmaf(x, y.y, o[k].y);
                        o[k].z = fmaf(x, y.z, o[k].z);
                        o[k].w = fmaf(x, y.w, o[k].w);
                    }
                }
                m = mm;
            }
        }
        if (live && sub == 0 && mine) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t th = (size_t)t * a.Hq + g * G + hh;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float y[4] = {o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv};
                store_vec<T, 4>(static_cast<T *>(a.out) + th * D + 4 * (cg + k * (32 / G)), y);
            }
            if (a.lse && cg == 0) a.lse[th] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
        }
    }
}

template <typename T, int D, int G>
cudaError_t launch_merge(const AttnArgs &a, int num_sms, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Few pairs have many states each (their keys are split further): eight
    // warps a pair while the pairs leave most of the card empty, else one.  Decode rows of
    // 8 KV heads behind 4096 keys, eight against one, both launches: 128 pairs 20.6 and 25.8
    // us, 384 35.0 and 36.7, 512 40.8 and 40.5, 640 50.5 and 47.9, 1024 68.6 and 61.7.
    const long long pairs = (long long)a.T * a.Hkv;
    if (pairs <= 4LL * num_sms) {
        cfg.gridDim = dim3((unsigned)pairs);
        return cudaLaunchKernelEx(&cfg, shared_merge_kernel<T, D, G, 8>, a);
    }
    const long long blocks = (pairs + 7) / 8, most = 32LL * num_sms;
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    return cudaLaunchKernelEx(&cfg, shared_merge_kernel<T, D, G, 1>, a);
}

template <typename T, int D>
cudaError_t merge_any(const AttnArgs &a, int num_sms, cudaStream_t st) {
    switch (a.G) {
        case 1: return launch_merge<T, D, 1>(a, num_sms, st);
        case 2: return launch_merge<T, D, 2>(a, num_sms, st);
        case 4: return launch_merge<T, D, 4>(a, num_sms, st);
        case 8: return launch_merge<T, D, 8>(a, num_sms, st);
        default: return cudaErrorInvalidValue;
    }
}

template <int D>
cudaError_t launch_f32(const AttnArgs &a, int num_sms, cudaStream_t st) {
    const size_t smem = sizeof(Smem<D>);
    auto kern = shared_attn_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.workers);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) return e;
    return merge_any<float, D>(a, num_sms, st);
}

template <int D>
cudaError_t launch_bf16(const AttnArgs &a, int num_sms, cudaStream_t st) {
    cudaError_t e = launch_attn_tc(a, num_sms, st);
    if (e != cudaSuccess) return e;
    return merge_any<__nv_bfloat16, D>(a, num_sms, st);
}

}  // namespace shared
}  // namespace asmk

size_t asm_shared_attention_ws_bytes(int T, int Hq, int d, int num_sms) {
    using namespace asmk::shared;
    return ws_layout(T, Hq, d, num_sms < kMaxWorkers ? num_sms : kMaxWorkers).total;
}

cudaError_t asm_shared_attention_launch(const void *q, const void *k_pages, const void *v_pages, int n_pages,
                                        int page_size, const int32_t *table, int max_pages,
                                        const int32_t *prefix_table, int max_prefix_pages, const void *plan, int R,
                                        int NG, int T, int Hq, int Hkv, int d, float scale, asm_dtype dt, void *out,
                                        float *lse_out, void *ws, int num_sms, cudaStream_t st) {
    using namespace asmk;
    using namespace asmk::shared;
    const PlanLayout pl = plan_layout(R, NG, T, Hq / Hkv);
    const int workers = num_sms < kMaxWorkers ? num_sms : kMaxWorkers;
    const WsLayout wl = ws_layout(T, Hq, d, workers);
    const char *p = static_cast<const char *>(plan);
    char *w = static_cast<char *>(ws);
    AttnArgs a{};
    a.hdr = reinterpret_cast<const Header *>(p);
    a.first = reinterpret_cast<const int *>(p + pl.first);
    a.tiles = reinterpret_cast<const Tile *>(p + pl.tiles);
    a.tok = reinterpret_cast<const int2 *>(p + pl.tok);
    a.q = q; a.k_pages = k_pages; a.v_pages = v_pages;
    a.table = table; a.prefix_table = prefix_table;
    a.out = out; a.lse = lse_out;
    a.R = R; a.NG = NG; a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.d = d;
    a.S = page_size;
    while ((1 << a.shift) < page_size) ++a.shift;
    while ((1 << a.gshift) < a.G) ++a.gshift;
    a.n_pages = n_pages; a.max_pages = max_pages; a.max_prefix_pages = max_prefix_pages;
    a.workers = workers;
    a.sl2 = scale * kLog2e;
    a.ws_ml = reinterpret_cast<float2 *>(w + wl.ml);
    a.ws_o = reinterpret_cast<float *>(w + wl.o);
    a.ws_err = reinterpret_cast<int *>(w);
    if (dt == ASM_BF16) return d == 128 ? launch_bf16<128>(a, num_sms, st) : launch_bf16<64>(a, num_sms, st);
    return d == 128 ? launch_f32<128>(a, num_sms, st) : launch_f32<64>(a, num_sms, st);
}
