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
// 64 keys at a time in shared memory as fp32; 16 x 16 threads, each with MR
// query rows and 4 keys of S = Q K^T, then MR rows and D / 16 columns of
// O += P V.  The 16 threads of a row share a half-warp, which keeps its
// statistics and its row of P to itself.  MR = 1 (16 rows a block) serves
// decode tiles, MR = 4 (64 rows) longer ones.

constexpr int kThreads = 256;
constexpr int kKB = 64;  // keys per block step

template <int D>
struct Smem {
    static constexpr int LD = D + 4, LP = kKB + 4;
    float q[64 * LD], k[kKB * LD], v[kKB * LD], p[64 * LP];
    int page[kKB];
};

template <int D>
__device__ void load_keys(const AttnArgs &a, const Seg &s, int k1, int kb, const int *list, Smem<D> &sm) {
    constexpr int LD = Smem<D>::LD, C = D / 4;
    const int tid = threadIdx.x;
    if (tid < kKB) {
        const int key = kb + tid;
        int id = -1;
        if (key < k1) {
            id = list[key >> a.shift];
            if (id < 0 || id >= a.n_pages) {
                id = -1;
                atomicExch(a.ws_err, (int)ASM_ERR_INVALID_ARG);
            }
        }
        sm.page[tid] = id;
    }
    __syncthreads();
    for (int i = tid; i < kKB * C; i += kThreads) {
        const int r = i / C, c = (i - r * C) * 4, id = sm.page[r];
        float kx[4] = {0.f, 0.f, 0.f, 0.f}, vx[4] = {0.f, 0.f, 0.f, 0.f};
        if (id >= 0) {
            const long long off = ((((long long)id * a.Hkv + s.g) << a.shift) + ((kb + r) & (a.S - 1))) * D + c;
            load_vec<float, 4>(static_cast<const float *>(a.k_pages) + off, kx);
            load_vec<float, 4>(static_cast<const float *>(a.v_pages) + off, vx);
        }
        store_vec<float, 4>(sm.k + r * LD + c, kx);
        store_vec<float, 4>(sm.v + r * LD + c, vx);
    }
    __syncthreads();
}

template <int D, int MR>
__device__ void run_segment(const AttnArgs &a, const Seg &s, Smem<D> &sm) {
    constexpr int LD = Smem<D>::LD, LP = Smem<D>::LP, BR = 16 * MR, NC = D / 64;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int rows = s.t.ntok * a.G;
    const int k0 = s.k * kUnitKeys, k1 = min((s.k + s.n) * kUnitKeys, s.t.keys);  // keys of the segment
    const bool local = s.t.flags & kLocal;
    const int *list = local ? a.table + (size_t)s.t.owner * a.max_pages
                            : a.prefix_table + (size_t)s.t.owner * a.max_prefix_pages;
    for (int rb = 0; rb < rows; rb += BR) {
        __syncthreads();  // the previous rows' queries have been used
        for (int i = tid; i < BR * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4, rr = rb + r;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (rr < rows)
                load_vec<float, 4>(static_cast<const float *>(a.q) +
                                       ((size_t)(s.t.tok0 + rr / a.G) * a.Hq + s.g * a.G + rr % a.G) * D + c, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= a.sl2;
            store_vec<float, 4>(sm.q + r * LD + c, x);
        }
        float m[MR], l[MR], o[MR][4 * NC];
        int lim[MR];  // keys the row sees
#pragma unroll
        for (int i = 0; i < MR; ++i) {
            m[i] = kNegInf;
            l[i] = 0.f;
            const int rr = rb + ty * MR + i;
            lim[i] = min(k1, local ? s.t.base + rr / a.G + 1 : s.t.keys);
#pragma unroll
            for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.f;
        }
        for (int kb = k0; kb < k1; kb += kKB) {
            __syncthreads();
            load_keys<D>(a, s, k1, kb, list, sm);
            float sc[MR][4];
#pragma unroll
            for (int i = 0; i < MR; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 kx[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kx[j] = *reinterpret_cast<const float4 *>(sm.k + (tx + 16 * j) * LD + d);
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    const float4 qx = *reinterpret_cast<const float4 *>(sm.q + (ty * MR + i) * LD + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float t = sc[i][j];
                        t = fmaf(qx.x, kx[j].x, t); t = fmaf(qx.y, kx[j].y, t);
                        t = fmaf(qx.z, kx[j].z, t); t = fmaf(qx.w, kx[j].w, t);
                        sc[i][j] = t;
                    }
                }
            }
            bool masked = false;
#pragma unroll
            for (int i = 0; i < MR; ++i) {
                float mx = kNegInf;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (kb + tx + 16 * j >= lim[i]) sc[i][j] = kNegInf;
                    mx = fmaxf(mx, sc[i][j]);
                }
                masked |= kb + kKB > lim[i];
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
                    sm.p[(ty * MR + i) * LP + tx + 16 * j] = p;
                }
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
                l[i] = l[i] * al + ps;
#pragma unroll
                for (int c = 0; c < 4 * NC; ++c) o[i][c] *= al;
            }
            __syncwarp();
            const int kn = min(kKB, k1 - kb);
            for (int k = 0; k < kn; k += 4) {
                float4 px[MR];
#pragma unroll
                for (int i = 0; i < MR; ++i) px[i] = *reinterpret_cast<const float4 *>(sm.p + (ty * MR + i) * LP + k);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float4 vx = *reinterpret_cast<const float4 *>(sm.v + (k + e) * LD + 64 * c + 4 * tx);
#pragma unroll
                        for (int i = 0; i < MR; ++i) {
                            const float p = e == 0 ? px[i].x : e == 1 ? px[i].y : e == 2 ? px[i].z : px[i].w;
                            // a weight of 0 at a key the row does not see must not meet its value
                            if (masked && p == 0.f) continue;
                            o[i][4 * c] = fmaf(p, vx.x, o[i][4 * c]);
                            o[i][4 * c + 1] = fmaf(p, vx.y, o[i][4 * c + 1]);
                            o[i][4 * c + 2] = fmaf(p, vx.z, o[i][4 * c + 2]);
                            o[i][4 * c + 3] = fmaf(p, vx.w, o[i][4 * c + 3]);
                        }
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < MR; ++i) {
            const int rr = rb + ty * MR + i;
            if (rr >= rows) continue;
            if (s.direct) {
                const size_t th = (size_t)(s.t.tok0 + rr / a.G) * a.Hq + s.g * a.G + rr % a.G;
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = o[i][4 * c + e] * inv;
                    store_vec<float, 4>(static_cast<float *>(a.out) + th * D + 64 * c + 4 * tx, x);
                }
                if (a.lse && tx == 0) a.lse[th] = l[i] == 0.f ? kNegInf : (m[i] + log2f(l[i])) * kLn2;
            } else {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    *reinterpret_cast<float4 *>(a.ws_o + partial_at(s.prow, rows, rr, 64 * c + 4 * tx, D)) =
                        make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
                if (tx == 0) a.ws_ml[s.prow + rr] = make_float2(m[i], l[i]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
shared_attn_kernel(const AttnArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
    const Header h = *a.hdr;
    if (!plan_ok(a, h)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.ws_err, (int)ASM_ERR_INVALID_ARG);
        return;
    }
    Walk walk(a, h, blockIdx.x);  // one block per worker
    Seg s;
    while (walk.step(s)) {
        if (s.t.ntok * a.G <= 16) run_segment<D, 1>(a, s, sm);
        else run_segment<D, 4>(a, s, sm);
    }
}

// ------------------------------------------------------------------ merge --
//
// NW warps per (token, query head): each reads its share of the partial
// states (32 statistics at a time, then their rows, eight in flight), and the
// warps meet in shared memory.  Pairs whose only state was written as output
// already are skipped; pairs without any key get (0, -inf).

constexpr int kMergeThreads = 256;

template <typename T, int D, int NW>
__global__ void __launch_bounds__(kMergeThreads)
shared_merge_kernel(const AttnArgs a) {
    constexpr int E = D / 32, PPB = kMergeThreads / 32 / NW;
    __shared__ float so[NW > 1 ? PPB * NW : 1][D];
    __shared__ float2 sml[NW > 1 ? PPB * NW : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % NW, pb = warp / NW;
    const Header h = *a.hdr;
    if (!plan_ok(a, h)) return;
    const long long pairs = (long long)a.T * a.Hq;
    for (long long base = (long long)blockIdx.x * PPB; base < pairs; base += (long long)gridDim.x * PPB) {
        const long long pr = base + pb;
        bool live = pr < pairs;
        const int t = live ? (int)(pr / a.Hq) : 0, hq = live ? (int)(pr - (long long)t * a.Hq) : 0;
        const int2 tt = live ? a.tok[t] : make_int2(-1, -1);
        live = live && tt.x >= 0;  // tokens outside every row are left as they are
        const int g = hq / a.G, hh = hq - g * a.G;
        long long row[2] = {0, 0};            // first partial row of the pair's segments
        int rows[2] = {0, 0}, at[2] = {0, 0}, n[2] = {0, 0};
        if (live) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = x == 0 ? tt.x : tt.y;
                if (i < 0) continue;
                const Tile tl = a.tiles[i];
                rows[x] = tl.ntok * a.G;
                n[x] = segments(tl.cost0 * a.Hkv + g * cost_of(rows[x], tl.units), rows[x], tl.units, h.range);
                if (x == 0 && n[x] == 1 && (tl.flags & kDirect)) live = false;  // already written
                row[x] = tl.row0 + (long long)g * tl.cap * rows[x];
                at[x] = (t - tl.tok0) * a.G + hh;
            }
        }
        const int tot = live ? n[0] + n[1] : 0;
        float m = kNegInf, l = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int e0 = sub * 32; e0 < tot; e0 += NW * 32) {
            const int e = e0 + lane;
            const long long r = e < n[0] ? row[0] + (long long)e * rows[0] + at[0]
                                         : row[1] + (long long)(e - n[0]) * rows[1] + at[1];
            const float2 ml = e < tot ? __ldcg(a.ws_ml + r) : make_float2(kNegInf, 0.f);
            const float mn = fmaxf(m, warp_max(ml.x)), ref = mn == kNegInf ? 0.f : mn;
            const float al = exp2f(m - ref), w = ml.y == 0.f ? 0.f : exp2f(ml.x - ref);
            m = mn;
            l = l * al + warp_sum(w * ml.y);
#pragma unroll
            for (int d = 0; d < E; ++d) o[d] *= al;
            const int cnt = min(32, tot - e0);
            for (int j0 = 0; j0 < cnt; j0 += 8) {
                float v[8][E];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int ee = e0 + min(j0 + j, cnt - 1);
                    const float *p = a.ws_o + (ee < n[0] ? partial_at(row[0] + (long long)ee * rows[0], rows[0], at[0], lane * E, D)
                                                         : partial_at(row[1] + (long long)(ee - n[0]) * rows[1], rows[1], at[1],
                                                                      lane * E, D));
#pragma unroll
                    for (int d = 0; d < E; ++d) v[j][d] = __ldcg(p + d);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float wj = j0 + j < cnt ? __shfl_sync(0xffffffffu, w, (j0 + j) & 31) : 0.f;
                    if (wj == 0.f) continue;  // an empty state's row may hold anything
#pragma unroll
                    for (int d = 0; d < E; ++d) o[d] = fmaf(wj, v[j][d], o[d]);
                }
            }
        }
        if (NW > 1) {
            __syncthreads();
            if (lane == 0) sml[warp] = make_float2(m, l);
#pragma unroll
            for (int d = 0; d < E; ++d) so[warp][lane * E + d] = o[d];
            __syncthreads();
            if (sub == 0) {
                float mm = m;
                for (int w = 1; w < NW; ++w) mm = fmaxf(mm, sml[warp + w].x);
                const float ref = mm == kNegInf ? 0.f : mm, al = exp2f(m - ref);
                l *= al;
#pragma unroll
                for (int d = 0; d < E; ++d) o[d] *= al;
                for (int w = 1; w < NW; ++w) {
                    const float x = exp2f(sml[warp + w].x - ref);
                    l = fmaf(x, sml[warp + w].y, l);
#pragma unroll
                    for (int d = 0; d < E; ++d) o[d] = fmaf(x, so[warp + w][lane * E + d], o[d]);
                }
                m = mm;
            }
        }
        if (live && sub == 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int d = 0; d < E; ++d) o[d] *= inv;
            store_vec<T, E>(static_cast<T *>(a.out) + (size_t)pr * D + lane * E, o);
            if (a.lse && lane == 0) a.lse[pr] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
        }
    }
}

template <typename T, int D>
cudaError_t launch_merge(const AttnArgs &a, int num_sms, cudaStream_t st) {
    // few pairs have many partial states each (the work is split further):
    // eight warps a pair while the pairs do not fill the card, else one
    const long long pairs = (long long)a.T * a.Hq;
    if (pairs <= 8LL * num_sms) {
        shared_merge_kernel<T, D, 8><<<(unsigned)pairs, kMergeThreads, 0, st>>>(a);
    } else {
        const long long blocks = (pairs + 7) / 8, most = 16LL * num_sms;
        shared_merge_kernel<T, D, 1><<<(unsigned)(blocks < most ? blocks : most), kMergeThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_f32(const AttnArgs &a, int num_sms, cudaStream_t st) {
    const size_t smem = sizeof(Smem<D>);
    auto kern = shared_attn_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<a.workers, kThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_merge<float, D>(a, num_sms, st);
}

template <int D>
cudaError_t launch_bf16(const AttnArgs &a, int num_sms, cudaStream_t st) {
    cudaError_t e = launch_attn_tc(a, num_sms, st);
    if (e != cudaSuccess) return e;
    return launch_merge<__nv_bfloat16, D>(a, num_sms, st);
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
    a.n_pages = n_pages; a.max_pages = max_pages; a.max_prefix_pages = max_prefix_pages;
    a.workers = workers;
    a.sl2 = scale * kLog2e;
    a.ws_ml = reinterpret_cast<float2 *>(w + wl.ml);
    a.ws_o = reinterpret_cast<float *>(w + wl.o);
    a.ws_err = reinterpret_cast<int *>(w);
    if (dt == ASM_BF16) return d == 128 ? launch_bf16<128>(a, num_sms, st) : launch_bf16<64>(a, num_sms, st);
    return d == 128 ? launch_f32<128>(a, num_sms, st) : launch_f32<64>(a, num_sms, st);
}
