// shared_attn_tc.cu -- attention of a ragged batch over shared prefixes and
// the rows' own pages on the tensor cores (bf16 storage).
//
// One CTA per SM takes one worker's range of the plan's line and works segment
// by segment: S = Q K^T and O += P V on tcgen05.mma, fp32 accumulators in
// tensor memory, the softmax in registers with a running maximum that is only
// raised when it grows by more than 8 (base 2; numerator and denominator share
// it, so a stale maximum is exact).  Warp roles:
//   warp 8     producer: a segment's queries (TMA over [T][Hkv][G][d]), then
//              the page ids of a unit (one lane per page, read one unit ahead)
//              and one TMA box per page and 64 columns, K and V tiles in turn
//              through a ring that runs on across segments;
//   warp 9, 10 one lane each issues the products of stream 0 and of stream 1
//              (an issuer's waits and address arithmetic run under the other
//              stream's products; one issuer for both left the tensor pipe
//              idle half of the time); warp 9 holds the tensor memory;
//   warps 0-3  softmax stream 0, warps 4-7 softmax stream 1: a thread per
//              query row (tensor-memory lane).  In units that end a tile's
//              keys they also clear the places of V behind the last key, and
//              the non-finite values of keys that some of the tile's rows do
//              not see (0 times a NaN would reach those rows); the epilogue
//              adds them back to the rows that do.
// The work is a sequence of steps that alternate between the streams, across
// segments too.  A tile of more than 128 rows gives each stream 128 of its
// rows, so a unit is two steps (one read of K and V serves 256 rows); in a
// smaller one a unit is one step, and a segment of two or more units leaves a
// state in both streams, which its epilogue joins.  A stream's next scores are
// issued right behind its P V, across segments too, so one stream's softmax
// and epilogue run under the other's products.
// Decode tiles with a few rows waste most of a product, which costs no time:
// a 128-key unit takes the tensor core 0.6 us and 64 KB take an SM's share of
// HBM 1.5 us.  It does cost power: 64 rows behind 32768 keys, call after call,
// run at the power limit.  Up to 32 rows are laid out four times, each warp of a
// stream takes a quarter of the keys, and the rows between them are zeros in Q
// and in P (64 rows: 357 us at first and 432 for many calls, with the rows that
// follow in memory 384 and 460).  Above that, warps without rows skip the softmax;
// 33 to 64 rows laid out twice gained 2% there but cost the shorter tiles 14%.
// Measured (hd 128, 8 KV heads, 32 heads; a burst of ten calls, and call after call
// for a second, when the power limit lowers the clock): 16 rows behind 16384 keys 46 us
// both ways, of which HBM streams 28; 64 rows with 8191 own keys behind 32768 366 us, 95%
// of the copy rate, and 415 to 435 (82%); 6 chunks of 257 to 511 tokens behind 16384
// keys 694 us, 870 TFLOP/s, and 770 (781), the tensor pipe active 41% of the time.
// Tensor memory columns: O_0 [0,128) O_1 [128,256) S_0 / P_0 [256,384)
// S_1 / P_1 [384,512).  A stream's products complete in issue order, so S_x(next)
// (issued after P_x V) overwrites P_x only once it was read, and its completion
// means that O_x is stable.  Every wait is bounded; after a timeout a warp waits no
// more and arrives at no mbarrier, so that the others run out too, and the error word
// is set.  The named barriers have no limit, so the softmax warps pass the same ones
// whatever has timed out: they follow the list of segments to its end, which a producer
// that gives up publishes as well.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "launch.h"
#include "shared.cuh"
#include "umma.cuh"

namespace asmk {
namespace shared {
namespace tc {

using namespace umma;

constexpr int kThreads = 352;
constexpr int kProducer = 8, kIssuer = 9;
constexpr int kSoftmax = 256;       // threads of the two softmax streams
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.f;
constexpr int kBox = 128 * 128;     // 128 rows x 64 columns of bf16
constexpr int kFixUnits = 4;        // units of a tile that some of its rows see in part
constexpr int kFix = 8;             // one stream is at most RING / 2 + 1 segments ahead of the other
constexpr int kSmallRows = 32;      // query rows of a short tile
constexpr int kBoxRows = 8;         // query rows of its boxes: a swizzle atom, at least one token
constexpr int kQuarterBoxes = kSmallRows / kBoxRows;

template <int D>
struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = HALVES * kBox;
    static constexpr int RING = D == 128 ? 4 : 8;   // K or V tiles in flight
};

// A segment as the producer hands it to the other warps; n = 0 ends the list.
// Sixteen places are more than the producer can be ahead of the slowest reader:
// it enters a segment only when the ring has taken all of the one before, so
// at most RING / 2 + 3 segments are in use at a time.
constexpr int kSegs = 16;
// Limits a softmax warp waits for the next segment: a producer in trouble takes one
// to give up and publish the end, and a warp that left before would leave the others at
// a barrier.
constexpr int kSegWaits = 64;
struct __align__(16) SegDesc {
    int tok0, rows, base, keys;      // first token, query rows; as in Tile
    int g, k, n, pre_keys;           // KV head, first unit, units; as in Tile
    long long prow;                  // first partial row
    int row, masked;                 // row; first unit that some of the tile's rows see in part
    int direct, group, pad[2];       // group: of the prefix keys
};

template <int D>
struct Smem {
    unsigned char q[2][Cfg<D>::TILE];
    unsigned char kv[Cfg<D>::RING][Cfg<D>::TILE];
    SegDesc seg[kSegs];
    float2 ml[2][128];                 // a row's (max, sum) in each stream
    float4 wl[8][kSmallRows];          // short tiles: a warp's (factor, share of the sum, maximum) of a row
    alignas(16) float ex[8][512];      // short tiles: the warps' outputs on their way to one sum
    uint32_t kinds[2][D / 8];          // short tiles: non-finite values among 8 columns: +inf, -inf << 8, NaN << 16
    alignas(16) uint32_t fix[kFix][kFixUnits][4];  // per segment (modulo kFix): keys whose V was cleared, from the first masked unit on
    uint64_t kv_full[Cfg<D>::RING], kv_empty[Cfg<D>::RING];
    uint64_t seg_full[kSegs], turn[2][Cfg<D>::RING / 2], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2];
    uint32_t tmem_base;
};
// read and written 16 bytes at a time
static_assert(offsetof(Smem<64>, ex) % 16 == 0 && offsetof(Smem<64>, fix) % 16 == 0, "alignment");
static_assert(offsetof(Smem<128>, ex) % 16 == 0 && offsetof(Smem<128>, fix) % 16 == 0, "alignment");

struct Maps {
    CUtensorMap k, v, q, q_small;
};

__device__ __forceinline__ void set_error(int *err, asm_status s) { atomicExch(err, (int)s); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// 2^t for two arguments on the FMA pipe: t = n + f, f in [-1/2, 1/2], 2^f by a
// polynomial of degree 5 fitted to it there (relative error 1.6e-7), 2^n
// added into the exponent.  t is clamped at -125, and so are a NaN and -infinity: the
// caller mends the sums of rows whose maximum is not finite.
__device__ __forceinline__ uint64_t exp2_poly_x2(uint64_t t2) {
    const uint64_t t = pack_f32x2(fmaxf(lo_f32(t2), -125.f), fmaxf(hi_f32(t2), -125.f));
    const uint64_t y = add_f32x2(t, pack_f32x2(12582912.f, 12582912.f));   // 1.5 * 2^23: n in the low bits
    const uint64_t n = add_f32x2(y, pack_f32x2(-12582912.f, -12582912.f));
    const uint64_t f = fma_f32x2(n, pack_f32x2(-1.f, -1.f), t);
    uint64_t p = fma_f32x2(pack_f32x2(0.001327647245f, 0.001327647245f), f, pack_f32x2(0.009675540961f, 0.009675540961f));
    p = fma_f32x2(p, f, pack_f32x2(0.05550713092f, 0.05550713092f));
    p = fma_f32x2(p, f, pack_f32x2(0.2402212024f, 0.2402212024f));
    p = fma_f32x2(p, f, pack_f32x2(0.693146944f, 0.693146944f));
    p = fma_f32x2(p, f, pack_f32x2(1.000000119f, 1.000000119f));
    return pack_u32x2((uint32_t)p + ((uint32_t)y << 23), (uint32_t)(p >> 32) + ((uint32_t)(y >> 32) << 23));
}

// Barrier of the softmax warps: both streams, or one.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory"); }
__device__ __forceinline__ void stream_sync(int x) {
    if (x == 0) asm volatile("bar.sync 2, 128;" ::: "memory");
    else asm volatile("bar.sync 3, 128;" ::: "memory");
}

// The same, with the or of a condition of all threads.
__device__ __forceinline__ bool softmax_any(bool c) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) : "r"((uint32_t)c), "n"(kSoftmax) : "memory");
    return r != 0;
}
__device__ __forceinline__ bool stream_any(int x, bool c) {
    uint32_t r;
    if (x == 0)
        asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, 2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                     : "=r"(r) : "r"((uint32_t)c) : "memory");
    else
        asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, 3, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                     : "=r"(r) : "r"((uint32_t)c) : "memory");
    return r != 0;
}

// Which of 8 bf16 values are +inf, -inf (<< 8) and NaN (<< 16).
__device__ __forceinline__ uint32_t non_finite(const uint4 &x) {
    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = (i & 1) ? y[i >> 1] >> 16 : y[i >> 1] & 0xffffu;
        if ((h & 0x7f80u) == 0x7f80u) r |= 1u << (i + ((h & 0x7fu) ? 16 : (h & 0x8000u) ? 8 : 0));
    }
    return r;
}

__device__ __forceinline__ int units_of(int keys) { return (keys + kUnitKeys - 1) / kUnitKeys; }

// First unit (of the tile) that holds a local key some row of the tile does
// not see, since it is a later token; the tile's units if there is none.
__device__ __forceinline__ int first_masked_unit(const Tile &t) {
    return min(units_of(t.pre_keys) + max(t.base + 1, 0) / kUnitKeys, t.units);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The largest of 32 scores; a NaN is the largest.
__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
    float m11[11];
#pragma unroll
    for (int i = 0; i < 10; ++i)
        m11[i] = max3_nan(__uint_as_float(v[3 * i]), __uint_as_float(v[3 * i + 1]), __uint_as_float(v[3 * i + 2]));
    m11[10] = max_nan(__uint_as_float(v[30]), __uint_as_float(v[31]));
    return max3_nan(max3_nan(max3_nan(m11[0], m11[1], m11[2]), max3_nan(m11[3], m11[4], m11[5]),
                             max3_nan(m11[6], m11[7], m11[8])), m11[9], m11[10]);
}

// A warp's rows of O times f (a lane's own).
template <int D>
__device__ __forceinline__ void scale_outputs(uint32_t t_o, float f) {
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(t_o + (uint32_t)c0, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st32(t_o + (uint32_t)c0, o);
    }
}

// Scores of places from n on: -inf.
__device__ __forceinline__ void mask32(uint32_t (&v)[32], int n) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i >= n) v[i] = 0xff800000u;
}

// Clears the places [r1, 128) of a V tile, and the non-finite values of keys
// [r0, r1), whose bits are set in `fix`; 128 threads.
template <int D>
__device__ __forceinline__ void clean_values(unsigned char *v, int r0, int r1, int thread, uint32_t *fix) {
    constexpr int CH = D / 8;
    for (int c = thread; c < (r1 - r0) * CH; c += 128) {
        const int r = r0 + c / CH, cc = c % CH;
        uint4 *p = reinterpret_cast<uint4 *>(v + (cc >> 3) * kBox + swz128(r, cc & 7));
        const uint4 x = *p;
        // bf16 exponents of all ones, in the halves of four words
        uint32_t y[4] = {x.x, x.y, x.z, x.w};
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (y[i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
            const uint32_t hi = (y[i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
            bad |= (lo | hi) != 0u;
            y[i] &= ~(lo | hi);
        }
        if (bad) {
            *p = make_uint4(y[0], y[1], y[2], y[3]);
            atomicOr(&fix[r >> 5], 1u << (r & 31));
        }
    }
    for (int c = thread; c < (kUnitKeys - r1) * CH; c += 128) {
        const int r = r1 + c / CH, cc = c % CH;
        *reinterpret_cast<uint4 *>(v + (cc >> 3) * kBox + swz128(r, cc & 7)) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
shared_attn_tc_kernel(const __grid_constant__ Maps maps, const AttnArgs a) {
    using C = Cfg<D>;
    constexpr int RING = C::RING;
    extern __shared__ unsigned char smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], 2);   // one arrival of each issuer, or two of one
        }
        for (int i = 0; i < kSegs; ++i) mbar_init(&sm.seg_full[i], 1);
        for (int i = 0; i < RING / 2; ++i) {
            mbar_init(&sm.turn[0][i], 1);
            mbar_init(&sm.turn[1][i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sm.q_full[x], 1);
            mbar_init(&sm.q_empty[x], 2);
            mbar_init(&sm.s_full[x], 1);
            mbar_init(&sm.p_full[x], 128);
            mbar_init(&sm.o_full[x], 1);
        }
        fence_mbar_init();
    }
    if (tid >= 32 && tid < 36) {   // the tensor maps' first use should not wait for them
        const CUtensorMap *m = tid == 32 ? &maps.k : tid == 33 ? &maps.v : tid == 34 ? &maps.q : &maps.q_small;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (tid < kFix * kFixUnits * 4) (&sm.fix[0][0][0])[tid] = 0;
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&sm.tmem_base)), "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    const Header h = *a.hdr;
    const bool fits = plan_ok(a, h);
    if (!fits && blockIdx.x == 0 && tid == 0) set_error(a.ws_err, ASM_ERR_INVALID_ARG);
    bool ok = true;
    // the lanes of a warp agree on a timeout, so that none leaves the others in a collective
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity)); };

    if (!fits) {
        // nothing to do
    } else if (warp == kProducer) {
        // ------------------------------------------------------ producer
        const int rows = min(a.S, kUnitKeys), boxes = kUnitKeys / rows;  // keys and boxes per page of a unit
        const int tok_x = kTileRows / a.G;                               // tokens of 128 query rows
        Walk walk(a, h, blockIdx.x);
        uint32_t segs = 0;
        auto publish = [&](const Seg &s, bool some) {
            if (lane == 0) {
                SegDesc d{};
                if (some) {
                    d.tok0 = s.t.tok0; d.rows = s.t.ntok * a.G; d.base = s.t.base; d.keys = s.t.keys;
                    d.g = s.g; d.k = s.k; d.n = s.n; d.pre_keys = s.t.pre_keys;
                    d.prow = s.prow; d.row = s.t.row; d.group = s.t.group; d.masked = first_masked_unit(s.t); d.direct = s.direct;
                }
                sm.seg[segs % kSegs] = d;
                mbar_arrive(&sm.seg_full[segs % kSegs]);
            }
            __syncwarp();
            ++segs;
        };
        Seg s, ns;                 // the list is one segment ahead of the loads
        bool some = walk.step(ns);
        publish(ns, some);
        uint32_t n = 0;            // ring items so far
        uint32_t qn[2] = {0, 0};   // fills of the query buffers
        int qb = 0;                // buffer of the next small tile
        int dirty[2] = {kQuarterBoxes, kQuarterBoxes};   // boxes of a quarter that may hold other than zeros
        while (ok && some) {
            s = ns;
            some = walk.step(ns);
            publish(ns, some);
            const int qrows = s.t.ntok * a.G;
            const bool dual = qrows > kTileRows, small = qrows <= kSmallRows;
            for (int x = 0; x < 2; ++x) {
                if (!dual && x != qb) continue;
                if (qn[x] > 0) wait(&sm.q_empty[x], (qn[x] - 1) & 1);
                if (!ok) break;
                ++qn[x];
                // a short tile: the same boxes in every quarter of the lanes, then zeros over
                // what earlier tiles left (a load from behind the last token gives zeros)
                const int live = small ? (qrows + kBoxRows - 1) / kBoxRows : kQuarterBoxes;
                const int loads = max(live, dirty[x]);
                dirty[x] = live;
                if (lane == 0) mbar_arrive_expect_tx(&sm.q_full[x], (uint32_t)(small ? C::TILE / kQuarterBoxes * loads : C::TILE));
                __syncwarp();
                if (small) {
                    const int b = lane % kQuarterBoxes;
                    if (lane < kTileRows / kBoxRows && b < loads) {
#pragma unroll
                        for (int hf = 0; hf < C::HALVES; ++hf)
                            tma_load_4d(sm.q[x] + hf * kBox + lane * kBoxRows * 128, &maps.q_small, 64 * hf, 0, s.g,
                                        b < live ? s.t.tok0 + b * (kBoxRows / a.G) : a.T, &sm.q_full[x]);
                    }
                } else if (lane == 0) {
#pragma unroll
                    for (int hf = 0; hf < C::HALVES; ++hf)
                        tma_load_4d(sm.q[x] + hf * kBox, &maps.q, 64 * hf, 0, s.g,
                                    s.t.tok0 + (dual ? x * tok_x : 0), &sm.q_full[x]);
                }
                __syncwarp();
            }
            if (!dual) qb ^= 1;
            const int *pre_list = a.prefix_table + (size_t)s.t.group * a.max_prefix_pages;
            const int *own_list = a.table + (size_t)s.t.row * a.max_pages;
            const int pu = units_of(s.t.pre_keys);
            auto page = [&](int unit, bool &used) {     // this lane's page of a unit
                const bool pre = unit < pu;
                const int key = (pre ? unit : unit - pu) * kUnitKeys + lane * rows;
                used = lane < boxes && unit < s.k + s.n && key < (pre ? s.t.pre_keys : s.t.keys);
                return used ? (pre ? pre_list : own_list)[key >> a.shift] : -1;
            };
            bool next_used;
            int ahead = page(s.k, next_used);
            for (int j = s.k; j < s.k + s.n && ok; ++j) {
                const int id = ahead;
                const bool used = next_used;
                ahead = page(j + 1, next_used);
                const bool bad = used && (id < 0 || id >= a.n_pages);
                if (bad) set_error(a.ws_err, ASM_ERR_INVALID_ARG);
                // past the cache (zero fill) for places behind the last key and bad ids
                const int c2 = used && !bad ? id * a.Hkv + s.g : a.n_pages * a.Hkv;
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = n % RING;
                    if (n >= RING) wait(&sm.kv_empty[slot], ((n / RING) - 1) & 1);
                    if (!ok) break;
                    ++n;
                    if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full[slot], C::TILE);
                    __syncwarp();
                    if (lane < boxes) {
#pragma unroll
                        for (int hf = 0; hf < C::HALVES; ++hf)
                            tma_load_3d(sm.kv[slot] + hf * kBox + lane * rows * 128, kv ? &maps.v : &maps.k, 64 * hf, 0, c2,
                                        &sm.kv_full[slot]);
                    }
                }
            }
        }
        if (some) publish(ns, false);     // given up: the list ends here
        // every copy that was issued has landed before the CTA may end
        for (uint32_t i = n > RING ? n - RING : 0; i < n; ++i)
            if (!mbar_wait(&sm.kv_full[i % RING], (i / RING) & 1)) ok = false;
        for (int x = 0; x < 2; ++x)
            if (qn[x] > 0 && !mbar_wait(&sm.q_full[x], (qn[x] - 1) & 1)) ok = false;
    } else if (warp >= kIssuer) {
        // ------------------------------------- product issuers (one lane each)
        if (lane == 0) {
            const int x = warp - kIssuer;
            const uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kUnitKeys >> 3) << 17) |
                                     ((uint32_t)(128 >> 4) << 24);
            const uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                     ((uint32_t)(128 >> 4) << 24);
            // addresses within a descriptor add up: all of shared memory lies below 2^18
            const uint64_t q_desc = desc_k_sw128(smem_addr(sm.q[0])), k_desc = desc_k_sw128(smem_addr(sm.kv[0])),
                           v_desc = desc_mn_sw128(smem_addr(sm.kv[0]), kBox);
            const uint32_t t_o = tmem + (uint32_t)(x * 128), t_s = t_o + 256;
            auto wait1 = [&](uint64_t *bar, uint32_t parity) { ok = ok && mbar_wait_lone(bar, parity); };
            // this stream's steps: unit j of a segment of n, every dj-th
            int n = 0, j = 0, dj = 1, qb = 0, next_qb = 0;
            uint32_t segs = 0, step = 0, unit0 = 0;     // before the segment
            uint32_t q_bits = 0;                        // phases of the query buffers
            uint32_t turn_bits = 0;
            bool dual = false;
            auto next = [&]() {      // false behind the last step
                j += dj;
                while (j >= n) {
                    step += (uint32_t)(dual ? 2 * n : n);
                    unit0 += (uint32_t)n;
                    wait1(&sm.seg_full[segs % kSegs], (segs / kSegs) & 1);
                    const SegDesc &d = sm.seg[segs++ % kSegs];
                    n = ok ? d.n : 0;
                    if (n == 0) return false;
                    dual = d.rows > kTileRows;
                    dj = dual ? 1 : 2;
                    j = dual ? 0 : (x ^ (int)(step & 1));
                    // both streams follow the fills of both query buffers
                    if (dual) {
                        qb = x;
                    } else {
                        qb = next_qb;
                        next_qb ^= 1;
                    }
                    if (j >= n) q_bits ^= 1u << qb;      // a single unit, on the other stream
                    else if (dual) q_bits ^= 1u << (x ^ 1);
                }
                return true;
            };
            auto issue_s = [&]() {
                // A tall tile's streams take their scores in turns, each when the other has
                // found its maximum: left alone, they fall into step and the tensor cores
                // idle during both softmaxes (prompt chunks: 805 against 715 us).
                if (dual && (x == 1 || j > 0)) {
                    const int i = (unit0 + (uint32_t)j) % (RING / 2);
                    wait1(&sm.turn[x][i], (turn_bits >> i) & 1);
                    turn_bits ^= 1u << i;
                }
                if (j < dj) {        // the stream's first step of the segment
                    wait1(&sm.q_full[qb], (q_bits >> qb) & 1);
                    q_bits ^= 1u << qb;
                }
                const uint32_t item = 2 * (unit0 + (uint32_t)j), slot = item % RING;
                wait1(&sm.kv_full[slot], (item / RING) & 1);
                if (!ok) return;
                tc_fence_after();
                const uint64_t qd = q_desc + (uint32_t)qb * (C::TILE >> 4), kd = k_desc + slot * (C::TILE >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    constexpr uint32_t box = kBox >> 4;
                    const uint32_t off = (uint32_t)(kk >> 2) * box + (uint32_t)(kk & 3) * 2;
                    umma_bf16(t_s, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                }
                umma_commit(&sm.s_full[x]);
                // a unit of a small tile has one issuer: it arrives for both
                umma_commit(&sm.kv_empty[slot]);
                if (!dual) mbar_arrive(&sm.kv_empty[slot]);
                if (j + dj >= n) {
                    umma_commit(&sm.q_empty[qb]);
                    if (dual || n == 1) mbar_arrive(&sm.q_empty[qb]);
                }
            };
            uint32_t p_bit = 0;      // phase of the stream's P tiles
            bool more = next();
            if (more) issue_s();
            while (ok && more) {
                const uint32_t item = 2 * (unit0 + (uint32_t)j) + 1, slot = item % RING;
                wait1(&sm.kv_full[slot], (item / RING) & 1);
                wait1(&sm.p_full[x], p_bit);
                p_bit ^= 1;
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = v_desc + slot * (C::TILE >> 4);
                const bool fresh = j < dj;
#pragma unroll
                for (int kk = 0; kk < kUnitKeys / 16; ++kk)
                    // 16 keys a step: 8 tensor-memory columns of P, 16 rows of V
                    umma_bf16_ts(t_o, t_s + (uint32_t)(kk * 8), vd + (uint32_t)(kk * (2048 >> 4)), idesc_o,
                                 (!fresh || kk > 0) ? 1u : 0u);
                if (j + dj >= n) umma_commit(&sm.o_full[x]);
                umma_commit(&sm.kv_empty[slot]);
                if (!dual) mbar_arrive(&sm.kv_empty[slot]);
                more = next();
                if (more) issue_s();
            }
        }
        __syncwarp();
    } else {
        // ----------------------------------------------------- softmax
        const int x = warp >> 2;            // stream
        const int qd = warp & 3;            // tensor-memory lane quarter
        const int row = qd * 32 + lane;     // row within the stream's 128
        const int st = tid & 127;           // thread of the stream
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const uint32_t t_s = tmem + lane_off + 256 + (uint32_t)(x * 128);
        const float sl2 = a.sl2;
        uint32_t sn = 0, on[2] = {0, 0};    // scores taken, outputs finished in each stream
        uint32_t step = 0, unit0 = 0;       // steps and units before this segment
        for (uint32_t seg = 0;; ++seg) {
            // read to its end even after a timeout: the warps meet at barriers
            bool got = false;
            for (int i = 0; i < kSegWaits && !got; ++i)
                got = __all_sync(0xffffffffu, mbar_wait(&sm.seg_full[seg % kSegs], (seg / kSegs) & 1));
            const SegDesc &s = sm.seg[seg % kSegs];
            const int n = got ? s.n : 0;
            ok = ok && got;
            if (n == 0) break;
            const int rows = s.rows, k0 = s.k, keys = s.keys, masked = s.masked;
            const bool dual = rows > kTileRows;
            const int j0 = dual ? 0 : (x ^ (int)(step & 1)), dj = dual ? 1 : 2;   // this stream's units
            const uint32_t item0 = 2 * unit0;
            step += (uint32_t)(dual ? 2 * n : n);
            unit0 += (uint32_t)n;
            if (j0 >= n) {                   // a single unit, on the other stream
                ++on[x ^ 1];
                continue;
            }
            const bool joint = dual || n > 1;             // both streams have steps
            const int pre_keys = s.pre_keys, pu = units_of(pre_keys);
            uint32_t(&fix)[kFixUnits][4] = sm.fix[seg % kFix];
            const bool fixable = masked < k0 + n;
            // V of this stream's unit j as the products may use it
            auto clean = [&](int j) {
                const int unit = k0 + j, key0 = (unit < pu ? unit : unit - pu) * kUnitKeys;
                const int valid = (unit < pu ? pre_keys : keys) - key0;
                if (unit < masked && valid >= kUnitKeys) return;
                const uint32_t item = item0 + 2 * (uint32_t)j + 1;
                wait(&sm.kv_full[item % RING], (item / RING) & 1);
                if (!ok) return;
                const int r0 = unit >= masked ? max(s.base + 1 - key0, 0) : kUnitKeys;
                clean_values<D>(sm.kv[item % RING], r0, min(valid, kUnitKeys), row,
                                fix[min(max(unit - masked, 0), kFixUnits - 1)]);
            };
            auto notes = [&]() {       // were values cleared?
                uint32_t f = 0;
                for (int fu = 0; fixable && fu < kFixUnits; ++fu) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(fix[fu]);
                    f |= w.x | w.y | w.z | w.w;
                }
                return f;
            };
            // the 32 values from column c on that were cleared of keys before `own`: add(i, value)
            auto add_back = [&](int own, int c, auto add) {
#pragma unroll 1
                for (int f = 0; f < kFixUnits * 4; ++f) {
                    uint32_t bits = fix[f >> 2][f & 3];
                    while (bits) {
                        const int key = (masked - pu) * kUnitKeys + 32 * f + __ffs(bits) - 1;
                        bits &= bits - 1;
                        if (key >= own) continue;
                        const int id = a.table[(size_t)s.row * a.max_pages + (key >> a.shift)];
                        if (id < 0 || id >= a.n_pages) continue;
                        const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.v_pages) +
                            ((((long long)id * a.Hkv + s.g) << a.shift) + (key & (a.S - 1))) * D + c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float y = __bfloat162float(vp[i]);
                            if (!(y - y == 0.f)) add(i, y);
                        }
                    }
                }
            };

            if (rows <= kSmallRows) {
                // ------------------------------------------------ short tile
                // The tile's rows lie in every quarter of the lanes, and the warp of a
                // quarter takes 32 of the unit's 128 keys: a softmax of a quarter of
                // the length, with a state of its own.  The weights of the other
                // keys are zeros, so its outputs are those of its keys.
                const bool live = lane < rows;
                const int own = live ? min(s.base + (lane >> a.gshift) + 1, keys) : keys;   // local keys the row sees
                float m_used = kNegInf, l = 0.f;
                for (int j = j0; j < n; j += dj) {
                    wait(&sm.s_full[x], sn & 1);
                    ++sn;
                    tc_fence_after();
                    const int vis = (k0 + j < pu ? pre_keys - (k0 + j) * kUnitKeys
                                                 : own - (k0 + j - pu) * kUnitKeys) - 32 * qd;
                    uint32_t v[32], pk[16];
                    tmem_ld32(t_s + (uint32_t)(32 * qd), v);
                    tmem_wait_ld();
                    if (__any_sync(0xffffffffu, vis < 32)) mask32(v, vis);
                    const float mt = max32(v) * sl2;
                    float alpha = 1.f;
                    if (live && !(mt <= m_used + kRescale)) {
                        alpha = ex2f(m_used - mt);
                        m_used = mt;
                        l *= alpha;
                    }
                    const float ref = !live ? -kNegInf : m_used == kNegInf ? 0.f : m_used;   // other rows: weights of 0
                    const uint64_t sl2x2 = pack_f32x2(sl2, sl2), negm2 = pack_f32x2(-ref, -ref);
                    uint64_t acc[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t t2 = fma_f32x2(pack_u32x2(v[2 * i], v[2 * i + 1]), sl2x2, negm2);
                        const uint64_t p2 = pack_f32x2(ex2f(lo_f32(t2)), ex2f(hi_f32(t2)));
                        acc[i & 1] = add_f32x2(acc[i & 1], p2);
                        pk[i] = pack_bf16(lo_f32(p2), hi_f32(p2));
                    }
                    const uint64_t a01 = add_f32x2(acc[0], acc[1]);
                    l += lo_f32(a01) + hi_f32(a01);
                    const uint32_t zero[16] = {0};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c != qd) tmem_st16(t_s + (uint32_t)(16 * c), zero);
                    tmem_st16(t_s + (uint32_t)(16 * qd), pk);
                    if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) scale_outputs<D>(tmem + lane_off + (uint32_t)(x * 128), alpha);
                    tmem_wait_st();
                    clean(j);
                    tc_fence_before();
                    if (ok) mbar_arrive(&sm.p_full[x]);
                }
                // the states of the quarters, of both streams if both have some, become one
                sm.ml[x][row] = make_float2(m_used, l);
                wait(&sm.o_full[x], on[x] & 1);
                if (joint) wait(&sm.o_full[x ^ 1], on[x ^ 1] & 1);
                ++on[x];
                if (joint) ++on[x ^ 1];
                auto meet = [&]() {
                    if (joint) softmax_sync();
                    else stream_sync(x);
                };
                meet();
                tc_fence_after();
                const uint32_t fixed = notes();
                const int w_lo = joint ? 0 : 4 * x, w_hi = joint ? 8 : 4 * x + 4;   // warps with states
                // columns per pass, and this thread's row and four columns of a pass
                int csh = 4;
                while ((1 << csh) < D && (rows << csh) <= 256) ++csh;
                const int cols = 1 << csh, it = joint ? tid : st, ir = it >> (csh - 2), ic = (it & (cols / 4 - 1)) * 4;
                float w_own;
                {
                    float ms[8], mo = kNegInf;
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        ms[w] = w >= w_lo && w < w_hi ? sm.ml[w >> 2][(w & 3) * 32 + lane].x : kNegInf;
#pragma unroll
                    for (int w = 0; w < 8; ++w) mo = max_nan(mo, ms[w]);
                    w_own = ex2f(m_used - (mo == kNegInf ? 0.f : mo));
                    sm.wl[warp][lane] = make_float4(w_own, w_own * l, mo, 0.f);   // factor, share of the sum, maximum
                }
                const int itk = ir >> a.gshift;
                const size_t th = (size_t)(s.tok0 + itk) * a.Hq + (size_t)s.g * a.G + (ir & (a.G - 1));
                float mi = kNegInf, li = 0.f, inv = 1.f;
                bool searched = false;
                uint32_t *kinds = sm.kinds[joint ? 0 : x];
                // The kinds of non-finite values that all rows see, by all threads, 16 bytes of a
                // key each: 1 to 2 us per unit, so that 5 * 10^7 keys of one segment stay within
                // the limit of the other warps' waits (a thread per row and column, key after
                // key: 0.27 us per key and pass).
                auto search = [&]() {
                    constexpr int CH = D / 8;
                    const int lots = (joint ? kSoftmax : 128) / CH, cc = it % CH, at = it / CH;
                    const int *pre_list = a.prefix_table + (size_t)s.group * a.max_prefix_pages;
                    const int *own_list = a.table + (size_t)s.row * a.max_pages;
                    if (it < CH) kinds[it] = 0;
                    meet();
                    uint32_t found = 0;
#pragma unroll 1
                    for (int u = k0; u < k0 + n; ++u) {
                        const int *list = u < pu ? pre_list : own_list;
                        const int key0 = (u < pu ? u : u - pu) * kUnitKeys;
                        const int end = min(u < pu ? pre_keys : min(s.base + 1, keys), key0 + kUnitKeys);
#pragma unroll 1
                        for (int key = key0 + at; key < end; key += 4 * lots) {
                            uint4 y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int k = key + e * lots, id = k < end ? list[k >> a.shift] : -1;
                                y[e] = make_uint4(0, 0, 0, 0);
                                if (id >= 0 && id < a.n_pages)
                                    y[e] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v_pages) +
                                        ((((long long)id * a.Hkv + s.g) << a.shift) + (k & (a.S - 1))) * D + 8 * cc);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) found |= non_finite(y[e]);
                        }
                    }
                    if (found) atomicOr(&kinds[cc], found);
                    meet();
                };
                // o[i]: the sum of the non-finite values, if there are any, of column c + i over
                // the segment's keys that a row with `own` local keys sees
                auto sum_non_finite = [&](int own, int c, float (&o)[4]) {
                    const uint32_t w = kinds[c >> 3] >> (c & 7);
                    float t[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        t[i] = ((w >> i) & 1u ? -kNegInf : 0.f) + ((w >> (8 + i)) & 1u ? kNegInf : 0.f) +
                               ((w >> (16 + i)) & 1u ? __int_as_float(0x7fffffff) : 0.f);
#pragma unroll 1
                    for (int f = 0; fixed && f < kFixUnits * 4; ++f) {
                        uint32_t bits = fix[f >> 2][f & 3];
                        while (bits) {
                            const int key = (masked - pu) * kUnitKeys + 32 * f + __ffs(bits) - 1;
                            bits &= bits - 1;
                            if (key >= own) continue;
                            const int id = a.table[(size_t)s.row * a.max_pages + (key >> a.shift)];
                            if (id < 0 || id >= a.n_pages) continue;
                            float y[4];
                            load_vec<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(a.v_pages) +
                                ((((long long)id * a.Hkv + s.g) << a.shift) + (key & (a.S - 1))) * D + c, y);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (!(y[i] - y[i] == 0.f)) t[i] += y[i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t[i] != 0.f) o[i] = t[i];   // a NaN is not 0 either
                };
                for (int c0 = 0; c0 < D; c0 += cols) {
#pragma unroll 1
                    for (int c = c0; c < c0 + cols; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(tmem + lane_off + (uint32_t)(x * 128 + c), o);
                        tmem_wait_ld();
                        if (live) {
                            float *e = &sm.ex[warp][(lane << csh) + c - c0];
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = m_used == kNegInf ? 0u : __float_as_uint(__uint_as_float(o[i]) * w_own);
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<uint4 *>(e + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                    meet();
                    float o[4] = {0.f, 0.f, 0.f, 0.f};
                    bool odd = false;
                    if (ir < rows) {
                        if (c0 == 0) {
#pragma unroll
                            for (int w = 0; w < 8; ++w)
                                if (w >= w_lo && w < w_hi) {
                                    const float4 y = sm.wl[w][ir];
                                    li += y.y;
                                    mi = y.z;
                                }
                            if (s.direct) inv = li == 0.f ? 0.f : 1.f / li;
                        }
#pragma unroll
                        for (int w = 0; w < 8; ++w)
                            if (w >= w_lo && w < w_hi) {
                                const float4 y = *reinterpret_cast<const float4 *>(&sm.ex[w][(ir << csh) + ic]);
                                o[0] += y.x; o[1] += y.y; o[2] += y.z; o[3] += y.w;
                            }
                        // Non-finite values: those cleared, and those that met the zeros of other
                        // quarters (0 times infinity is not a number).  The sum of the ones
                        // the row sees is the result; a NaN among the scores is in l already.
                        const float bad = (o[0] - o[0]) + (o[1] - o[1]) + (o[2] - o[2]) + (o[3] - o[3]);
                        odd = (fixed || bad != 0.f) && li == li;
                    }
                    // all have read the warps' outputs
                    if (joint ? softmax_any(odd) : stream_any(x, odd)) {
                        if (!searched) search();
                        searched = true;
                        if (odd) sum_non_finite(min(s.base + itk + 1, keys), c0 + ic, o);
                        meet();
                    }
                    if (ir < rows) {
                        if (s.direct) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[i] *= inv;
                            store_vec<__nv_bfloat16, 4>(static_cast<__nv_bfloat16 *>(a.out) + th * D + c0 + ic, o);
                        } else {
                            *reinterpret_cast<float4 *>(a.ws_o + partial_at(s.prow, rows, ir, c0 + ic, D)) =
                                make_float4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                if (ir < rows && ic == 0) {
                    if (!s.direct) a.ws_ml[s.prow + ir] = make_float2(mi, li);
                    else if (a.lse) a.lse[th] = li == 0.f ? kNegInf : (mi + log2f(li)) * kLn2;
                }
                tc_fence_before();
                if (fixed && it < kFixUnits * 4) fix[it >> 2][it & 3] = 0;
                continue;
            }

            const int r = dual ? x * 128 + row : row;       // row of the tile
            const bool live = r < rows;
            const bool warp_live = (dual ? x * 128 : 0) + qd * 32 < rows;
            const int tk = r >> a.gshift;
            const int own = live ? min(s.base + tk + 1, keys) : keys;   // local keys the row sees
            float m_used = kNegInf, l = 0.f;
            for (int j = j0; j < n; j += dj) {
                wait(&sm.s_full[x], sn & 1);
                ++sn;
                tc_fence_after();
                if (warp_live) {
                    const int vis = k0 + j < pu ? pre_keys - (k0 + j) * kUnitKeys
                                                : own - (k0 + j - pu) * kUnitKeys;   // keys of this unit the row sees
                    const bool part = __any_sync(0xffffffffu, vis < kUnitKeys);
                    // pass 1: the largest score
                    float mraw = kNegInf;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32(t_s + (uint32_t)(32 * c), v);
                        tmem_wait_ld();
                        if (part) mask32(v, vis - 32 * c);
                        mraw = max_nan(mraw, max32(v));
                    }
                    const float mt = mraw * sl2;
                    float alpha = 1.f;
                    if (live && !(mt <= m_used + kRescale)) {   // a NaN passes, and stays in the sum
                        alpha = ex2f(m_used - mt);
                        m_used = mt;
                        l *= alpha;
                    }
                    // tensor-memory access is warp-wide: rows that keep their maximum scale by 1
                    if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f))
                        scale_outputs<D>(tmem + lane_off + (uint32_t)(x * 128), alpha);
                    // pass 2: p = 2^(s scale log2(e) - m), rounded to bf16 for the product
                    // with V (the sum keeps fp32); P goes over columns of S already read
                    const float ref = m_used == kNegInf ? 0.f : m_used;
                    const uint64_t sl2x2 = pack_f32x2(sl2, sl2), negm2 = pack_f32x2(-ref, -ref);
                    uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (c == 0 && dual && st == 0 && ok && (x == 0 || j + 1 < n))
                            mbar_arrive(&sm.turn[x ^ 1][(item0 / 2 + (uint32_t)(j + x)) % (RING / 2)]);
                        uint32_t v[32], pk[16];
                        tmem_ld32(t_s + (uint32_t)(32 * c), v);
                        tmem_wait_ld();
                        if (part) {
                            mask32(v, vis - 32 * c);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const uint64_t t2 = fma_f32x2(pack_u32x2(v[2 * i], v[2 * i + 1]), sl2x2, negm2);
                                const uint64_t p2 = pack_f32x2(ex2f(lo_f32(t2)), ex2f(hi_f32(t2)));
                                acc[i & 3] = add_f32x2(acc[i & 3], p2);
                                pk[i] = pack_bf16(lo_f32(p2), hi_f32(p2));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const uint64_t t2 = fma_f32x2(pack_u32x2(v[2 * i], v[2 * i + 1]), sl2x2, negm2);
                                uint64_t p2;
                                if ((i & 3) == 3) p2 = exp2_poly_x2(t2);
                                else p2 = pack_f32x2(ex2f(lo_f32(t2)), ex2f(hi_f32(t2)));
                                acc[i & 3] = add_f32x2(acc[i & 3], p2);
                                pk[i] = pack_bf16(lo_f32(p2), hi_f32(p2));
                            }
                        }
                        tmem_st16(t_s + (uint32_t)(16 * c), pk);
                    }
                    const uint64_t a01 = add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3]));
                    l += lo_f32(a01) + hi_f32(a01);
                    tmem_wait_st();
                }
                clean(j);
                tc_fence_before();
                if (ok) mbar_arrive(&sm.p_full[x]);
            }
            // ------------------------------------------------------ epilogue
            // The polynomial's clamp has lost the NaN of a score of +inf (inf - inf) and the
            // zero weights of rows that saw scores of -inf alone.  A vote per unit that keeps
            // such rows off the polynomial costs tall tiles 2.8%.
            if (m_used == -kNegInf) l = m_used - m_used;
            if (m_used == kNegInf && l == l) l = 0.f;   // a NaN maximum gives way to a later unit's -inf, its sum stays
            if (joint) {
                sm.ml[x][row] = make_float2(m_used, l);
                wait(&sm.o_full[0], on[0] & 1);
                wait(&sm.o_full[1], on[1] & 1);
                ++on[0];
                ++on[1];
                softmax_sync();
            } else {
                wait(&sm.o_full[x], on[x] & 1);
                ++on[x];
                if (fixable) stream_sync(x);
            }
            tc_fence_after();
            const uint32_t fixed = notes();
            if (warp_live) {
                // the states of a small tile's streams, joined
                float w0 = 1.f, w1 = 0.f, m = m_used;
                const bool two = joint && !dual;
                bool none0 = false, none1 = false;
                if (two) {
                    const float2 s0 = sm.ml[0][row], s1 = sm.ml[1][row];
                    none0 = s0.x == kNegInf;
                    none1 = s1.x == kNegInf;
                    m = max_nan(s0.x, s1.x);
                    const float ref = m == kNegInf ? 0.f : m;
                    w0 = ex2f(s0.x - ref);
                    w1 = ex2f(s1.x - ref);
                    l = w0 * s0.y + w1 * s1.y;
                }
                const size_t th = (size_t)(s.tok0 + tk) * a.Hq + (size_t)s.g * a.G + (r & (a.G - 1));
                const float inv = s.direct ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                // of two streams, each writes half of the columns
                const int c_lo = two ? x * (D / 2) : 0, c_hi = two ? c_lo + D / 2 : D;
                const uint32_t t_o = tmem + lane_off + (two ? 0u : (uint32_t)(x * 128));
#pragma unroll 1
                for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + (uint32_t)c0, o);
                    if (two) {
                        uint32_t o1[32];
                        tmem_ld32(t_o + 128u + (uint32_t)c0, o1);
                        tmem_wait_ld();
                        // a stream that saw no key of the row holds no value for it
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float u0 = none0 ? 0.f : __uint_as_float(o[i]) * w0;
                            o[i] = __float_as_uint(none1 ? u0 : fmaf(__uint_as_float(o1[i]), w1, u0));
                        }
                    } else {
                        tmem_wait_ld();
                    }
                    // non-finite values of keys that only some rows see: back into the rows that do
                    if (fixed && live)
                        add_back(own, c0, [&](int i, float y) {
                            o[i] = __float_as_uint(__uint_as_float(o[i]) + y);
                        });
                    if (live) {
                        if (s.direct) {
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + th * D + c0;
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                uint32_t pk[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    pk[e] = pack_bf16(__uint_as_float(o[i + 2 * e]) * inv,
                                                      __uint_as_float(o[i + 2 * e + 1]) * inv);
                                *reinterpret_cast<uint4 *>(dst + i) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<uint4 *>(a.ws_o + partial_at(s.prow, rows, r, c0 + i, D)) =
                                    make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                }
                if (live && (!two || x == 0)) {
                    if (!s.direct) a.ws_ml[s.prow + r] = make_float2(m, l);
                    else if (a.lse) a.lse[th] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
                }
            }
            tc_fence_before();
            // the other stream's outputs and statistics have been read
            if (joint) softmax_sync();
            if (fixed) {
                if (!joint) stream_sync(x);
                if (row < kFixUnits * 4) fix[row >> 2][row & 3] = 0;
            }
        }
    }
    if (!ok && lane == 0) set_error(a.ws_err, ASM_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

}  // namespace tc
}  // namespace shared

bool make_map_3d(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t rows);
bool make_map_qrows(CUtensorMap *m, const void *q, int B, int Hkv, int G, int d, int rows);

namespace shared {

template <int D>
cudaError_t launch_tc(const AttnArgs &a, int num_sms, cudaStream_t st) {
    tc::Maps maps;
    memset(&maps, 0, sizeof(maps));
    const uint64_t heads = (uint64_t)a.n_pages * a.Hkv;
    const uint32_t box = (uint32_t)(a.S < kUnitKeys ? a.S : kUnitKeys);
    if (!make_map_3d(&maps.k, a.k_pages, D, a.S, heads, box) || !make_map_3d(&maps.v, a.v_pages, D, a.S, heads, box) ||
        !make_map_qrows(&maps.q, a.q, a.T, a.Hkv, a.G, D, kTileRows) ||
        !make_map_qrows(&maps.q_small, a.q, a.T, a.Hkv, a.G, D, tc::kBoxRows))
        return cudaErrorInvalidValue;
    auto kern = tc::shared_attn_tc_kernel<D>;
    const size_t smem = sizeof(tc::Smem<D>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.workers);
    cfg.blockDim = dim3(tc::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

cudaError_t launch_attn_tc(const AttnArgs &a, int num_sms, cudaStream_t st) {
    return a.d == 128 ? launch_tc<128>(a, num_sms, st) : launch_tc<64>(a, num_sms, st);
}

}  // namespace shared
}  // namespace asmk
