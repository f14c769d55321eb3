// shared.cuh -- the plan of a shared-prefix attention call: what the plan
// kernel writes and the attention and merge kernels read.
//
// A tile is a run of tokens with the G query heads of a KV head: at most 128
// query rows, or 256 when the run is longer than that.  Its keys are those of
// a prefix, or a row's own, or both: a row with more than 128 query rows fills
// its tiles by itself, so they hold the prefix and the local keys and no
// state has to be joined; the shorter rows between such rows share prefix
// tiles, and each has a tile of its local keys.  A unit is 128 prefix or 128
// local keys of one tile for one KV head.  The (tile, KV head) pairs, tile by
// tile and head by head, are laid end to end by their cost and the line is
// cut into equal ranges, one per worker (CTA): the work is balanced whatever
// the lengths are, and a long key list is split as far as there are workers.
// A worker takes the units that begin in its range; a pair whose units fall
// to several workers leaves one partial state per worker (a segment), which
// the merge kernel joins.
#pragma once

#include <stdint.h>

namespace asmk {
namespace shared {

constexpr int kUnitKeys = 128;
constexpr int kTileRows = 128, kDualRows = 256;
constexpr int kMaxRows = 4096;   // batch rows (requests), and prefix groups
constexpr int kMagic = 0x53504c4e;

struct __align__(16) Tile {
    int tok0, ntok;    // tokens of the batch
    int group, row;    // prefix and row of its keys
    int pre_keys;      // prefix keys (they come first)
    int keys;          // local keys the last token sees
    int base;          // local keys before the token tok0 itself
    int units;         // ceil(pre_keys / kUnitKeys) + ceil(keys / kUnitKeys)
    int direct;        // the tile holds all keys of its tokens
    int cap;           // segments at most, per KV head
    long long cost0;   // cost of all tiles before, for one KV head
    long long row0;    // partial rows of all tiles before
    int pad[2];
};

// Cost of a tile for one KV head: cost_head for its queries and its epilogue,
// then so much per unit.  A 256-row unit costs about twice a 128-row one (the
// tensor cores against HBM): with 5 in place of 4 the chunks of six rows take
// 850 us against 700, with 3 720.  A short tile's head is worth one unit: with
// 1.5, 600 rows of one local unit behind a shared prefix take 180 us against
// 159, with half a unit 16 decode rows 47.7 against 45.6.
// A range is at least as long as the dearest unit of the plan, so that it holds
// the start of a unit of every pair it crosses.
__host__ __device__ inline int cost_unit(int rows) { return rows > kTileRows ? 4 : 2; }
__host__ __device__ inline int cost_head(int rows) { return rows > kTileRows ? 4 : 2; }
__host__ __device__ inline long long cost_of(int rows, int units) {
    return units > 0 ? cost_head(rows) + (long long)cost_unit(rows) * units : 0;
}

struct Header {
    int magic, R, NG, T, Hq, Hkv, page_size, max_pages, max_prefix_pages, workers, ntiles;
    int range;         // cost per worker
    long long W;       // cost of all (tile, KV head) pairs
    double inv_range;
};

// Byte offsets in the plan buffer.
constexpr int kMaxWorkers = 1024;
struct PlanLayout {
    size_t first, tiles, tok, total;  // first: the tile each worker's range begins in
};
inline __host__ __device__ long long max_tiles(int R, int NG, int T, int G) {
    const long long rows = R < T ? R : T, groups = NG < T ? NG : T;
    const long long full = ((long long)T * G + kDualRows - 1) / kDualRows;
    // a local and a prefix tile for every row and group with tokens, the full
    // ones, and the runs that rows of more than 128 query rows cut off
    return rows + groups + 4 * full;
}
inline __host__ __device__ PlanLayout plan_layout(int R, int NG, int T, int G) {
    PlanLayout p;
    p.first = 256;
    p.tiles = p.first + sizeof(int) * kMaxWorkers;
    p.tok = (p.tiles + sizeof(Tile) * (size_t)max_tiles(R, NG, T, G) + 255) & ~(size_t)255;
    p.total = (p.tok + sizeof(int2) * (size_t)T + 255) & ~(size_t)255;
    return p;
}

// Partial rows: every (tile, KV head) pair has at most 2 + cost / range
// segments of its rows, and the cost / range sum to at most the workers.
inline __host__ __device__ long long max_partial_rows(int T, int Hq, int workers) {
    return 4LL * T * Hq + (long long)(workers + 1) * kDualRows;
}
struct WsLayout {
    size_t ml, o, total;
};
inline __host__ __device__ WsLayout ws_layout(int T, int Hq, int d, int workers) {
    WsLayout w;
    const size_t rows = (size_t)max_partial_rows(T, Hq, workers);
    w.ml = 256;  // word 0: device-side error code
    w.o = (w.ml + sizeof(float2) * rows + 255) & ~(size_t)255;
    w.total = (w.o + sizeof(float) * rows * d + 255) & ~(size_t)255;
    return w;
}

// What one call of the attention reads and writes.
struct AttnArgs {
    const Header *hdr;
    const int *first;         // [workers]
    const Tile *tiles;
    const int2 *tok;          // [T] (the tile with its local keys, its prefix tile), -1 for none
    const void *q;            // [T][Hq][d]
    const void *k_pages, *v_pages;  // [n_pages][Hkv][S][d]
    const int *table;         // [R][max_pages]
    const int *prefix_table;  // [NG][max_prefix_pages]
    void *out;                // [T][Hq][d]
    float *lse;               // [T][Hq] or null
    int R, NG, T, Hq, Hkv, G, gshift, d, S, shift, n_pages, max_pages, max_prefix_pages, workers;
    float sl2;                // softmax scale * log2(e)
    float2 *ws_ml;            // partial (max, sum), base-2 logits
    float *ws_o;              // partial unnormalised outputs
    int *ws_err;
};

// Does the plan belong to this call?
__device__ __forceinline__ bool plan_ok(const AttnArgs &a, const Header &h) {
    return h.magic == kMagic && h.R == a.R && h.NG == a.NG && h.T == a.T && h.Hq == a.Hq && h.Hkv == a.Hkv &&
           h.page_size == a.S && h.workers == a.workers && h.max_pages == a.max_pages && h.max_prefix_pages == a.max_prefix_pages;
}

__device__ __forceinline__ int div_range(long long c, const Header &h) {
    int q = (int)((double)c * h.inv_range);   // off by one at most: c < 2^53
    if ((long long)q * h.range > c) --q;
    else if ((long long)(q + 1) * h.range <= c) ++q;
    return q;
}
// Worker that has the unit k of a pair whose cost begins at c0.
__device__ __forceinline__ int worker_of(long long c0, int rows, int k, const Header &h) {
    return div_range(c0 + cost_head(rows) + (long long)cost_unit(rows) * k, h);
}
// Segments of a pair.
__device__ __forceinline__ int segments(long long c0, int rows, int units, const Header &h) {
    return units > 0 ? worker_of(c0, rows, units - 1, h) - worker_of(c0, rows, 0, h) + 1 : 0;
}

// Partial states: the statistics of a segment's rows follow one another; its
// outputs are stored 4 columns of all rows at a time, so that threads that
// hold one row each write together: element (row, column).
__device__ __forceinline__ size_t partial_at(long long first_row, int rows, int row, int col, int D) {
    return (size_t)first_row * D + ((size_t)(col >> 2) * rows + row) * 4 + (col & 3);
}

// The segments of one worker, in order; the next tile's descriptor is read ahead.
struct Seg {
    Tile t;
    int g, k, n;          // KV head, first unit, units
    bool direct;          // no other segment or tile has keys of these tokens
    long long prow;       // first partial row
};
struct Walk {
    long long c, end;     // cost: where the current pair begins, where the range ends
    int w, i, g, last, Hkv, G;
    const Header &h;
    const Tile *tiles;
    Tile t, next;
    __device__ Walk(const AttnArgs &a, const Header &h_, int w_)
        : w(w_), g(0), last(h_.ntiles - 1), Hkv(a.Hkv), G(a.G), h(h_), tiles(a.tiles) {
        const long long begin = (long long)w * h.range;
        end = min(h.W, begin + h.range);
        c = end;
        i = 0;
        if (begin < end) {
            i = a.first[w];
            t = tiles[i];
            next = tiles[min(i + 1, last)];
            const long long per = cost_of(t.ntok * G, t.units);
            g = (int)((begin - t.cost0 * Hkv) / per);
            c = t.cost0 * Hkv + g * per;
        }
    }
    __device__ bool step(Seg &s) {
        while (c < end) {
            const int rows = t.ntok * G, cu = cost_unit(rows);
            const long long u0 = c + cost_head(rows), lo = (long long)w * h.range;
            // units that begin within [lo, end)
            const int k0 = lo <= u0 ? 0 : (int)((lo - u0 + cu - 1) / cu);
            const int k1 = t.units == 0 || end <= u0 ? 0 : (int)min((long long)t.units, (end - u0 + cu - 1) / cu);
            const bool some = k0 < k1;
            if (some) {
                s.t = t;
                s.g = g;
                s.k = k0;
                s.n = k1 - k0;
                s.direct = t.direct && s.n == t.units;
                s.prow = t.row0 + ((long long)g * t.cap + (w - worker_of(c, rows, 0, h))) * rows;
            }
            c += cost_of(rows, t.units);
            if (++g == Hkv) {
                g = 0;
                ++i;
                t = next;
                next = tiles[min(i + 1, last)];
            }
            if (some) return true;
        }
        return false;
    }
};

// shared_attn_tc.cu: the tensor-core kernel (bf16)
cudaError_t launch_attn_tc(const AttnArgs &a, int num_sms, cudaStream_t st);

}  // namespace shared
}  // namespace asmk
