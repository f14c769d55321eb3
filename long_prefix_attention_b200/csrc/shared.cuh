// shared.cuh -- the plan of a shared-prefix attention call: what the plan
// kernel writes and the attention and merge kernels read.
//
// A tile is a run of tokens of one row (its local pages) or of one prefix
// group (the group's prefix pages) with the G query heads of a KV head: at
// most 128 query rows, or 256 when the run is longer than that.  A unit is
// 128 keys of one tile for one KV head.  The units of all (tile, KV head)
// pairs form one sequence, tile by tile and head by head, which is cut into
// equal ranges, one per worker (CTA): the work is balanced whatever the
// lengths are, and a long key list is split as far as there are workers.  A
// pair whose units fall to several workers leaves one partial state per
// worker (a segment); the merge kernel joins them.
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
    int owner;         // row (local) or group (prefix)
    int flags;         // kLocal / kDirect
    int keys;          // keys the tile's last token sees
    int base;          // local: keys that lie before the token tok0 itself
    int units;         // ceil(keys / kUnitKeys)
    int cap;           // segments at most, per KV head
    long long unit0;   // units of all tiles before, times one KV head
    long long row0;    // partial rows of all tiles before
};
constexpr int kLocal = 1;   // keys in the row's own pages, causal
constexpr int kDirect = 2;  // the tile holds all keys of its tokens

struct Header {
    int magic, R, NG, T, Hq, Hkv, page_size, max_pages, max_prefix_pages, workers, ntiles;
    int upc;           // units per worker
    long long W;       // units of all (tile, KV head) pairs
};

// Byte offsets in the plan buffer.
constexpr int kMaxWorkers = 1024;
struct PlanLayout {
    size_t first, tiles, tok, total;  // first: the tile each worker's range begins in
};
inline __host__ __device__ long long max_tiles(int R, int NG, int T, int G) {
    const long long rows = R < T ? R : T, groups = NG < T ? NG : T;
    const long long full = ((long long)T * G + kDualRows - 1) / kDualRows;
    return rows + groups + 2 * full;
}
inline __host__ __device__ PlanLayout plan_layout(int R, int NG, int T, int G) {
    PlanLayout p;
    p.first = 256;
    p.tiles = p.first + sizeof(int) * kMaxWorkers;
    p.tok = (p.tiles + sizeof(Tile) * (size_t)max_tiles(R, NG, T, G) + 255) & ~(size_t)255;
    p.total = (p.tok + sizeof(int2) * (size_t)T + 255) & ~(size_t)255;
    return p;
}

// Partial rows: every (tile, KV head) pair has at most 2 + units / upc
// segments of its rows, and the units / upc sum to at most the workers.
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
    const int2 *tok;          // [T] (local tile, prefix tile) of a token, -1 for none
    const void *q;            // [T][Hq][d]
    const void *k_pages, *v_pages;  // [n_pages][Hkv][S][d]
    const int *table;         // [R][max_pages]
    const int *prefix_table;  // [NG][max_prefix_pages]
    void *out;                // [T][Hq][d]
    float *lse;               // [T][Hq] or null
    int R, NG, T, Hq, Hkv, G, d, S, shift, n_pages, max_pages, max_prefix_pages, workers;
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

// Segments of the units [c0, c0 + n) when every worker has upc.
__device__ __forceinline__ int segments(long long c0, int n, int upc) {
    return n > 0 ? (int)((c0 + n - 1) / upc - c0 / upc) + 1 : 0;
}

// First partial row of segment s of (tile, g).
__device__ __forceinline__ long long partial_row(const Tile &t, int G, int g, int s) {
    return t.row0 + ((long long)g * t.cap + s) * ((long long)t.ntok * G);
}

// shared_attn_tc.cu: the tensor-core kernel (bf16)
cudaError_t launch_attn_tc(const AttnArgs &a, int num_sms, cudaStream_t st);

}  // namespace shared
}  // namespace asmk
