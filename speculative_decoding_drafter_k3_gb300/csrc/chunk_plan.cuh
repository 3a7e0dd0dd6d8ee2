// chunk_plan.cuh -- how the chunk attention's work is laid out and cut: its
// parameters, the line of items, a CTA's pieces of it, and what pieces leave
// for one another.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_common.cuh"
#include "chunk_cut.h"
#include "k3da.h"

namespace k3da_chunk {

using namespace k3da_cache;

constexpr int kTile = 128;         // keys of a tile: two pages
constexpr int kSlotRows = 128;     // query rows of a slot
// An item's fixed cost (its first loads, its epilogue or fold), and the
// shortest slice, both in keys; below, of the small kernel's items and slices.
// Swept: 64 items x up to 8191 keys, 4 heads, e4m3 39.7 us with 128, 36.5 with
// 512, 35.9 with 768 (but then one token over 2000 10.1 or 12.2 us, by the
// slices, instead of 9.7 to 10.5); ragged prefills 96.4 with 128, 91.4 with 384,
// 94.5 with 1024.
constexpr int kOverhead = 384, kMinSlice = 256;
constexpr int kSmallOverhead = 512, kMinSmallSlice = 512;

struct ChunkParams {
    __nv_bfloat16 *out;
    float *lse;
    const uint8_t *scales;
    const int32_t *page_table;
    const int32_t *ctx_lens;
    const int32_t *cu_seqlens;
    int32_t *status;
    const __nv_bfloat16 *q;
    long long q_stride;
    struct Cut *cuts;
    float2 *part_ml;  // [kCtas][2][part_rows] (m in log2 units, l)
    float *part_o;    // [kCtas][2][part_rows][64]
    long long num_pages;
    int page_stride, R, T, Hq, Hkv;
    int G;    // query heads per kv head
    int tpt;  // tokens of a slot
    int mask;
    int pass;       // which items: kLong, kSmall or kAll
    int part_rows;  // rows of a partial result
    int second;     // the other pass goes before this one
    float scale_log2;
};

// A request whose chunk is this small (query rows of a kv head) is the small
// kernel's, but in calls that are all latency (kAll).
constexpr int kSmallRows = 16;
enum { kLong, kSmall, kAll };

constexpr size_t kCutBytes = 8192;
static_assert(kCtas * sizeof(Cut) <= kCutBytes, "room for the cuts");
// Workspace of a pass whose partial results have `rows` rows.
constexpr size_t part_bytes(int rows) {
    return kCutBytes + static_cast<size_t>(kCtas) * 2 * rows * (sizeof(float2) + kD * sizeof(float));
}
constexpr size_t kWorkspace = part_bytes(2 * kSlotRows) + part_bytes(kSmallRows);

// -------------------------------------------------------------- the line --

struct Plan {
    long long prefix[kMaxRequests + 1];  // where request r's items begin on the line
    long long warp_sum[16];
};

__device__ __forceinline__ int overhead(const ChunkParams &p) { return p.pass == kSmall ? kSmallOverhead : kOverhead; }

// Length of the first `pairs` items of one head: each sees `base` keys (and,
// causal, its own tokens and the ones before) and costs the overhead.
__device__ __forceinline__ long long line_of(const ChunkParams &p, long long base, long long pairs) {
    const long long own = p.mask == K3DA_MASK_CAUSAL ? p.tpt * pairs * (pairs + 1) : 0;  // 2 tpt (1 + 2 + ... + pairs)
    return pairs * (base + overhead(p)) + own;
}

// A request's first row, new and cached tokens, clamped to what the call has
// room for; true when nothing had to be.
struct Request {
    int row, n, ctx;
    __device__ __forceinline__ bool fetch(const ChunkParams &p, int r) {
        const int a = load_here(p.cu_seqlens + r), b = load_here(p.cu_seqlens + r + 1), c = load_here(p.ctx_lens + r);
        const int cap = p.page_stride * kP;
        row = min(max(a, 0), p.T);
        n = min(max(b, row), p.T) - row;
        ctx = min(max(c, 0), cap);
        const bool fits = p.mask == K3DA_MASK_CONTEXT || static_cast<long long>(ctx) + n <= cap;
        return a == row && b == row + n && (n == 0 || (c == ctx && fits));
    }
    // Items of one kv head in this pass.
    __device__ __forceinline__ int pairs(const ChunkParams &p) const {
        const bool small = p.pass != kAll && n <= kSmallRows && n * p.G <= kSmallRows;
        if (n == 0 || small != (p.pass == kSmall)) return 0;
        return small ? 1 : (n + 2 * p.tpt - 1) / (2 * p.tpt);
    }
    // Keys of the line before a causal chunk's own.
    __device__ __forceinline__ long long base(const ChunkParams &p) const {
        return static_cast<long long>(ctx) + (p.mask == K3DA_MASK_FULL ? n : 0);
    }
};

// All threads; syncs.  The first THREADS take two requests each at a time.
// False, and no plan, where the pass has no items.
template <int THREADS>
__device__ __forceinline__ bool build_plan(const ChunkParams &p, Plan *pl, bool report) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (t == 0) pl->prefix[0] = 0;
    long long done = 0;
    for (int r0 = 0; r0 < p.R; r0 += 2 * THREADS) {
        const bool mine = t < THREADS;
        long long cost[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + 2 * t + k;
            if (!mine || r >= p.R) continue;
            Request q;
            if (!q.fetch(p, r) && report && p.status) atomicOr(p.status, K3DA_STATUS_BAD_LENGTH);
            cost[k] = p.Hkv * line_of(p, q.base(p), q.pairs(p));
        }
        long long sum = cost[0] + cost[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long up = __shfl_up_sync(kFull, sum, off);
            if (lane >= off) sum += up;
        }
        if (mine && lane == 31) pl->warp_sum[warp] = sum;
        if (!__syncthreads_or(mine && sum > 0) && p.R <= 2 * THREADS) return false;
        if (mine) {
            long long before = done;
            for (int w = 0; w < warp; ++w) before += pl->warp_sum[w];
            const int r = r0 + 2 * t;
            if (r + 1 <= p.R) pl->prefix[r + 1] = before + sum - cost[1];
            if (r + 2 <= p.R) pl->prefix[r + 2] = before + sum;
        }
        __syncthreads();
        done = pl->prefix[min(r0 + 2 * THREADS, p.R)];
    }
    return done > 0;
}

// A piece: the tiles [t0, t1) of one item that fall into this CTA's slice.
struct Piece {
    int h;
    int tok0;    // the item's first token in the chunk
    int tokens;
    int ctx, n, r;
    int row;     // its first row; -1: no more pieces
    int limit;   // keys its last row sees
    int keys0;   // ... the last row of slot 0
    int nt;      // tiles of the item
    int t0, t1;
    int alt;     // one slot's worth of rows: the slots take the tiles in turn
    int seq;     // number of the piece among those with tiles
    int q;       // where its Q is: slot 0's half of the Q room, and (bits 1, 2) how often
                 // the halves were filled before, mod 2
    int base;    // steps (small kernel: pages) before it
    // The tiles of slot s: from, from + step, ... below end.
    __device__ __forceinline__ int from(int s) const { return alt ? t0 + s : t0; }
    __device__ __forceinline__ int step() const { return alt ? 2 : 1; }
    __device__ __forceinline__ int end(int s) const {
        const int keys = alt || s == 1 ? limit : keys0;
        return keys <= 0 ? 0 : min(t1, (keys - 1) / kTile + 1);
    }
    // The step of slot s's tile t: tile by tile, slot 0 first.
    __device__ __forceinline__ int step_of(int s, int t) const {
        const int d = t - t0;
        if (alt) return base + d;
        return base + d + (s == 0 ? d : min(d + 1, max(end(0) - t0, 0)));
    }
    __device__ __forceinline__ int steps() const { return t1 - t0 + (alt ? 0 : max(end(0) - t0, 0)); }
};

// Keys that the chunk's token i sees.
__device__ __forceinline__ int keys_seen(const ChunkParams &p, int ctx, int n, int i) {
    const long long c = p.mask == K3DA_MASK_CAUSAL ? static_cast<long long>(ctx) + i + 1
                        : p.mask == K3DA_MASK_FULL ? static_cast<long long>(ctx) + n
                                                   : ctx;
    const int cap = p.page_stride * kP;
    return c < cap ? static_cast<int>(c) : cap;
}

// The CTA's pieces, in order (the scheduler's).
struct Walk {
    long long lo, hi;         // the slice
    long long share;          // floor(total / slices)
    int slices, rest_of;      // ... and what is left
    long long at;             // where the next item begins
    long long start, length;  // the last item
    int r, h, pair;
    Request q;  // r's

    // Start of slice c: ceil(c * total / slices).
    __device__ __forceinline__ long long slice(int c) const {
        return c * share + (c * rest_of + slices - 1) / slices;
    }
    // (Wide divisions take hundreds of cycles, and nothing is loaded before
    // this is done.)
    __device__ __forceinline__ static long long quotient(long long a, long long b) {
        if ((a | b) >> 31 == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
        return a / b;
    }
    __device__ void begin(const ChunkParams &p, const Plan *pl, int cta) {
        const long long total = pl->prefix[p.R];
        const long long most = p.pass == kSmall ? total / kMinSmallSlice : total / kMinSlice;
        slices = most < 1 ? 1 : most > kCtas ? kCtas : static_cast<int>(most);
        share = quotient(total, slices);
        rest_of = static_cast<int>(total - share * slices);
        lo = hi = at = 0;
        r = h = pair = 0;
        if (cta >= slices || total == 0) return;
        lo = slice(cta);
        hi = slice(cta + 1);
        int a = 0, b = p.R;
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (pl->prefix[mid] <= lo) a = mid;
            else b = mid;
        }
        r = a;
        q.fetch(p, r);
        const long long keys = q.base(p);
        const long long head = line_of(p, keys, q.pairs(p));
        long long rest = lo - pl->prefix[r];
        h = static_cast<int>(quotient(rest, head));
        rest -= h * head;
        int x = 0, y = q.pairs(p);
        while (y - x > 1) {
            const int mid = (x + y) >> 1;
            if (line_of(p, keys, mid) <= rest) x = mid;
            else y = mid;
        }
        pair = x;
        at = pl->prefix[r] + h * head + line_of(p, keys, pair);
    }

    // First tile of an item's part from `offset` (in the item) on.
    __device__ __forceinline__ static int tile_at(const ChunkParams &p, long long offset, int nt) {
        const long long t = (offset - overhead(p) + kTile - 1) / kTile;
        return offset <= overhead(p) ? 0 : t < nt ? static_cast<int>(t) : nt;
    }

    __device__ bool next(const ChunkParams &p, Piece &it) {
        while (at < hi) {
            it.r = r;
            it.h = h;
            it.ctx = q.ctx;
            it.n = q.n;
            it.tok0 = pair * 2 * p.tpt;
            it.tokens = min(2 * p.tpt, it.n - it.tok0);
            it.row = q.row + it.tok0;
            it.alt = it.tokens <= p.tpt;
            it.limit = keys_seen(p, it.ctx, it.n, it.tok0 + it.tokens - 1);
            it.nt = static_cast<int>((static_cast<long long>(it.limit) + kTile - 1) / kTile);
            it.keys0 = keys_seen(p, it.ctx, it.n, it.tok0 + min(p.tpt, it.tokens) - 1);
            start = at;
            const int count = q.pairs(p);
            const long long keys = q.base(p);
            length = line_of(p, keys, pair + 1) - line_of(p, keys, pair);
            it.t0 = lo <= at ? 0 : tile_at(p, lo - at, it.nt);
            it.t1 = hi >= at + length ? it.nt : tile_at(p, hi - at, it.nt);
            at += length;
            if (++pair == count) {
                pair = 0;
                if (++h == p.Hkv) {
                    h = 0;
                    while (++r < p.R) {
                        q.fetch(p, r);
                        if (q.pairs(p) > 0) break;
                    }
                }
            }
            if (it.t0 < it.t1 || (it.nt == 0 && start >= lo)) return true;
        }
        return false;
    }

    // The slice that holds this position of the line.
    __device__ int slice_of(long long pos) const {
        int a = 0, b = slices;
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (slice(mid) <= pos) a = mid;
            else b = mid;
        }
        return a;
    }
};

// What was taken out of a piece's V: for +inf, -inf and NaN and each dim,
// ~piece (24 bits) over the first key that had one, counted from the keys
// every row sees (8 bits: an item has at most 256 tokens).  atomicMin then
// lets a later piece's entries replace an earlier one's: nothing is reset.
struct Records {
    uint32_t first[3][kD];
    int piece;  // the last piece that left something here
    int pad[3];
};

// Byte of 16-byte chunk `chunk` of a 128-byte row in a 128B-swizzled tile.
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// The small kernel (k3da_chunk_small.cu).
int launch_small(const ChunkParams &p, const void *kv_pool, bool quant, cudaStream_t stream);

}  // namespace k3da_chunk
