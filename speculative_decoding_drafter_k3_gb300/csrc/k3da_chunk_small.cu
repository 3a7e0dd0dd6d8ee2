// k3da_chunk_small.cu -- the chunk attention of requests that bring few query
// rows (at most 16 a kv head: decoded tokens, mostly), sm_103a.
//
// Same items, line and cuts as the long chunks' kernel (chunk_plan.cuh), but
// an item is bound by reading its cache, and what 128-row products and the
// widening of codes to bf16 tiles in shared memory cost would be the bound
// instead (64 requests of 8000 e4m3 tokens, 24/4 heads: 144 us there).  Here a
// warp takes a page by itself: 16-row products (mma.sync) with the page's
// fragments straight from where TMA put them, a running maximum, sum and O of
// its own in registers, and no barrier but the page's.  Eight such warps share
// an item's pages; they merge when its piece ends.
//
// Quantised pages stay codes in shared memory: a code is a half-precision
// number as it is (one conversion for two), K's scale multiplies a finished
// score, and V's goes into the weight: w = 2^(s + e - m'), with a running
// maximum m' of s + e beside the maximum m of s that the sum keeps.  Both are
// exponents, so scales of any size meet no range.  q is scaled by a power of
// two into half precision's range (exact but for dims 2^-39 below the row's
// largest).
//
// Rounding: scores, statistics, O and partial results are fp32; weights are
// rounded once (bf16, or half precision for codes), the output once.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

#include "chunk_plan.cuh"
#include "k3da.h"
#include "sm103.cuh"
#include "tensor_maps.h"

namespace k3da_chunk {
namespace {

using namespace sm103;

// Page warps; one more schedules.
constexpr int page_warps(bool quant) { return quant ? 12 : 8; }
constexpr int kRing = 4;     // pieces published ahead
constexpr int kRecords = 8;  // pieces whose non-finite records are alive at once
// Spread of V's exponents up to which one reference exponent serves a piece's
// keys: a weight then is off by 2^-25 of a reference that is at most 2^10
// above the largest, 2^-15 of that, where a half's own rounding is 2^-12.
constexpr int kNear = 10;
constexpr int kORow = kD + 4;  // floats of a row in the merge room (the pad spreads rows over the banks)

template <bool QUANT>
struct Smem {
    // A stage is a page.  A warp loads its
    // pages itself, into stages of its own: K as soon as the scores of the
    // page before are done, V after its product.
    static constexpr int kOwn = 1;  // stages of a warp
    static constexpr int kWarps = page_warps(QUANT);
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kStages = kWarps * kOwn;
    static constexpr int kTileBytes = kP * kD * (QUANT ? 1 : 2);  // K or V
    static constexpr int kStageBytes = QUANT ? 2 * kTileBytes + 256 : 2 * kTileBytes;
    static constexpr int kMerge = kStages * kStageBytes;
    static constexpr int kStats = kMerge + kWarps * kSmallRows * kORow * 4;
    static constexpr int kRec = kStats + kWarps * kSmallRows * 16;
    static constexpr int kPlan = kRec + kRecords * static_cast<int>(sizeof(Records));
    static constexpr int kPieces = kPlan + static_cast<int>(sizeof(Plan));
    static constexpr int kBars = kPieces + kRing * static_cast<int>(sizeof(Piece));
    static constexpr int kNumBars = 2 * kStages + 2 * kRing + 2;
    static constexpr int kTail = kBars + kNumBars * 8;
    static constexpr int kBytes = kTail + 16 + 1024;
    static_assert(kBytes <= 227 * 1024 && kStats % 16 == 0 && kRec % 8 == 0 && kPlan % 8 == 0 && kBars % 8 == 0, "layout");
};

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 codes (low, high byte of the low or high half) as two halves.
__device__ __forceinline__ uint32_t halves_lo(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// 2^(b - 127) of an e8m0 byte (2^-127 is a subnormal), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fffffffu : max(b << 23, 0x00400000u));
}
__device__ __forceinline__ float exponent_of(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7fffffffu) : static_cast<float>(static_cast<int>(b) - 127);
}

// A scale that is not a normal power of two: 2^-127, NaN.
__device__ __forceinline__ bool odd_scale(uint32_t b) { return b - 1u >= 254u; }
// The scales of the thread's two keys of a tile, from their two bytes.
using u64 = unsigned long long;
__device__ __forceinline__ u64 powers(uint32_t b, int t4) {
    const uint32_t lo = (b << 23) & 0x7f800000u, hi = (b << 15) & 0x7f800000u;
    return pack_f32x2(__uint_as_float(t4 & 1 ? hi : lo), __uint_as_float(t4 & 1 ? lo : hi));
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
    return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(kFull, v, 1);
    return v + __shfl_xor_sync(kFull, v, 2);
}

__device__ __forceinline__ int pages_of(const Piece &it) { return min(2 * it.t1, (it.limit + kP - 1) / kP) - 2 * it.t0; }

// The first of a piece's pages that is the warp's: page x of the CTA is warp
// x % kWarps's, and the piece's begin at `base`.
template <bool QUANT>
__device__ __forceinline__ int first_page(int warp, int base) {
    constexpr int kWarps = Smem<QUANT>::kWarps;
    const int d = warp - base % kWarps;
    return d < 0 ? d + kWarps : d;
}

// The whole warp's wait: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status) {
    return __all_sync(kFull, mbar_wait(bar, parity, abort_flag, status));
}

// A page warp's loads: its pages, in order, over the pieces published so far.
template <bool QUANT>
struct Loader {
    using L = Smem<QUANT>;
    int warp, lane;
    uint8_t *stages;
    uint32_t bar_k, bar_v;
    uint64_t policy;
    int piece, page, pages, idx;  // the piece it is in, the warp's next page there, how many pages, how many taken
    int r, h, page0;
    int mine;   // row of K of the warp's page idx & ~31 + lane, -1 where the id is no page
    int yk, yv; // pages of the warp whose K, V are on their way or there
    int row;    // of page yk - 1

    __device__ __forceinline__ void begin(int w, int l, uint8_t *smem, uint32_t bk, uint32_t bv) {
        warp = w;
        lane = l;
        stages = smem + w * L::kOwn * L::kStageBytes;
        bar_k = bk + 8 * w * L::kOwn;
        bar_v = bv + 8 * w * L::kOwn;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));  // no page is read twice
        piece = -1;
        page = pages = idx = yk = yv = 0;
    }

    // Row of the next page's K (-1: no page), or -2 where it is not known
    // yet.  n: the piece the warp is in, whose publication it has seen.
    __device__ __forceinline__ int take(const ChunkParams &p, const Piece *pieces, uint32_t bar_piece, int n) {
        while (page >= pages) {
            const int next = piece + 1;
            if (next > n &&
                (next >= n + kRing || !__all_sync(kFull, mbar_test(bar_piece + 8 * (next % kRing), (next / kRing) & 1))))
                return -2;
            const Piece &it = pieces[next % kRing];
            if (it.row < 0) return -2;
            piece = next;
            page0 = 2 * it.t0;
            pages = pages_of(it);
            page = first_page<QUANT>(warp, it.base);
            idx = 0;
            r = it.r;
            h = it.h;
        }
        if ((idx & 31) == 0) {
            mine = -1;
            if (page + L::kWarps * lane < pages) {
                const long long id = page_of(p.page_table, p.page_stride, p.num_pages, r, (page0 + page + L::kWarps * lane) * kP);
                if (id >= 0) mine = static_cast<int>((id * 2 * p.Hkv + h) * kP);
            }
        }
        const int at = __shfl_sync(kFull, mine, idx & 31);
        ++idx;
        page += L::kWarps;
        return at;
    }

    // One tile and its scales: dst, their place in the stage.
    __device__ __forceinline__ void issue(const ChunkParams &p, const CUtensorMap &map, uint32_t bar, uint8_t *stage, int is_v,
                                          int at) {
        uint8_t *dst = stage + is_v * L::kTileBytes, *sc = stage + 2 * L::kTileBytes + is_v * kP;
        if (at < 0) {
            for (int e = lane; e < L::kTileBytes / 16; e += 32)
                reinterpret_cast<uint4 *>(dst)[e] = make_uint4(0, 0, 0, 0);
            if (QUANT && lane < kP / 16) reinterpret_cast<uint4 *>(sc)[lane] = make_uint4(0, 0, 0, 0);
            fence_proxy_async();  // the stage's next load comes after
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        } else if (lane == 0) {
            const int src = at + is_v * p.Hkv * kP;
            mbar_arrive_expect_tx(bar, L::kTileBytes + (QUANT ? kP : 0));
            tma_load_2d(smem_u32(dst), &map, 0, src, bar, policy);
            if (QUANT) bulk_load(smem_u32(sc), p.scales + src, kP, bar);
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool k(const ChunkParams &p, const CUtensorMap &map, const Piece *pieces, uint32_t bar_piece,
                                      int n) {
        const int at = take(p, pieces, bar_piece, n);
        if (at == -2) return false;
        if (at < 0 && lane == 0 && p.status) atomicOr(p.status, K3DA_STATUS_BAD_PAGE);
        row = at;
        issue(p, map, bar_k + 8 * (yk % L::kOwn), stages + yk % L::kOwn * L::kStageBytes, 0, at);
        ++yk;
        return true;
    }
    __device__ __forceinline__ void v(const ChunkParams &p, const CUtensorMap &map) {
        issue(p, map, bar_v + 8 * (yv % L::kOwn), stages + yv % L::kOwn * L::kStageBytes, 1, row);
        ++yv;
    }

    // Pages up to y + kOwn: all of the stages but page y's are free.
    __device__ __forceinline__ void fill(const ChunkParams &p, const CUtensorMap &map, const Piece *pieces,
                                         uint32_t bar_piece, int n, int y) {
        while (yk < y + L::kOwn && k(p, map, pieces, bar_piece, n)) v(p, map);
    }
    // After page y's scores.
    __device__ __forceinline__ void next_k(const ChunkParams &p, const CUtensorMap &map, const Piece *pieces,
                                           uint32_t bar_piece, int n, int y) {
        if (yk == y + L::kOwn) k(p, map, pieces, bar_piece, n);
    }
    // After its product.
    __device__ __forceinline__ void next_v(const ChunkParams &p, const CUtensorMap &map, const Piece *pieces,
                                           uint32_t bar_piece, int n, int y) {
        if (yv < yk) v(p, map);
        fill(p, map, pieces, bar_piece, n, y + 1);
    }
    // Waits (with a limit) for loads that no page was read from: a wait gave
    // up before.
    __device__ __forceinline__ void drain() {
        for (int s = 0; s < 2 * L::kOwn; ++s) {
            const int last = s < L::kOwn ? yk - 1 - s : yv - 1 - (s - L::kOwn);
            if (last < 0) continue;
            const uint32_t bar = (s < L::kOwn ? bar_k : bar_v) + 8 * (last % L::kOwn);
            const unsigned long long t0 = global_ns();
            while (!mbar_try_wait(bar, (last / L::kOwn) & 1) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
    }
};

template <bool QUANT>
__global__ void __launch_bounds__(Smem<QUANT>::kThreads, 1)
    k3da_chunk_small_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ ChunkParams p) {
    using L = Smem<QUANT>;
    constexpr int kWarps = L::kWarps, kThreads = L::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    Plan *pl = reinterpret_cast<Plan *>(smem + L::kPlan);
    Records *recs = reinterpret_cast<Records *>(smem + L::kRec);
    Piece *pieces = reinterpret_cast<Piece *>(smem + L::kPieces);
    float *merge_o = reinterpret_cast<float *>(smem + L::kMerge);      // [kWarps][16][kORow]
    float4 *merge_s = reinterpret_cast<float4 *>(smem + L::kStats);    // [kWarps][16] (m, l, m' of O)
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kTail);
    const uint32_t bars = smem_u32(smem + L::kBars);
    const uint32_t bar_k = bars;                       // [kStages] K loaded
    const uint32_t bar_v = bar_k + 8 * L::kStages;     // [kStages] V loaded
    const uint32_t bar_piece = bar_v + 8 * L::kStages; // [kRing] piece published
    const uint32_t bar_pdone = bar_piece + 8 * kRing;      // [kRing] ... and read by every page warp
    const uint32_t bar_left = bar_pdone + 8 * kRing;       // the page warps' results are in the merge room
    const uint32_t bar_merged = bar_left + 8;              // ... and read
    const int warp = __shfl_sync(kFull, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    build_plan<256>(p, pl, blockIdx.x == 0);
    if (pl->prefix[p.R] == 0) {
        if (threadIdx.x == 0) p.cuts[blockIdx.x] = Cut{};
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_k + 8 * s, 1);
            mbar_init(bar_v + 8 * s, 1);
        }
        for (int s = 0; s < kRing; ++s) {
            mbar_init(bar_piece + 8 * s, 1);
            mbar_init(bar_pdone + 8 * s, kWarps);
        }
        mbar_init(bar_left, kWarps);
        mbar_init(bar_merged, kWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (!QUANT) {
        for (int e = threadIdx.x; e < kRecords; e += kThreads) recs[e].piece = -1;
        for (int e = threadIdx.x; e < kRecords * 3 * kD; e += kThreads)
            (&recs[e / (3 * kD)].first[0][0])[e % (3 * kD)] = 0xffffffffu;
    }
    __syncthreads();

    if (warp == kWarps) {
        // --------------------------------------------------------- pieces --
        if (lane == 0) {
            Walk walk;
            walk.begin(p, pl, blockIdx.x);
            Cut cut = {};
            int x = 0, seq = 0;
            for (int n = 0;; ++n) {
                Piece &it = pieces[n % kRing];
                if (!mbar_wait(bar_pdone + 8 * (n % kRing), ((n / kRing) & 1) ^ 1, abort_flag, p.status)) break;
                const bool more = walk.next(p, it);
                if (!more) it.row = -1;
                it.base = x;
                it.seq = seq;
                if (more && it.t0 < it.t1) {
                    ++seq;
                    x += pages_of(it);
                }
                if (more && it.t0 > 0) cut.has[0] = 1;
                if (more && it.t0 == 0 && it.t0 < it.t1 && it.t1 < it.nt) {
                    cut.has[1] = 1;
                    cut.row = it.row;
                    cut.tokens = it.tokens;
                    cut.head = it.h;
                    cut.last = walk.slice_of(walk.start + walk.length - 1);
                }
                mbar_arrive(bar_piece + 8 * (n % kRing));
                if (!more) break;
            }
            p.cuts[blockIdx.x] = cut;
        }
    } else {
        // ----------------------------------------------------- page warps --
        const int g = lane >> 2, t4 = lane & 3;  // a fragment's row or column group, and the thread in it
        Loader<QUANT> load;
        load.begin(warp, lane, smem, bar_k, bar_v);
        int y = 0;  // pages this warp is done with
        for (int n = 0;; ++n) {
            const Piece &it = pieces[n % kRing];
            if (!warp_wait(bar_piece + 8 * (n % kRing), (n / kRing) & 1, abort_flag, p.status)) break;
            if (it.row < 0) break;
            const int limit = it.limit, piece = it.seq;
            const int page0 = 2 * it.t0, pages = pages_of(it);
            load.fill(p, kv_map, pieces, bar_piece, n, y);
            const int least = keys_seen(p, it.ctx, it.n, 0);  // keys that every row sees
            // Rows g and g + 8 of the item (token major, the heads of a token
            // together); the thread has dims 16 t4 .. 16 t4 + 15 of each, and
            // so of every key: the order of dims in a product is free.
            uint32_t qf[2][8];
            int sees[2];
            float row_scale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rho = g + 8 * i, token = rho / p.G;
                const bool valid = token < it.tokens;
                sees[i] = valid ? keys_seen(p, it.ctx, it.n, token) : 0;
                uint4 a = make_uint4(0, 0, 0, 0), b = a;
                if (valid) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        p.q + static_cast<long long>(it.row + token) * p.q_stride + (it.h * p.G + rho - token * p.G) * kD + 16 * t4);
                    a = __ldg(src);
                    b = __ldg(src + 1);
                }
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                row_scale[i] = p.scale_log2;
                if (QUANT) {
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, max((w[e] & 0x7fffu) << 16, w[e] & 0x7fff0000u));
                    top = max(top, __shfl_xor_sync(kFull, top, 1));
                    top = max(top, __shfl_xor_sync(kFull, top, 2));
                    // 2^(14 - e) for a largest magnitude of 2^e; as it is for
                    // a row that is zero or not finite.
                    const uint32_t ex = top >> 23;
                    const uint32_t f = ex == 0 || ex == 255 ? 127u : min(268u - ex, 253u);
                    const float up = __uint_as_float(f << 23);
                    row_scale[i] *= __uint_as_float((254u - f) << 23);
#pragma unroll
                    for (int e = 0; e < 8; ++e) qf[i][e] = pack_half2(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) qf[i][e] = w[e];
                }
            }
            float o[8][4];
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int q = 0; q < 4; ++q) o[d][q] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            // While V's exponents in the piece are within kNear of one another.
            bool near = QUANT, alive = true;
            int e_hi = -1, e_lo = 256;
            for (int j = first_page<QUANT>(warp, it.base); j < pages; j += kWarps, ++y) {
                const int st = warp * L::kOwn + y % L::kOwn;
                if (!warp_wait(bar_k + 8 * st, (y / L::kOwn) & 1, abort_flag, p.status)) {
                    alive = false;
                    break;
                }
                uint8_t *kt = smem + st * L::kStageBytes, *vt = kt + L::kTileBytes;
                const uint8_t *ks = kt + 2 * L::kTileBytes, *vs = ks + kP;
                const int key0 = (page0 + j) * kP;
                const bool masked = key0 + kP > least;
                // The thread's scores of tile i are of the keys 8 i + k0 and
                // 8 i + k1.  Codes lie 64 bytes a row, so keys 2 and 3 of
                // every four change places, which spreads a product's V rows
                // over the banks.
                const int k0 = QUANT ? 2 * t4 + (t4 & 1) : 2 * t4, k1 = QUANT ? 2 * t4 + 1 - (t4 & 1) : 2 * t4 + 1;
                float s[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) s[i][q] = 0.f;
                    if (QUANT) {
                        const int row = 8 * i + (g ^ (g >> 1 & 1));
                        const uint4 w = *reinterpret_cast<const uint4 *>(kt + row * kD + 16 * t4);
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            mma16816<true>(s[i], qf[0][2 * q], qf[1][2 * q], qf[0][2 * q + 1], qf[1][2 * q + 1],
                                           halves_lo(in[q]), halves_hi(in[q]));
                    } else {
                        const int row = 8 * i + g;
                        const uint4 w = *reinterpret_cast<const uint4 *>(kt + swz(row, 2 * t4));
                        const uint4 y = *reinterpret_cast<const uint4 *>(kt + swz(row, 2 * t4 + 1));
                        mma16816<false>(s[i], qf[0][0], qf[1][0], qf[0][1], qf[1][1], w.x, w.y);
                        mma16816<false>(s[i], qf[0][2], qf[1][2], qf[0][3], qf[1][3], w.z, w.w);
                        mma16816<false>(s[i], qf[0][4], qf[1][4], qf[0][5], qf[1][5], y.x, y.y);
                        mma16816<false>(s[i], qf[0][6], qf[1][6], qf[0][7], qf[1][7], y.z, y.w);
                    }
                }
                // Scores in log2 units, masked.
                float top[2] = {-INFINITY, -INFINITY};
                const uint32_t kb = QUANT ? *reinterpret_cast<const uint16_t *>(ks + 2 * lane) : 0u;
                const bool plain = QUANT && !masked && !__any_sync(kFull, odd_scale(kb & 255u) || odd_scale(kb >> 8));
                if (plain) {
                    const u64 rs[2] = {pack_f32x2(row_scale[0], row_scale[0]), pack_f32x2(row_scale[1], row_scale[1])};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const u64 f = powers(*reinterpret_cast<const uint16_t *>(ks + 8 * i + 2 * t4), t4);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float2 v = unpack_f32x2(mul_f32x2(mul_f32x2(pack_f32x2(s[i][2 * q], s[i][2 * q + 1]), rs[q]), f));
                            s[i][2 * q] = v.x;
                            s[i][2 * q + 1] = v.y;
                            top[q] = fmax3(top[q], v.x, v.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float f0 = 1.f, f1 = 1.f;
                        if (QUANT) {
                            const uint32_t b = *reinterpret_cast<const uint16_t *>(ks + 8 * i + 2 * t4);
                            f0 = scale_of(t4 & 1 ? b >> 8 : b & 255u);
                            f1 = scale_of(t4 & 1 ? b & 255u : b >> 8);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            s[i][q] *= row_scale[q >> 1];
                            if (QUANT) s[i][q] *= q & 1 ? f1 : f0;
                            if (masked && key0 + 8 * i + (q & 1 ? k1 : k0) >= sees[q >> 1]) s[i][q] = -INFINITY;
                            top[q >> 1] = fmaxf(top[q >> 1], s[i][q]);
                        }
                    }
                }
                __syncwarp();
                load.next_k(p, kv_map, pieces, bar_piece, n, y);
                if (!warp_wait(bar_v + 8 * st, (y / L::kOwn) & 1, abort_flag, p.status)) {
                    alive = false;
                    break;
                }
                if (!QUANT && masked) {
                    // As in the long chunks' kernel: V rows past the last key
                    // to zero, infinities and NaN of a key that not every row
                    // sees out of V and into the records.
                    Records *rec = recs + piece % kRecords;
                    const uint32_t tag = ~static_cast<uint32_t>(piece) << 8;
#pragma unroll 1
                    for (int e = lane; e < kP * 8; e += 32) {
                        const int key = key0 + (e >> 3), c = e & 7;
                        if (key < least) continue;
                        uint4 *at = reinterpret_cast<uint4 *>(vt + swz(e >> 3, c));
                        if (key >= limit) {
                            *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint4 w = *at;
                        uint32_t v[4] = {w.x, w.y, w.z, w.w};
                        bool bad = false;
#pragma unroll
                        for (int q = 0; q < 4; ++q) bad |= (v[q] & 0x7f80u) == 0x7f80u || (v[q] & 0x7f800000u) == 0x7f800000u;
                        if (!bad) continue;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint32_t b = v[q >> 1] >> (16 * (q & 1)) & 0xffffu;
                            if ((b & 0x7f80u) != 0x7f80u) continue;
                            atomicMin(&rec->first[b & 0x7fu ? 2 : b >> 15][8 * c + q], tag | (key - least));
                            v[q >> 1] &= q & 1 ? 0x0000ffffu : 0xffff0000u;
                        }
                        *at = make_uint4(v[0], v[1], v[2], v[3]);
                        rec->piece = piece;
                    }
                    fence_proxy_async();  // the stage's next load comes after
                    __syncwarp();
                }
                // Weights, in place of the scores.
                float base[2], fo[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mn = fmaxf(m[i], quad_max(top[i]));
                    base[i] = mn == -INFINITY ? 0.f : mn;
                    fo[i] = exp2_approx(m[i] - base[i]);
                    l[i] *= fo[i];
                    m[i] = mn;
                }
                if (QUANT) {
                    const uint32_t vb = *reinterpret_cast<const uint16_t *>(vs + 2 * lane);
                    const int hi = max(e_hi, static_cast<int>(__reduce_max_sync(kFull, max(vb & 255u, vb >> 8))));
                    const int lo = min(e_lo, static_cast<int>(__reduce_min_sync(kFull, min(vb & 255u, vb >> 8))));
                    near = near && plain && hi < 255 && hi - lo <= kNear;
                    if (near) {
                        e_hi = hi;
                        e_lo = lo;
                    }
                }
                if (near) {
                    const uint32_t shift = static_cast<uint32_t>(e_hi - 127) * 0x0101u;
                    const u64 nb[2] = {pack_f32x2(-base[0], -base[0]), pack_f32x2(-base[1], -base[1])};
                    u64 sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const u64 g2 = powers(*reinterpret_cast<const uint16_t *>(vs + 8 * i + 2 * t4) - shift, t4);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const u64 w = exp2_f32x2(add_f32x2(pack_f32x2(s[i][2 * q], s[i][2 * q + 1]), nb[q]));
                            sum[q] = add_f32x2(sum[q], w);
                            const float2 v = unpack_f32x2(mul_f32x2(w, g2));
                            s[i][2 * q] = v.x;
                            s[i][2 * q + 1] = v.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = unpack_f32x2(sum[i]);
                        l[i] += v.x + v.y;
                        const float mn = m[i] + static_cast<float>(e_hi - 127);
                        fo[i] = exp2_approx(mo[i] - (mn == -INFINITY ? 0.f : mn));
                        mo[i] = mn;
                    }
                } else {
                    float base_o[2] = {base[0], base[1]};
                    if (QUANT) {
                        float top_o[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t b = *reinterpret_cast<const uint16_t *>(vs + 8 * i + 2 * t4);
                            const float e0 = exponent_of(t4 & 1 ? b >> 8 : b & 255u), e1 = exponent_of(t4 & 1 ? b & 255u : b >> 8);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                l[q >> 1] += exp2_approx(s[i][q] - base[q >> 1]);
                                s[i][q] = s[i][q] == -INFINITY ? -INFINITY : s[i][q] + (q & 1 ? e1 : e0);
                                top_o[q >> 1] = fmaxf(top_o[q >> 1], s[i][q]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float mn = fmaxf(mo[i], quad_max(top_o[i]));
                            base_o[i] = mn == -INFINITY ? 0.f : mn;
                            fo[i] = exp2_approx(mo[i] - base_o[i]);
                            mo[i] = mn;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            s[i][q] = exp2_approx(s[i][q] - base_o[q >> 1]);
                            if (!QUANT) l[q >> 1] += s[i][q];
                        }
                }
                if (__any_sync(kFull, fo[0] != 1.f || fo[1] != 1.f)) {
#pragma unroll
                    for (int d = 0; d < 8; ++d)
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[d][q] *= fo[q >> 1];
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 16 keys a product
                    uint32_t a[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float w0 = s[2 * c + (q >> 1)][2 * (q & 1)], w1 = s[2 * c + (q >> 1)][2 * (q & 1) + 1];
                        a[q] = QUANT ? pack_half2(w0, w1) : pack2(w0, w1);
                    }
                    if (QUANT) {
                        // Four dims of four keys a thread: bytes to pairs of
                        // keys, pairs to halves.  Column g of product d is
                        // dim 32 (d / 4) + 4 g + d % 4.
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t w[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int row = 16 * c + 8 * (q >> 1) + (q & 1 ? k1 : k0);
                                w[q] = *reinterpret_cast<const uint32_t *>(vt + row * kD + 32 * hf + 4 * g);
                                if (masked) {
                                    // NaN codes meet weights of zero: none is
                                    // left past the last key, or at all.
                                    const uint32_t nan = ((w[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                    w[q] = key0 + row >= limit ? 0u : w[q] - (nan >> 7);
                                }
                            }
                            const uint32_t lo0 = __byte_perm(w[0], w[1], 0x5140), lo1 = __byte_perm(w[0], w[1], 0x7362);
                            const uint32_t hi0 = __byte_perm(w[2], w[3], 0x5140), hi1 = __byte_perm(w[2], w[3], 0x7362);
                            mma16816<true>(o[4 * hf + 0], a[0], a[1], a[2], a[3], halves_lo(lo0), halves_lo(hi0));
                            mma16816<true>(o[4 * hf + 1], a[0], a[1], a[2], a[3], halves_hi(lo0), halves_hi(hi0));
                            mma16816<true>(o[4 * hf + 2], a[0], a[1], a[2], a[3], halves_lo(lo1), halves_lo(hi1));
                            mma16816<true>(o[4 * hf + 3], a[0], a[1], a[2], a[3], halves_hi(lo1), halves_hi(hi1));
                        }
                    } else {
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const int row = 16 * c + (lane & 15);
                            uint32_t b[4];
                            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                                         : "r"(smem_u32(vt) + swz(row, 2 * d + (lane >> 4)))
                                         : "memory");
                            mma16816<false>(o[2 * d], a[0], a[1], a[2], a[3], b[0], b[1]);
                            mma16816<false>(o[2 * d + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
                        }
                    }
                }
                __syncwarp();
                load.next_v(p, kv_map, pieces, bar_piece, n, y);
            }
            if (!alive) break;
            // ---------------------------------------------------- merging --
            if (n > 0 && !warp_wait(bar_merged, (n - 1) & 1, abort_flag, p.status)) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float sum = quad_sum(l[i]);
                if (t4 == 0) merge_s[warp * kSmallRows + g + 8 * i] = make_float4(m[i], sum, QUANT ? mo[i] : m[i], 0.f);
                float *dst = merge_o + (warp * kSmallRows + g + 8 * i) * kORow;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const int dim = QUANT ? 32 * (d >> 2) + 8 * t4 + (d & 3) : 8 * d + 2 * t4;
                    dst[dim] = o[d][2 * i];
                    dst[dim + (QUANT ? 4 : 1)] = o[d][2 * i + 1];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_left);
            if (!warp_wait(bar_left, n & 1, abort_flag, p.status)) break;
            if (warp < 8) {
                // A row's four dims a thread.
                const int rho = threadIdx.x >> 4, dim = 4 * (threadIdx.x & 15), token = rho / p.G;
                float mt = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, merge_s[w * kSmallRows + rho].x);
                const float me = mt == -INFINITY ? 0.f : mt;
                float lt = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 st = merge_s[w * kSmallRows + rho];
                    const float4 part = *reinterpret_cast<const float4 *>(merge_o + (w * kSmallRows + rho) * kORow + dim);
                    const float f = exp2_approx(st.z - me);
                    lt += st.y * exp2_approx(st.x - me);
                    v[0] += part.x * f;
                    v[1] += part.y * f;
                    v[2] += part.z * f;
                    v[3] += part.w * f;
                }
                const bool whole = it.t0 == 0 && it.t1 == it.nt;
                const float norm = whole ? 1.f / lt : 1.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = lt == 0.f ? 0.f : v[q] * norm;
                const Records &rec = recs[piece % kRecords];
                const int row_sees = token < it.tokens ? keys_seen(p, it.ctx, it.n, token) : 0;
                if (!QUANT && pages > 0 && rec.piece == piece) {
                    const uint32_t tag = ~static_cast<uint32_t>(piece) << 8;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        for (int kind = 0; kind < 3; ++kind) {
                            const uint32_t e = rec.first[kind][dim + q];
                            if ((e & 0xffffff00u) != tag || least + static_cast<int>(e & 0xffu) >= row_sees) continue;
                            v[q] = kind == 2 ? __uint_as_float(0x7fffffffu) : v[q] + (kind == 0 ? INFINITY : -INFINITY);
                        }
                }
                if (token < it.tokens) {
                    const long long at = static_cast<long long>(it.row + token) * p.Hq + it.h * p.G + rho - token * p.G;
                    const int part = (blockIdx.x * 2 + (it.t0 > 0 ? 0 : 1)) * kSmallRows + rho;
                    if (whole) {
                        *reinterpret_cast<uint2 *>(p.out + at * kD + dim) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
                        if (dim == 0 && p.lse) p.lse[at] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * 0.6931471805599453f;
                    } else {
                        *reinterpret_cast<float4 *>(p.part_o + static_cast<long long>(part) * kD + dim) =
                            make_float4(v[0], v[1], v[2], v[3]);
                        if (dim == 0) p.part_ml[part] = make_float2(mt, lt);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_merged);
                mbar_arrive(bar_pdone + 8 * (n % kRing));
            }
        }
        load.drain();
    }
    // The kernel this one may have started beside is complete before it is.
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <bool QUANT>
int launch(const CUtensorMap &kv_map, const ChunkParams &p, bool after_long, cudaStream_t stream) {
    // Set at every call: a context has its own copy of the attribute.
    if (cudaFuncSetAttribute(k3da_chunk_small_kernel<QUANT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem<QUANT>::kBytes) != cudaSuccess)
        return K3DA_ECUDA;
    cudaLaunchConfig_t lc;
    std::memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3(kCtas);
    lc.blockDim = dim3(Smem<QUANT>::kThreads);
    lc.dynamicSmemBytes = Smem<QUANT>::kBytes;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = after_long ? 1 : 0;
    return cudaLaunchKernelEx(&lc, k3da_chunk_small_kernel<QUANT>, kv_map, p) == cudaSuccess ? K3DA_OK : K3DA_ECUDA;
}

}  // namespace

int launch_small(const ChunkParams &p, const void *kv_pool, bool quant, bool after_long, cudaStream_t stream) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    CUtensorMap kv_map;
    if (encode == nullptr || !pool_map(encode, &kv_map, kv_pool, p.num_pages, p.Hkv, quant)) return K3DA_ECUDA;
    return quant ? launch<true>(kv_map, p, after_long, stream) : launch<false>(kv_map, p, after_long, stream);
}

}  // namespace k3da_chunk
