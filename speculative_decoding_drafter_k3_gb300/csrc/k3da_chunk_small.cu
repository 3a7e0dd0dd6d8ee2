// k3da_chunk_small.cu -- the chunk attention of requests that bring few query
// rows (at most 16 a kv head: decoded tokens, mostly), sm_103a.
//
// Same items, line and cuts as the long chunks' kernel (chunk_plan.cuh), but
// an item is bound by reading its cache, and what 128-row products and the
// widening of codes to bf16 tiles in shared memory cost would be the bound
// instead.  Here a warp takes a page by itself: products of 16 keys by 8 rows
// (mma.sync), the cache's fragments straight from where TMA put them, a
// running maximum, sum and O of its own in registers, and no barrier but its
// tiles'.  8 such warps (11 for codes: a page of them is more arithmetic a
// byte) share an item's pages; another hands out the pieces and folds the
// warps' results.
//
// Quantised pages stay codes: a code is a half-precision number as it is (one
// conversion for two), K's scale multiplies a finished score, and V's goes
// into the weight: w = 2^(s + e - m'), with a reference m' beside the maximum
// m of s that the sum keeps.  As a rule V's exponents e of a piece lie close
// together, and m' = m + max e - 15, so that one exp serves sum and weight;
// else m' is 15 below the running maximum of s + e.  (15: half precision then
// holds weights down to 2^-39 of the largest.)  Both are exponents, so scales
// of any size meet no range.  q is scaled by a power of two into half
// precision's range (exact but for dims 2^-31 below the row's largest, which
// lose bits, and are gone 2^-39 below).
//
// Measured (64 decoded tokens over 8000 each, 24/4 heads): e4m3 54 us, 4.9
// TB/s of cache, where the long chunks' kernel takes 133; bf16 90 us, 5.8
// TB/s, against 92.  About 9 us of either are launches, plan, first loads
// and the fold of cut items; the rest streams at 5.6 to 6.0 TB/s.  15 warps of
// 128 registers took as long, and a quarter more where two tiles of rows spill
// (8 x 2 tokens over 60000, 16/2 heads, e4m3: 37 us with 11).
//
// Rounding: scores, statistics, O and partial results are fp32; weights are
// rounded once (bf16, or half precision for codes: see kHead), the output once.
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

// Page warps; one more schedules and merges.
constexpr int page_warps(bool quant) { return quant ? 11 : 8; }
constexpr int kRing = 4;     // pieces published ahead
constexpr int kRecords = 8;  // pieces whose non-finite records are alive at once
// With codes, the largest weight is 2^kHead in half precision (its largest
// number is 65504): a weight is off by 2^-12 of itself, or, where half's
// numbers are subnormal, by 2^-25 of 2^-kHead of the reference, 2^-40.  Keys
// that are alike all err one way, so it is their sum that counts: with the
// reference at 1 instead, 60000 keys of 2^-15.3 next to a key of 1 were lost,
// 8% of the output.
constexpr int kHead = 15;
// Spread of V's exponents up to which one reference exponent serves a piece's
// keys.  The reference then is at most 2^10 above the largest weight, and n
// keys lose n 2^-30 of that at most: 2^-13 of 131072.
constexpr int kNear = 10;
constexpr int kORow = kD + 4;  // floats of a row in the merge room (the pad spreads rows over the banks)

template <bool QUANT>
struct Smem {
    static constexpr int kWarps = page_warps(QUANT);
    static constexpr int kThreads = 32 * (kWarps + 1);
    // A warp loads its own tiles (K, V, K, V, ... of its pages) into its own
    // places in turn, each as soon as the tile there is done with.
    static constexpr int kOwn = QUANT ? 3 : 2;
    static constexpr int kTiles = kWarps * kOwn;
    static constexpr int kTileBytes = kP * kD * (QUANT ? 1 : 2);
    static constexpr int kScales = kTiles * kTileBytes;  // [kTiles][64]
    static constexpr int kMerge = kScales + (QUANT ? kTiles * kP : 0);
    static constexpr int kStats = kMerge + kWarps * kSmallRows * kORow * 4;
    static constexpr int kRec = kStats + kWarps * kSmallRows * 16;
    static constexpr int kPlan = kRec + kRecords * static_cast<int>(sizeof(Records));
    static constexpr int kPieces = kPlan + static_cast<int>(sizeof(Plan));
    static constexpr int kBars = kPieces + kRing * static_cast<int>(sizeof(Piece));
    static constexpr int kNumBars = kTiles + kRing + 2;
    static constexpr int kTail = kBars + kNumBars * 8;
    static constexpr int kBytes = kTail + 16 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(kMerge % 16 == 0 && kStats % 16 == 0 && kRec % 8 == 0 && kPlan % 8 == 0 && kBars % 8 == 0, "alignment");
};

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
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
using u64 = unsigned long long;

// Over the lanes of the same t4: the keys of a product's tile.
__device__ __forceinline__ float keys_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
    v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
    return fmaxf(v, __shfl_xor_sync(kFull, v, 16));
}
__device__ __forceinline__ float keys_sum(float v) {
    v += __shfl_xor_sync(kFull, v, 4);
    v += __shfl_xor_sync(kFull, v, 8);
    return v + __shfl_xor_sync(kFull, v, 16);
}

// An 8 x 8 tile of 16-bit numbers, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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
    uint8_t *tiles, *scales;  // the warp's
    uint32_t bars;
    uint64_t policy;
    int piece, page, pages, idx;  // the piece it is in, the warp's next page there, how many pages, how many taken
    int r, h, page0;
    int mine;   // row of K of the warp's page idx & ~31 + lane, -1 where the id is no page
    int issued;  // tiles on their way or there
    int place;  // of the next one
    int row;    // its page's

    __device__ __forceinline__ void begin(int w, int l, uint8_t *smem, uint32_t b) {
        warp = w;
        lane = l;
        tiles = smem + w * L::kOwn * L::kTileBytes;
        scales = smem + L::kScales + w * L::kOwn * kP;
        bars = b + 8 * w * L::kOwn;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));  // no page is read twice
        piece = -1;
        page = pages = idx = issued = place = 0;
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

    // The tiles that find a place when `done` were done with.
    __device__ __forceinline__ void fill(const ChunkParams &p, const CUtensorMap &map, const Piece *pieces,
                                         uint32_t bar_piece, int n, int done) {
        while (issued < done + L::kOwn) {
            const int is_v = issued & 1;
            if (!is_v) {
                const int at = take(p, pieces, bar_piece, n);
                if (at == -2) return;
                if (at < 0 && lane == 0 && p.status) atomicOr(p.status, K3DA_STATUS_BAD_PAGE);
                row = at;
            }
            uint8_t *dst = tiles + place * L::kTileBytes, *sc = scales + place * kP;
            const uint32_t bar = bars + 8 * place;
            if (__builtin_expect(row < 0, 0)) {
                for (int e = lane; e < L::kTileBytes / 16; e += 32)
                    reinterpret_cast<uint4 *>(dst)[e] = make_uint4(0, 0, 0, 0);
                if (QUANT && lane < kP / 16) reinterpret_cast<uint4 *>(sc)[lane] = make_uint4(0, 0, 0, 0);
                fence_proxy_async();  // the place's next load comes after
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            } else if (elect_one()) {
                const int src = row + is_v * p.Hkv * kP;
                mbar_arrive_expect_tx(bar, L::kTileBytes + (QUANT ? kP : 0));
                tma_load_2d(smem_u32(dst), &map, 0, src, bar, policy);
                if (QUANT) bulk_load(smem_u32(sc), p.scales + src, kP, bar);
            }
            __syncwarp();
            ++issued;
            place = place + 1 == L::kOwn ? 0 : place + 1;
        }
    }
    // Waits (with a limit) for loads that no product read: a wait gave up
    // before.
    __device__ __forceinline__ void drain() {
        for (int j = max(issued - L::kOwn, 0); j < issued; ++j) {
            const unsigned long long t0 = global_ns();
            while (!mbar_try_wait(bars + 8 * (j % L::kOwn), (j / L::kOwn) & 1) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
    }
};

// The page warps' results of a piece, folded, and out: sixteen dims of a row
// a lane, eight rows at a time.
template <bool QUANT>
__device__ __forceinline__ void merge_piece(const ChunkParams &p, const Piece &it, const float *merge_o,
                                            const float4 *merge_s, const Records *recs, int lane) {
    constexpr int kWarps = Smem<QUANT>::kWarps;
    const bool whole = it.t0 == 0 && it.t1 == it.nt;
    const Records &rec = recs[it.seq % kRecords];
    const bool hidden = !QUANT && it.t0 < it.t1 && rec.piece == it.seq;
    const int dim0 = 16 * (lane & 3);
#pragma unroll 1
    for (int rho = lane >> 2; rho < it.tokens * p.G; rho += 8) {
        // (Unrolled no further: the page loops want the instruction cache.)
        float mt = -INFINITY, zt = -INFINITY;
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) {
            mt = fmaxf(mt, merge_s[w * kSmallRows + rho].x);
            if (QUANT) zt = fmaxf(zt, merge_s[w * kSmallRows + rho].z);
        }
        const float me = mt == -INFINITY ? 0.f : mt;
        // With codes the O are folded at the largest of their references: the
        // way from there to the scores' maximum is as far as V's scales reach,
        // past what one factor can hold, and comes last, in two.
        const float ze = !QUANT ? me : zt == -INFINITY ? 0.f : zt;
        float lt = 0.f, v[16] = {};
#pragma unroll 2
        for (int w = 0; w < kWarps; ++w) {
            const float4 st = merge_s[w * kSmallRows + rho];
            const float4 *part = reinterpret_cast<const float4 *>(merge_o + (w * kSmallRows + rho) * kORow + dim0);
            const float f = exp2_approx(st.z - ze);
            lt += st.y * exp2_approx(st.x - me);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 x = part[q];
                v[4 * q] += x.x * f;
                v[4 * q + 1] += x.y * f;
                v[4 * q + 2] += x.z * f;
                v[4 * q + 3] += x.w * f;
            }
        }
        const float half_way = QUANT ? exp2_approx(0.5f * (ze - me)) : 1.f;
        const float norm = (whole ? 1.f / lt : 1.f) * half_way;
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = lt == 0.f ? 0.f : QUANT ? v[q] * norm * half_way : v[q] * norm;
        const int token = rho / p.G;
        if (hidden) {
            const int least = keys_seen(p, it.ctx, it.n, 0), sees = keys_seen(p, it.ctx, it.n, token);
            const uint32_t tag = ~static_cast<uint32_t>(it.seq) << 8;
#pragma unroll
            for (int q = 0; q < 16; ++q)
#pragma unroll 1
                for (int kind = 0; kind < 3; ++kind) {
                    const uint32_t e = rec.first[kind][dim0 + q];
                    if ((e & 0xffffff00u) != tag || least + static_cast<int>(e & 0xffu) >= sees) continue;
                    v[q] = kind == 2 ? __uint_as_float(0x7fffffffu) : v[q] + (kind == 0 ? INFINITY : -INFINITY);
                }
        }
        if (whole) {
            const long long at = static_cast<long long>(it.row + token) * p.Hq + it.h * p.G + rho - token * p.G;
            uint4 *out = reinterpret_cast<uint4 *>(p.out + at * kD + dim0);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                out[q] = make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                                    pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
            if (dim0 == 0 && p.lse) p.lse[at] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * 0.6931471805599453f;
        } else {
            const int part = (blockIdx.x * 2 + (it.t0 > 0 ? 0 : 1)) * kSmallRows + rho;
            float4 *out = reinterpret_cast<float4 *>(p.part_o + static_cast<long long>(part) * kD + dim0);
#pragma unroll
            for (int q = 0; q < 4; ++q) out[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            if (dim0 == 0) p.part_ml[part] = make_float2(mt, lt);
        }
    }
}

// The tile a page warp is at.
template <bool QUANT>
struct Turn {
    int done = 0, place = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        ++done;
        if (++place == Smem<QUANT>::kOwn) {
            place = 0;
            phase ^= 1u;
        }
    }
};

// What a page warp keeps of a piece.  Products are of 16 keys (or dims) by 8
// rows, so that the 4 to 8 rows of most items fill them: S^T = K q^T and
// O^T += V^T w^T.  The thread has rows 8 n + 2 t4 and one more of each row
// tile n, and of a 16-key tile i the keys 16 i + kg and + 8.
template <int NT>
struct Rows {
    // Of row 8 n + g: dims 16 t4 .. 16 t4 + 15 (and so of every key: a
    // product's order of dims is free).
    uint32_t q[NT][8];
    float scale[NT][2];
    int sees[NT][2];
    float m[NT][2], l[NT][2];
    float mo[NT][2];   // reference of O: m, or with codes kHead below the maximum of s + e
    float o[NT][4][4];
    // Codes: while V's exponents in the piece are within kNear of one another.
    bool near;
    int e_hi, e_lo;
};

// One page, over NT tiles of 8 rows.
template <bool QUANT, int NT>
__device__ __forceinline__ bool take_page(Rows<NT> &R, Loader<QUANT> &load, const ChunkParams &p, const CUtensorMap &kv_map,
                                          const Piece *pieces, uint32_t bar_piece, int n, Turn<QUANT> &turn, int key0,
                                          int least, int limit, Records *rec, int piece, int lane,
                                          volatile int *abort_flag) {
    using L = Smem<QUANT>;
    const int g = lane >> 2, t4 = lane & 3;
    if (!warp_wait(load.bars + 8 * turn.place, turn.phase, abort_flag, p.status)) return false;
    const uint8_t *kt = load.tiles + turn.place * L::kTileBytes, *ks = load.scales + turn.place * kP;
    const bool masked = page_masked(key0, least);
    // Code tiles have rows of 64 bytes, 16-byte chunks swizzled by bits 1 and
    // 2 of the row.  With keys 2 and 3 of every four exchanged, a thread's
    // loads of V (below) meet no bank twice.
    const int kg = QUANT ? g ^ (g >> 1 & 1) : g;
    float s[NT][4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 16 * i + kg;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][i][e] = 0.f;
        if (QUANT) {
            const uint32_t at = row * kD + 16 * (t4 ^ (g >> 1 & 3));
            const uint4 u = *reinterpret_cast<const uint4 *>(kt + at), v = *reinterpret_cast<const uint4 *>(kt + at + 8 * kD);
            const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a0 = halves_lo(a[e]), a1 = halves_lo(b[e]), a2 = halves_hi(a[e]), a3 = halves_hi(b[e]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<true>(s[nt][i], a0, a1, a2, a3, R.q[nt][2 * e], R.q[nt][2 * e + 1]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 a = *reinterpret_cast<const uint4 *>(kt + swz(row, 2 * t4 + c));
                const uint4 b = *reinterpret_cast<const uint4 *>(kt + swz(row + 8, 2 * t4 + c));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816<false>(s[nt][i], a.x, b.x, a.y, b.y, R.q[nt][4 * c], R.q[nt][4 * c + 1]);
                    mma16816<false>(s[nt][i], a.z, b.z, a.w, b.w, R.q[nt][4 * c + 2], R.q[nt][4 * c + 3]);
                }
            }
        }
    }
    // Scores in log2 units, masked.
    float top[NT][2];
    const uint32_t kb = QUANT ? *reinterpret_cast<const uint16_t *>(ks + 2 * lane) : 0u;
    const bool plain = !masked && (!QUANT || !__any_sync(kFull, odd_scale(kb & 255u) || odd_scale(kb >> 8)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
    if (__builtin_expect(plain, 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = QUANT ? __uint_as_float(static_cast<uint32_t>(ks[16 * i + 8 * h + kg]) << 23) : 1.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    u64 v = mul_f32x2(pack_f32x2(s[nt][i][2 * h], s[nt][i][2 * h + 1]), pack_f32x2(R.scale[nt][0], R.scale[nt][1]));
                    if (QUANT) v = mul_f32x2(v, pack_f32x2(f, f));
                    const float2 w = unpack_f32x2(v);
                    s[nt][i][2 * h] = w.x;
                    s[nt][i][2 * h + 1] = w.y;
                    top[nt][0] = fmaxf(top[nt][0], w.x);
                    top[nt][1] = fmaxf(top[nt][1], w.y);
                }
            }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = 16 * i + 8 * h + kg;
                const float f = QUANT ? scale_of(ks[key]) : 1.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float &v = s[nt][i][2 * h + c];
                        v *= R.scale[nt][c];
                        if (QUANT) v *= f;
                        if (key0 + key >= R.sees[nt][c] && masked) v = -INFINITY;
                        top[nt][c] = fmaxf(top[nt][c], v);
                    }
            }
    }
    __syncwarp();
    turn.next();
    load.fill(p, kv_map, pieces, bar_piece, n, turn.done);
    if (!warp_wait(load.bars + 8 * turn.place, turn.phase, abort_flag, p.status)) return false;
    uint8_t *vt = load.tiles + turn.place * L::kTileBytes;
    const uint8_t *vs = load.scales + turn.place * kP;
    if (QUANT && __builtin_expect(masked, 0)) {
        // Weights of zero must meet no NaN: none past the last key, nor in a
        // key that not every row sees (where the largest code stands for it).
#pragma unroll 1
        for (int e = lane; e < kP * 4; e += 32) {
            const int key = key0 + (e >> 2);
            if (key < least) continue;
            uint4 *at = reinterpret_cast<uint4 *>(vt + 16 * e);
            const uint4 w = *at;
            uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t nan = ((v[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                v[q] = key >= limit ? 0u : v[q] - (nan >> 7);
            }
            *at = make_uint4(v[0], v[1], v[2], v[3]);
        }
        fence_proxy_async();  // the stage's next load comes after
        __syncwarp();
    }
    if (!QUANT && __builtin_expect(masked, 0)) {
        // As in the long chunks' kernel: V rows past the last key
        // to zero, infinities and NaN of a key that not every row
        // sees out of V and into the records.
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
    float base[NT][2], fo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float mn = fmaxf(R.m[nt][c], keys_max(top[nt][c]));
            base[nt][c] = mn == -INFINITY ? 0.f : mn;
            fo[nt][c] = exp2_approx(R.m[nt][c] - base[nt][c]);
            R.l[nt][c] *= fo[nt][c];
            R.m[nt][c] = mn;
        }
    if (QUANT) {
        const uint32_t vb = *reinterpret_cast<const uint16_t *>(vs + 2 * lane);
        const int hi = max(R.e_hi, static_cast<int>(__reduce_max_sync(kFull, max(vb & 255u, vb >> 8))));
        const int lo = min(R.e_lo, static_cast<int>(__reduce_min_sync(kFull, min(vb & 255u, vb >> 8))));
        R.near = R.near && plain && hi < 255 && hi - lo <= kNear;
        if (R.near) {
            R.e_hi = hi;
            R.e_lo = lo;
        }
    }
    if (__builtin_expect(QUANT ? R.near : plain, 1)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const u64 nb = pack_f32x2(-base[nt][0], -base[nt][1]);
            u64 sum = 0ull;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u64 w = exp2_f32x2(add_f32x2(pack_f32x2(s[nt][i][2 * h], s[nt][i][2 * h + 1]), nb));
                    sum = add_f32x2(sum, w);
                    if (QUANT) {  // 2^(e - e_hi + kHead)
                        const float f = __uint_as_float((vs[16 * i + 8 * h + kg] + 127u + kHead - R.e_hi) << 23);
                        w = mul_f32x2(w, pack_f32x2(f, f));
                    }
                    const float2 v = unpack_f32x2(w);
                    s[nt][i][2 * h] = v.x;
                    s[nt][i][2 * h + 1] = v.y;
                }
            const float2 v = unpack_f32x2(sum);
            R.l[nt][0] += v.x;
            R.l[nt][1] += v.y;
            if (QUANT) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float mn = R.m[nt][c] + static_cast<float>(R.e_hi - 127 - kHead);
                    fo[nt][c] = exp2_approx(R.mo[nt][c] - (mn == -INFINITY ? 0.f : mn));
                    R.mo[nt][c] = mn;
                }
            }
        }
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float base_o = base[nt][c];
                if (QUANT) {
                    // V's exponents join the scores for the weights.
                    float top_o = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &v = s[nt][i][2 * h + c];
                            R.l[nt][c] += exp2_approx(v - base[nt][c]);
                            if (v != -INFINITY) v += exponent_of(vs[16 * i + 8 * h + kg]);
                            top_o = fmaxf(top_o, v);
                        }
                    const float mn = fmaxf(R.mo[nt][c], keys_max(top_o) - kHead);
                    base_o = mn == -INFINITY ? 0.f : mn;
                    fo[nt][c] = exp2_approx(R.mo[nt][c] - base_o);
                    R.mo[nt][c] = mn;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float &v = s[nt][i][2 * h + c];
                        v = exp2_approx(v - base_o);
                        if (!QUANT) R.l[nt][c] += v;
                    }
            }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (!__any_sync(kFull, fo[nt][0] != 1.f || fo[nt][1] != 1.f)) continue;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) R.o[nt][d][e] *= fo[nt][e & 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 16 keys a product
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[nt][h] = transposed(QUANT ? pack_half2(s[nt][i][2 * h], s[nt][i][2 * h + 1])
                                            : pack2(s[nt][i][2 * h], s[nt][i][2 * h + 1]));
        if (QUANT) {
            // Four dims of four keys a thread: bytes to pairs of keys, pairs
            // to halves.  Row g of dim tile 2 hf + u is dim 32 hf + 4 g + 2 u,
            // row g + 8 the one after.
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 16 * i + 8 * (e >> 1) + 2 * t4 + ((e ^ t4) & 1);
                    w[e] = *reinterpret_cast<const uint32_t *>(vt + key * kD + 16 * ((2 * hf + (g >> 2)) ^ t4) + 4 * (g & 3));
                }
                const uint32_t lo0 = __byte_perm(w[0], w[1], 0x5140), lo1 = __byte_perm(w[0], w[1], 0x7362);
                const uint32_t hi0 = __byte_perm(w[2], w[3], 0x5140), hi1 = __byte_perm(w[2], w[3], 0x7362);
                const uint32_t a[8] = {halves_lo(lo0), halves_hi(lo0), halves_lo(hi0), halves_hi(hi0),
                                       halves_lo(lo1), halves_hi(lo1), halves_lo(hi1), halves_hi(hi1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816<true>(R.o[nt][2 * hf], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
                    mma16816<true>(R.o[nt][2 * hf + 1], a[4], a[5], a[6], a[7], b[nt][0], b[nt][1]);
                }
            }
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint32_t a[4];
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                             : "=r"(a[0]), "=r"(a[2]), "=r"(a[1]), "=r"(a[3])
                             : "r"(smem_u32(vt) + swz(16 * i + (lane & 15), 2 * d + (lane >> 4)))
                             : "memory");
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<false>(R.o[nt][d], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
            }
        }
    }
    __syncwarp();
    turn.next();
    load.fill(p, kv_map, pieces, bar_piece, n, turn.done);
    return true;
}

// Piece n, over NT tiles of 8 rows, up to the warp's results in the merge
// room.  False when a wait gave up.
template <bool QUANT, int NT>
__device__ __forceinline__ bool take_piece(const ChunkParams &p, const CUtensorMap &kv_map, const Piece *pieces,
                                           uint32_t bar_piece, int n, Loader<QUANT> &load, Turn<QUANT> &turn,
                                           Records *recs, float *merge_o, float4 *merge_s, uint32_t bar_merged, int warp,
                                           int lane, volatile int *abort_flag) {
    const int g = lane >> 2, t4 = lane & 3;  // a fragment's row or column group, and the thread in it
    const Piece &it = pieces[n % kRing];
    const int limit = it.limit, piece = it.seq;
    const int page0 = 2 * it.t0, pages = pages_of(it);
    const int least = keys_seen(p, it.ctx, it.n, 0);  // keys that every row sees
    // The item's rows: token major, the heads of a token together.
    Rows<NT> R;
    uint4 qa[NT], qb[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int rho = g + 8 * nt, token = rho / p.G;
        qa[nt] = qb[nt] = make_uint4(0, 0, 0, 0);
        if (token < it.tokens) {
            const uint4 *src =
                reinterpret_cast<const uint4 *>(p.q + static_cast<long long>(it.row + token) * p.q_stride +
                                                (it.h * p.G + rho - token * p.G) * kD + 16 * t4);
            qa[nt] = load_here(src);
            qb[nt] = load_here(src + 1);
        }
    }
    // While they come: the piece's first tiles.
    load.fill(p, kv_map, pieces, bar_piece, n, turn.done);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const uint4 a = qa[nt], b = qb[nt];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        float scale = p.scale_log2;
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
            scale *= __uint_as_float((254u - f) << 23);
#pragma unroll
            for (int e = 0; e < 8; ++e) R.q[nt][e] = pack_half2(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) R.q[nt][e] = w[e];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int mine = (8 * nt + 2 * t4 + c) / p.G;
            R.scale[nt][c] = __shfl_sync(kFull, scale, 4 * (2 * t4 + c));
            R.sees[nt][c] = mine < it.tokens ? keys_seen(p, it.ctx, it.n, mine) : 0;
            R.m[nt][c] = R.mo[nt][c] = -INFINITY;
            R.l[nt][c] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) R.o[nt][d][e] = 0.f;
    }
    R.near = QUANT;
    R.e_hi = -1;
    R.e_lo = 256;
    for (int j = first_page<QUANT>(warp, it.base); j < pages; j += Smem<QUANT>::kWarps) {
        if (!take_page<QUANT, NT>(R, load, p, kv_map, pieces, bar_piece, n, turn, (page0 + j) * kP, least, limit,
                                  recs + piece % kRecords, piece, lane, abort_flag))
            return false;
    }
    // Into the merge room.
    if (n > 0 && !warp_wait(bar_merged, (n - 1) & 1, abort_flag, p.status)) return false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float *dst = merge_o + (warp * kSmallRows + 8 * nt + 2 * t4) * kORow;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float sum = keys_sum(R.l[nt][c]);
            if (g == 0)
                merge_s[warp * kSmallRows + 8 * nt + 2 * t4 + c] =
                    make_float4(R.m[nt][c], sum, QUANT ? R.mo[nt][c] : R.m[nt][c], 0.f);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dim = QUANT ? 32 * (d >> 1) + 4 * g + 2 * (d & 1) + (e >> 1) : 16 * d + g + 8 * (e >> 1);
                dst[(e & 1) * kORow + dim] = R.o[nt][d][e];
            }
    }
    return true;
}

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
    const uint32_t bar_piece = bars + 8 * L::kTiles;   // [kRing] piece published; before them, the tiles' own
    const uint32_t bar_left = bar_piece + 8 * kRing;   // the page warps' results are in the merge room
    const uint32_t bar_merged = bar_left + 8;          // ... and read, and the piece's place is free
    const int warp = __shfl_sync(kFull, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;

    // What needs none of the call's data, while the kernel in front ends.
    if (threadIdx.x == 0) *abort_flag = 0;
    if (threadIdx.x < L::kNumBars)
        mbar_init(bars + 8 * threadIdx.x, threadIdx.x == (bar_left - bars) / 8 ? kWarps : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (!QUANT) {
        for (int e = threadIdx.x; e < kRecords; e += kThreads) recs[e].piece = -1;
        for (int e = threadIdx.x; e < kRecords * 3 * kD; e += kThreads)
            (&recs[e / (3 * kD)].first[0][0])[e % (3 * kD)] = 0xffffffffu;
    }
    // The second pass's kernel starts once every CTA of the first has let it,
    // which each does behind its own wait: what came before both is complete
    // when the second begins.  It waits for the first at its end alone.
    if (threadIdx.x == 0) prefetch_map(&kv_map);
    if (!p.second) wait_for_stream();
    let_next_start();
    if (!build_plan<256>(p, pl, blockIdx.x == 0)) {
        if (threadIdx.x == 0) p.cuts[blockIdx.x] = Cut{};
        wait_for_stream();
        return;
    }
    __syncthreads();  // (without it the loops below are compiled 7% slower: for warps that may have come apart)

    if (warp == kWarps) {
        // ------------------------------------ pieces, and what becomes of them --
        Walk walk;
        Cut cut = {};
        int x = 0, seq = 0, published = 0;
        bool more = true;
        if (lane == 0) walk.begin(p, pl, blockIdx.x);
        for (int n = 0;; ++n) {
            while (more && published < n + kRing) {
                if (lane == 0) {
                    Piece &it = pieces[published % kRing];
                    more = walk.next(p, it);
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
                    mbar_arrive(bar_piece + 8 * (published % kRing));
                    if (!more) p.cuts[blockIdx.x] = cut;
                }
                more = __shfl_sync(kFull, more, 0);
                ++published;
            }
            if (n == published - 1) break;  // the end's mark
            if (!warp_wait(bar_left, n & 1, abort_flag, p.status)) {
                // The combine reads every CTA's cut: where this one's is not
                // known yet, none.
                if (lane == 0 && more) p.cuts[blockIdx.x] = Cut{};
                break;
            }
            merge_piece<QUANT>(p, pieces[n % kRing], merge_o, merge_s, recs, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_merged);
        }
    } else {
        // ----------------------------------------------------- page warps --
        Loader<QUANT> load;
        load.begin(warp, lane, smem, bars);
        Turn<QUANT> turn;
        for (int n = 0;; ++n) {
            const Piece &it = pieces[n % kRing];
            if (!warp_wait(bar_piece + 8 * (n % kRing), (n / kRing) & 1, abort_flag, p.status)) break;
            if (it.row < 0) break;
            // (The rare case is not in the way of the other's registers.)
            const bool done = it.tokens * p.G > 8
                                  ? take_piece<QUANT, 2>(p, kv_map, pieces, bar_piece, n, load, turn, recs, merge_o, merge_s,
                                                         bar_merged, warp, lane, abort_flag)
                                  : take_piece<QUANT, 1>(p, kv_map, pieces, bar_piece, n, load, turn, recs, merge_o, merge_s,
                                                         bar_merged, warp, lane, abort_flag);
            if (!done) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_left);
        }
        load.drain();
    }
    // The kernel this one may have started beside is complete before it is.
    wait_for_stream();
}

template <bool QUANT>
int launch(const CUtensorMap &kv_map, const ChunkParams &p, cudaStream_t stream) {
    if (!allow_smem<2 + QUANT>(reinterpret_cast<const void *>(k3da_chunk_small_kernel<QUANT>), Smem<QUANT>::kBytes))
        return cuda_failed();
    return launch_beside(k3da_chunk_small_kernel<QUANT>, dim3(kCtas), Smem<QUANT>::kThreads, Smem<QUANT>::kBytes,
                         stream, kv_map, p);
}

}  // namespace

int launch_small(const ChunkParams &p, const void *kv_pool, bool quant, cudaStream_t stream) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    CUtensorMap kv_map;
    if (encode == nullptr || !pool_map(encode, &kv_map, kv_pool, p.num_pages, p.Hkv, quant, true)) return cuda_failed();
    return quant ? launch<true>(kv_map, p, stream) : launch<false>(kv_map, p, stream);
}

}  // namespace k3da_chunk
