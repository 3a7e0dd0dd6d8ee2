// k3da_chunk.cu -- attention of ragged chunks of new tokens over the paged
// cache (sm_103a): k3da_chunk_attn.
//
// For row i of request r's chunk and query head h (kv head g = h / G):
//   o = sum_c softmax_c(scale * q . k_c) v_c,   lse = log sum_c exp(scale * q . k_c)
// over the cache tokens c the mask shows: c <= ctx_r + i (causal), all
// ctx_r + n_r (full), or the ctx_r before the chunk (context).  A row that
// sees nothing gets o = 0 and lse = -inf.
//
// Work.  An item is a request, a kv head and 2 * tpt consecutive tokens of
// the chunk, tpt = floor(128 / G): two slots of up to 128 query rows (token
// major, the G heads of a token together), each one M = 128 accumulator.  An
// item's keys come in tiles of 128 (two pages).  All items are laid on one
// line, request by request, head by head, each as long as the keys its last
// row sees plus a constant, and the line is cut into equal slices, one a
// CTA: equal in keys and fixed costs together, whatever the lengths (a CTA
// with more items has a few tiles less).  An item that a cut falls into leaves partial results, which
// the combine kernel folds in order.  Each CTA finds its slice by itself: a
// scan over the requests, then closed forms.
//
// Chunks of at most 16 rows a kv head have a kernel of their own
// (k3da_chunk_small.cu); what follows is the others'.
//
// Both slots of an item read the same K/V tiles (shared).  An item whose
// tokens fit one slot (a draft block, a chunk's tail) gives its tiles to the
// two slots in turn (alternate), both with the same rows.
// Either way a slot's tile is worked on by two softmax warpgroups, one for
// each page: a thread has 64 scores of a row in registers.  The two share the
// row's running maximum (each leaves its page's in shared memory, and reads
// the other's) and one O.  Four softmax warps a scheduler hide each other's
// latencies; two (a slot's 128 columns in one thread) did not, and their
// unrolled code did not fit the instruction cache.
//
// Tensor memory holds three S of 128 columns for the two slots, taken in
// turn by the CTA's steps (a step: one slot's tile), P over its own S, and an
// O a slot.  The third S is Q K^T of the next step, ready when its slot has
// formed the last weights; and since the step after that has to wait for a P V
// of the other slot, the slots fall out of step by themselves: one forms
// weights, which the exponential units bound, while the other loads, looks for
// maxima and waits.
//
// The other warps: a scheduler that cuts the CTA's slice into pieces and
// loads Q, a K/V loader, an issuer of Q K^T, one of P V for each slot, and a
// few that prepare tiles (below).
//
// The preparing warps zero the V rows past an item's last key (stale slots
// may hold anything, and 0 * NaN is NaN), and where only some of an item's
// rows see a key, they take infinities and NaN out of that V row and record
// the first key that had one for each dim: what a row sees is always a prefix
// of the keys, so the epilogue puts them back for just the rows that see
// them.  Quantised tiles they widen to bf16 on the way (the scale is a power
// of two, so the bf16 are exact); both cache types share all the rest.
//
// Rounding: scores, softmax statistics and O are fp32 throughout (partials
// too); P is rounded to bf16 once for the P V product, the output once.
//
// Measured: 2048 tokens over 6144 (24/4 heads) bf16 106 us, 850 TFLOP/s; e4m3
// 135 us; 8192 over 8192 e4m3 784 us, 790 TFLOP/s.  Bound by issue slots (67%
// taken; 73% with codes) and the slots' chain: two slots' tile takes 2000
// cycles, its exponentials and its products 1024 each.  8 x 8 tokens over
// 16k to 131k bf16: 102.6 us, 5.6 TB/s of cache.  (0.7% of a prefill and 1% of
// this are the votes in which a warp agrees on its waits.)
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <cstring>

#include "cache_common.cuh"
#include "chunk_plan.cuh"
#include "k3da.h"
#include "sm103.cuh"
#include "tensor_maps.h"

namespace {

using namespace k3da_chunk;
using namespace sm103;

constexpr int kGroups = 4;         // softmax warpgroups: u has slot u / 2, page u % 2 of its tiles
constexpr int kRing = 4;           // pieces published ahead
constexpr int kRecords = 8;        // pieces whose non-finite records are alive at once
constexpr float kRescale = 8.0f;   // log2 units the running maximum may lag behind
// Warps: four softmax warpgroups, then single warps, then the preparing ones
// (widening codes takes more of them than looking tiles over).
constexpr int kLoadWarp = 16, kSchedWarp = 17, kQkWarp = 18, kPvWarp = 19, kPrepWarp = 21;
constexpr int kBufs = 3;           // S buffers
__host__ __device__ constexpr int prep_warps(bool quant) { return quant ? 7 : 3; }
__host__ __device__ constexpr int threads_of(bool quant) { return 32 * (kPrepWarp + prep_warps(quant)); }
// Registers a thread.  bf16: 768 threads launched with 80, 512 x 88 + 256 x
// 64; e4m3: 896 launched with 72, 512 x 88 + 384 x 48.
__host__ __device__ constexpr int softmax_regs(bool) { return 88; }
__host__ __device__ constexpr int other_regs(bool quant) { return quant ? 48 : 64; }
// Tensor memory columns of S buffer b (each page's P, 32 columns of bf16
// pairs, over the first half of its S) and of slot s's O.
__device__ __forceinline__ uint32_t col_s(int b) { return 128u * b; }
__device__ __forceinline__ uint32_t col_o(int s) { return 384u + 64u * s; }
constexpr uint32_t kTmemCols = 512u;
constexpr uint32_t kIdescQK = idesc_f16(128, kTile, false);
constexpr uint32_t kIdescPV = idesc_f16(128, kD, true);

// ----------------------------------------------------------- shared memory --

template <bool QUANT>
struct Smem {
    // bf16 tiles of K and of V.  V's are held until the weights of their keys
    // are formed, K's not, so that more of V leaves as many of both on their
    // way.  (Widened tiles are made together: the same of both.)
    static constexpr int kKs = QUANT ? 3 : 4, kVs = QUANT ? 3 : 6;
    static constexpr int kRaw = QUANT ? 4 : 0;     // quantised tiles: K codes, V codes, K scales, V scales
    static constexpr int kRawBytes = 2 * kTile * kD + 2 * kTile;
    static constexpr int kTileBytes = kTile * kD * 2;
    // Two halves: a shared item's slots, or two alternate items' Q in turn.
    static constexpr int kQBytes = kSlotRows * kD * 2;
    static constexpr int kQ = 0;
    static constexpr int kKv = kQ + 2 * kQBytes;
    static constexpr int kV = kKv + kKs * kTileBytes;
    static constexpr int kRawOff = kV + kVs * kTileBytes;
    static constexpr int kPlan = kRawOff + kRaw * kRawBytes;
    static constexpr int kRec = kPlan + static_cast<int>(sizeof(Plan));
    static constexpr int kXch = kRec + kRecords * static_cast<int>(sizeof(Records));
    static constexpr int kPieces = kXch + (5 * kGroups + 1) * kSlotRows * 4;
    static constexpr int kBars = kPieces + kRing * static_cast<int>(sizeof(Piece));
    static constexpr int kNumBars = 2 * kKs + 3 * kVs + 2 * kRaw + 2 * kRing + 4 + 7 * kBufs + 2 * 2 + 2;
    static constexpr int kTail = kBars + kNumBars * 8;  // TMEM address, abort flag
    static constexpr int kBytes = kTail + 16 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(kKv % 1024 == 0 && kRawOff % 128 == 0 && kPlan % 16 == 0 && kRec % 8 == 0 && kXch % 8 == 0 &&
                      kBars % 8 == 0,
                  "alignment");
};

// Keeps uses of loaded tensor memory behind the wait for it.
__device__ __forceinline__ void pin32(uint32_t *r) {
#pragma unroll
    for (int j = 0; j < 32; j += 8)
        asm volatile("" : "+r"(r[j]), "+r"(r[j + 1]), "+r"(r[j + 2]), "+r"(r[j + 3]), "+r"(r[j + 4]), "+r"(r[j + 5]),
                     "+r"(r[j + 6]), "+r"(r[j + 7]));
}

__device__ __forceinline__ void pin8(uint32_t *r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}

// Two e4m3 codes as bf16 times 2^-120: the sign, and the other seven bits
// where bf16's exponent ends.  BYTES (of prmt) extends two of the four bytes
// to halfwords, with their signs.
template <int BYTES>
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
    uint32_t h;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(h) : "r"(codes), "n"(BYTES));
    return (h * 16u) & 0x87f087f0u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Waits, with a limit, until a load that was issued has arrived.
__device__ __forceinline__ void land(uint32_t full, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(full, parity) && global_ns() - t0 < kWaitLimitNs) {
    }
}

// True where every lane of the (converged) warp says so.
__device__ __forceinline__ bool agreed(bool mine) { return __all_sync(kFull, mine); }

template <bool QUANT>
__global__ void __launch_bounds__(threads_of(QUANT), 1)
    k3da_chunk_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ ChunkParams p) {
    using L = Smem<QUANT>;
    constexpr int kThreads = threads_of(QUANT), kPrepWarps = prep_warps(QUANT);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // 1 KB aligned, and still known to be shared memory
    Plan *pl = reinterpret_cast<Plan *>(smem + L::kPlan);
    Records *recs = reinterpret_cast<Records *>(smem + L::kRec);
    // [2][kGroups][128] a page's row maximum and, above it, the tile it is of
    // (by the slot's count of tiles, and its parity).
    volatile unsigned long long *xmax = reinterpret_cast<unsigned long long *>(smem + L::kXch);
    float *xl = reinterpret_cast<float *>(smem + L::kXch) + 4 * kGroups * kSlotRows;  // [kGroups][128] shares of the row sums
    float *xm = xl + kGroups * kSlotRows;                     // [128] slot 1's base of the exponents
    Piece *pieces = reinterpret_cast<Piece *>(smem + L::kPieces);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kTail + 8);
    uint32_t *taddr_slot = reinterpret_cast<uint32_t *>(smem + L::kTail);
    const uint32_t bars = smem_u32(smem + L::kBars);
    const uint32_t bar_kfull = bars;                       // [kKs] K loaded (QUANT: unused, as the next two)
    const uint32_t bar_kempty = bar_kfull + 8 * L::kKs;    // [kKs] ... and multiplied
    const uint32_t bar_vfull = bar_kempty + 8 * L::kKs;    // [kVs] V loaded
    const uint32_t bar_prep = bar_vfull + 8 * L::kVs;      // [kVs] ... and prepared (QUANT: K too)
    const uint32_t bar_empty = bar_prep + 8 * L::kVs;      // [kVs] ... and multiplied by both slots that take it
    const uint32_t bar_rfull = bar_empty + 8 * L::kVs;     // [kRaw] quantised tile loaded
    const uint32_t bar_rempty = bar_rfull + 8 * L::kRaw;    // [kRaw] ... and widened
    const uint32_t bar_piece = bar_rempty + 8 * L::kRaw;    // [kRing] piece published
    const uint32_t bar_pdone = bar_piece + 8 * kRing;       // [kRing] ... and read by everybody
    const uint32_t bar_qfull = bar_pdone + 8 * kRing;       // [2] a half of the Q room filled
    const uint32_t bar_qempty = bar_qfull + 16;             // [2] ... and read
    // A slot's k-th tile has the barriers k % 3 of its own three: each side
    // then waits for every phase of the barriers it waits on, and none can be
    // two phases ahead (the slot's tile k + 3 needs the buffer of tile k).
    const uint32_t bar_sfull = bar_qempty + 16;             // [2][kBufs] S written
    const uint32_t bar_pfull = bar_sfull + 16 * kBufs;      // [2][kBufs] P written
    const uint32_t bar_bfree = bar_pfull + 16 * kBufs;      // [kBufs] P of the buffer read
    const uint32_t bar_pvdone = bar_bfree + 8 * kBufs;      // [2][kBufs] a slot's P V complete
    const uint32_t bar_ofree = bar_pvdone + 16 * kBufs;     // [2] an item's O read
    const uint32_t bar_sums = bar_ofree + 16;               // [2] both pages' row sums left
    const uint32_t bar_xch = bar_sums + 16;                 // slot 1's half of an alternate item is ready
    const uint32_t bar_done = bar_xch + 8;                  // every issuer's products are complete
    const int warp = __shfl_sync(kFull, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;

    // What needs none of the call's data, while the kernel in front ends.
    if (threadIdx.x == 0) *abort_flag = 0;
    if (threadIdx.x < L::kNumBars) {
        const uint32_t bar = bars + 8 * threadIdx.x;
        auto of = [&](uint32_t first, int n) { return bar >= first && bar < first + 8 * n; };
        const int count = of(bar_prep, L::kVs) || of(bar_rempty, L::kRaw) ? kPrepWarps
                          : of(bar_empty, L::kVs)                         ? 2
                          : of(bar_pdone, kRing)                          ? kThreads / 32 - 1  // every warp but the scheduler
                          : of(bar_pfull, 2 * kBufs) || of(bar_ofree, 2) || of(bar_sums, 2) || of(bar_xch, 1) ? 8
                          : of(bar_done, 1)                                                                   ? 3
                                                                                                              : 1;
        mbar_init(bar, count);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int e = threadIdx.x; e < kRecords; e += kThreads) recs[e].piece = -1;
    for (int e = threadIdx.x; e < 2 * kGroups * kSlotRows; e += kThreads) xmax[e] = ~0ull;  // of no tile
    for (int e = threadIdx.x; e < kRecords * 3 * kD; e += kThreads)
        (&recs[e / (3 * kD)].first[0][0])[e % (3 * kD)] = 0xffffffffu;
    // The second pass's kernel starts once every CTA of the first has let it,
    // which each does behind its own wait: what came before both is complete
    // when the second begins.  It waits for the first at its end alone.
    if (threadIdx.x == 0) {
        prefetch_map(&kv_map);
        prefetch_map(&q_map);
    }
    if (!p.second) wait_for_stream();
    let_next_start();
    if (!build_plan<512>(p, pl, blockIdx.x == 0)) {  // every chunk is small
        if (threadIdx.x == 0) p.cuts[blockIdx.x] = Cut{};
        wait_for_stream();
        return;
    }
    if (warp == kLoadWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(taddr_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *taddr_slot;
    bool alive = true;
    if (warp < 4 * kGroups) regs_raise<softmax_regs(QUANT)>();
    else regs_lower<other_regs(QUANT)>();

    if (warp == kSchedWarp) {
        // ---------------------------------------------- pieces and their Q --
        if (lane == 0) {
            Walk walk;
            walk.begin(p, pl, blockIdx.x);
            Cut cut = {};
            const uint32_t box = static_cast<uint32_t>(p.G) * p.tpt * 128;
            int seq = 0, base = 0, half = 0;
            uint32_t fills[2] = {0, 0};  // of each half of the Q room
            for (int n = 0; alive; ++n) {
                const int slot = n % kRing;
                if (!mbar_wait(bar_pdone + 8 * slot, ((n / kRing) & 1) ^ 1, abort_flag, p.status)) {
                    alive = false;
                    break;
                }
                Piece &it = pieces[slot];
                const bool more = walk.next(p, it);
                if (!more) it.row = -1;
                const bool tiles = more && it.t0 < it.t1;
                const int alt = it.alt, h = it.h, row = it.row;
                half = alt ? half ^ 1 : 0;
                it.seq = seq;
                it.base = base;
                it.q = half | (fills[0] & 1) << 1 | (fills[1] & 1) << 2;
                if (tiles) {
                    base += it.steps();
                    ++seq;
                }
                if (more && it.t0 > 0) cut.has[0] = 1;
                if (tiles && it.t0 == 0 && it.t1 < it.nt) {
                    cut.has[1] = 1;
                    cut.row = row;
                    cut.tokens = it.tokens;
                    cut.head = h;
                    cut.last = walk.slice_of(walk.start + walk.length - 1);
                }
                mbar_arrive(bar_piece + 8 * slot);
                if (!more) break;
                if (!tiles) continue;
                for (int s = 0; s < 2 && alive; ++s) {
                    if (alt && s != half) continue;
                    const uint32_t full = bar_qfull + 8 * s;
                    const uint32_t n_fills = s ? fills[1] : fills[0];
                    if (!mbar_wait(bar_qempty + 8 * s, (n_fills & 1) ^ 1, abort_flag, p.status)) {
                        alive = false;
                        break;
                    }
                    if (s) ++fills[1];
                    else ++fills[0];
                    mbar_arrive_expect_tx(full, box);
                    tma_load_3d(smem_u32(smem + L::kQ) + s * L::kQBytes, &q_map, 0, h * p.G,
                                row + (alt ? 0 : s * p.tpt), full);
                }
            }
            p.cuts[blockIdx.x] = cut;
            // Loads in flight land before the CTA leaves: the warps that use
            // them may give up, now or later.
            for (int s = 0; s < 2; ++s) {
                const uint32_t n_fills = s ? fills[1] : fills[0];
                if (n_fills > 0) land(bar_qfull + 8 * s, (n_fills - 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp < 4 * kGroups) {
        // ------------------------------------------------------ softmax --
        const int u = warp >> 2, s = u >> 1, page = u & 1;
        const int rho = threadIdx.x & (kSlotRows - 1);  // this thread's row of the slot
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const int ti = rho / p.G, gi = rho - ti * p.G;
        int k = 0;       // tiles of this slot so far
        uint32_t turn = 0, round = 0;  // k % kBufs, k / kBufs mod 2
        int sums = 0;    // pieces with tiles for it so far
        int merges = 0;  // alternate pieces with tiles for both slots so far
        for (int n = 0; alive; ++n) {
            const Piece &it = pieces[n % kRing];
            if (!agreed(mbar_wait(bar_piece + 8 * (n % kRing), (n / kRing) & 1, abort_flag, p.status))) break;
            if (it.row < 0) break;
            const int alt = it.alt;
            const int token = (alt ? 0 : s * p.tpt) + ti;  // in the item
            const bool row_valid = ti < p.tpt && token < it.tokens;
            const bool warp_valid = __any_sync(kFull, row_valid);
            const int sees = row_valid ? keys_seen(p, it.ctx, it.n, it.tok0 + token) : 0;
            const int least = keys_seen(p, it.ctx, it.n, it.tok0 + (alt ? 0 : s * p.tpt));  // ... of the slot's rows
            const int from = it.from(s), t_end = it.end(s), step = it.step();
            const bool mine = from < t_end;
            float m = -INFINITY, l = 0.f;
            const int shared_end = alt ? 0 : it.end(0);
            uint32_t buf = mine ? static_cast<uint32_t>(it.step_of(s, from)) % kBufs : 0;
            for (int t = from; t < t_end; t += step) {
                if (!agreed(mbar_wait(bar_sfull + 8 * (s * kBufs + turn), round, abort_flag, p.status))) {
                    alive = false;
                    break;
                }
                const uint32_t pfull = bar_pfull + 8 * (s * kBufs + turn);
                const uint32_t cols = lanes + col_s(buf) + kP * page;
                // The slot's next tile is two steps on, but one where slot 0
                // has none in between.
                buf += s == 0 || alt || t + 1 < shared_end ? 2 : 1;
                if (buf >= kBufs) buf -= kBufs;
                if (++turn == kBufs) {
                    turn = 0;
                    round ^= 1;
                }
                ++k;
                if (!warp_valid) {
                    // No row of this warp's: it only keeps step.
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pfull);
                    continue;
                }
                fence_after();
                const int key0 = t * kTile + kP * page;
                uint32_t x[kP];
                tmem_ld32(cols, x);
                tmem_ld32(cols + 32, x + 32);
                tmem_wait_ld();
                pin32(x);
                pin32(x + 32);
                if (page_masked(key0, least)) {
                    const int lim = sees - key0;
#pragma unroll
                    for (int j = 0; j < kP; ++j) x[j] = j < lim ? x[j] : 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) mx[j] = fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 4]));
#pragma unroll
                for (int j = 8; j < kP; j += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mx[q] = fmax3(mx[q], __uint_as_float(x[j + q]), __uint_as_float(x[j + 4 + q]));
                float rmax = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
                // The row's other page: its maximum.  A word of maximum and
                // tile number needs no barrier; the warp that has the other
                // page comes by at about the same time.  (A NaN is dropped
                // here and not from the scores: it reaches the row's sum.)
                {
                    volatile unsigned long long *leave = xmax + (k & 1) * kGroups * kSlotRows + rho;
                    leave[u * kSlotRows] = static_cast<unsigned long long>(k) << 32 | __float_as_uint(rmax);
                    unsigned long long got = leave[(u ^ 1) * kSlotRows];
                    if (static_cast<int>(got >> 32) != k) {
                        const unsigned long long t0 = global_ns();
                        do {
                            got = leave[(u ^ 1) * kSlotRows];
                        } while (static_cast<int>(got >> 32) != k && !*abort_flag && global_ns() - t0 < kWaitLimitNs);
                        if (static_cast<int>(got >> 32) != k) {
                            *abort_flag = 1;
                            if (p.status) atomicOr(p.status, K3DA_STATUS_TIMEOUT);
                        }
                    }
                    rmax = fmaxf(rmax, __uint_as_float(static_cast<uint32_t>(got)));
                }
                // The base of the exponents follows the row's maximum only
                // when that passes it by 2^8: P up to 256 is as exact, and O
                // is left alone.
                const bool first = t == from;
                const bool need = !first && rmax > m + kRescale;
                const float m_new = first || need ? rmax : m;
                const float m_eff = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet
                const float f = need ? exp2_approx(m - m_eff) : 1.f;
                m = m_new;
                if (__any_sync(kFull, need)) {
                    // A row's two threads scale one half of its O each, once
                    // the slot's last P V is complete.
                    const uint32_t last = k - 2;
                    if (!agreed(mbar_wait(bar_pvdone + 8 * (s * kBufs + last % kBufs), last / kBufs & 1,
                                                           abort_flag, p.status))) {
                        alive = false;
                        break;
                    }
                    fence_after();
#pragma unroll 1
                    for (int d0 = 32 * page; d0 < 32 * page + 32; d0 += 8) {
                        uint32_t o[8];
                        tmem_ld8(lanes + col_o(s) + d0, o);
                        tmem_wait_ld();
                        pin8(o);
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st8(lanes + col_o(s) + d0, o);
                    }
                }
                const unsigned long long sl2 = pack_f32x2(p.scale_log2, p.scale_log2);
                const unsigned long long nm2 = pack_f32x2(-m_eff, -m_eff);
                unsigned long long sum[2] = {0ull, 0ull};
                // Weights of 32 keys at a time, in stages of independent
                // operations.
#pragma unroll
                for (int j = 0; j < kP; j += 32) {
                    unsigned long long e[16];
                    uint32_t pk[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        e[q] = fma_f32x2(pack_f32x2(__uint_as_float(x[j + 2 * q]), __uint_as_float(x[j + 2 * q + 1])), sl2, nm2);
#pragma unroll
                    for (int q = 0; q < 16; ++q) e[q] = exp2_f32x2(e[q]);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float2 w = unpack_f32x2(e[q]);
                        pk[q] = pack2(w.x, w.y);
                        sum[q & 1] = add_f32x2(sum[q & 1], e[q]);
                    }
                    tmem_st16(cols + j / 2, pk);
                }
                const float2 tot = unpack_f32x2(add_f32x2(sum[0], sum[1]));
                l = l * f + (tot.x + tot.y);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull);
            }
            if (!alive) break;
            // ------------------------------------------------- epilogue --
            if (mine) {
                const uint32_t last = k - 1;
                if (!agreed(mbar_wait(bar_pvdone + 8 * (s * kBufs + last % kBufs), last / kBufs & 1, abort_flag, p.status)))
                    break;
                xl[u * kSlotRows + rho] = l;
                if (s == 1 && page == 0) xm[rho] = m;
            }
            const int next = n % kRing;
            if (alt && s == 1) {
                // Slot 0 merges: its warps own the same tensor memory lanes.
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (mine) mbar_arrive(bar_xch);
                    mbar_arrive(bar_pdone + 8 * next);
                }
                continue;
            }
            if (mine) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_sums + 8 * s);
                if (!agreed(mbar_wait(bar_sums + 8 * s, sums & 1, abort_flag, p.status))) break;
                ++sums;
                l = xl[2 * s * kSlotRows + rho] + xl[(2 * s + 1) * kSlotRows + rho];
            }
            const bool both = alt && it.from(1) < it.end(1);
            float wa = 1.f, wb = 0.f;
            if (both) {
                if (!agreed(mbar_wait(bar_xch, merges & 1, abort_flag, p.status))) break;
                ++merges;
                const float mb = xm[rho], lb = xl[2 * kSlotRows + rho] + xl[3 * kSlotRows + rho];
                const float mt = fmaxf(m, mb);
                const float me = mt == -INFINITY ? 0.f : mt;
                wa = exp2_approx(m - me);
                wb = exp2_approx(mb - me);
                l = l * wa + lb * wb;
                m = mt;
            }
            fence_after();
            const bool whole = it.t0 == 0 && it.t1 == it.nt;
            const float norm = whole ? 1.f / l : 1.f;
            const int row = it.row + token;
            const int head = it.h * p.G + gi;
            const int part = (blockIdx.x * 2 + (it.t0 > 0 ? 0 : 1)) * 2 * kSlotRows + s * kSlotRows + rho;
            const int piece = it.seq;
            const Records &rec = recs[piece % kRecords];
            const bool dirty = mine && rec.piece == piece;
            const int common = keys_seen(p, it.ctx, it.n, it.tok0);  // keys every row of the item sees
            if (page == 0 && row_valid) {
                if (!whole) p.part_ml[part] = make_float2(m, l);
                else if (p.lse)
                    p.lse[static_cast<long long>(row) * p.Hq + head] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            }
            // Half of the dims each, 8 at a time: the registers are the main
            // loop's.
#pragma unroll 1
            for (int d0 = 32 * page; d0 < 32 * page + 32; d0 += 8) {
                uint32_t o[8];
                if (mine) {
                    tmem_ld8(lanes + col_o(s) + d0, o);
                    tmem_wait_ld();
                    pin8(o);
                    if (both) {
                        uint32_t ob[8];
                        tmem_ld8(lanes + col_o(1) + d0, ob);
                        tmem_wait_ld();
                        pin8(ob);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * wa + __uint_as_float(ob[j]) * wb);
                    }
                }
                if (!row_valid) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[j]) * norm);
                if (dirty) {
                    const uint32_t tag = ~static_cast<uint32_t>(piece) << 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
#pragma unroll 1
                        for (int q = 0; q < 3; ++q) {
                            const uint32_t e = rec.first[q][d0 + j];
                            if ((e & 0xffffff00u) != tag || common + static_cast<int>(e & 0xffu) >= sees) continue;
                            o[j] = q == 2 ? 0x7fffffffu : __float_as_uint(__uint_as_float(o[j]) + (q == 0 ? INFINITY : -INFINITY));
                        }
                    }
                }
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(o[j]);
                // Each row is another line: a store takes a cycle a thread,
                // whatever it brings.
                if (whole) {
                    *reinterpret_cast<uint4 *>(p.out + (static_cast<long long>(row) * p.Hq + head) * kD + d0) =
                        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                } else {
                    store32(p.part_o + static_cast<long long>(part) * kD + d0, v);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if (mine) mbar_arrive(bar_ofree + 8 * s);
                if (both) mbar_arrive(bar_ofree + 8);
                mbar_arrive(bar_pdone + 8 * next);
            }
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------ K/V loads --
        constexpr int kPageTile = kP * kD * (QUANT ? 1 : 2);  // bytes of a page's K or V of one head
        uint64_t again, once;  // pages are read again where the request has more items
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        int issued[2] = {0, 0};  // tiles of K (codes: of both), of V
        const bool issuer = elect_one();
        for (int n = 0; alive; ++n) {
            const Piece &it = pieces[n % kRing];
            if (!agreed(mbar_wait(bar_piece + 8 * (n % kRing), (n / kRing) & 1, abort_flag, p.status))) break;
            if (it.row < 0) break;
            const int t0 = it.t0, t1 = it.t1, pages = min((it.limit + kP - 1) / kP, 2 * t1), r = it.r, h = it.h;
            // 32 pages at a time, one a lane: row of its K, -1 where the id
            // is no page, -2 past the item's last key.  The next ones are
            // asked for half way.
            auto rows_at = [&](int t) {
                const int pg = 2 * t + lane;
                if (pg >= pages) return -2;
                const long long page = page_of(p.page_table, p.page_stride, p.num_pages, r, pg * kP);
                return page < 0 ? -1 : static_cast<int>((page * 2 * p.Hkv + h) * kP);
            };
            int mine = -2, next = t0 < t1 ? rows_at(t0) : -2;
            const uint64_t policy = it.n <= 2 * p.tpt ? once : again;
            for (int t = t0; t < t1; ++t) {
                const int ahead = (t - t0) & 15;
                if (ahead == 0) mine = next;
                if (ahead == 8) next = rows_at(t + 8);
                // K, then V (codes: both, with their scales, in one place).
#pragma unroll
                for (int part = 0; part < (QUANT ? 1 : 2); ++part) {
                    const int ring = QUANT ? L::kRaw : part ? L::kVs : L::kKs, x = issued[part], st = x % ring;
                    const uint32_t full = (QUANT ? bar_rfull : part ? bar_vfull : bar_kfull) + 8 * st;
                    if (!agreed(mbar_wait((QUANT ? bar_rempty : part ? bar_empty : bar_kempty) + 8 * st, ((x / ring) & 1) ^ 1,
                                          abort_flag, p.status))) {
                        alive = false;
                        break;
                    }
                    uint8_t *dst = smem + (QUANT ? L::kRawOff + st * L::kRawBytes
                                                 : (part ? L::kV : L::kKv) + st * L::kTileBytes);
                    uint32_t bytes = 0;
                    int krow[2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        krow[half] = __shfl_sync(kFull, mine, 2 * ahead + half);
                        if (krow[half] >= 0) bytes += QUANT ? 2 * kPageTile + 2 * kP : kPageTile;
                        if (krow[half] == -1) {
                            if (lane == 0 && p.status) atomicOr(p.status, K3DA_STATUS_BAD_PAGE);
                            for (int e = lane; e < kPageTile / 16; e += 32) {
                                reinterpret_cast<uint4 *>(dst + half * kPageTile)[e] = make_uint4(0, 0, 0, 0);
                                if (QUANT) reinterpret_cast<uint4 *>(dst + (2 + half) * kPageTile)[e] = make_uint4(0, 0, 0, 0);
                            }
                            if (QUANT)
                                for (int e = lane; e < kP; e += 32)
                                    dst[4 * kPageTile + half * kP + e] = dst[4 * kPageTile + (2 + half) * kP + e] = 0;
                            fence_proxy_async();
                        }
                    }
                    __syncwarp();
                    if (issuer) {
                        if (bytes > 0) mbar_arrive_expect_tx(full, bytes);
                        else mbar_arrive(full);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (krow[half] < 0) continue;
                            const int vrow = krow[half] + p.Hkv * kP;
                            tma_load_2d(smem_u32(dst + half * kPageTile), &kv_map, 0, part ? vrow : krow[half], full, policy);
                            if (QUANT) {
                                tma_load_2d(smem_u32(dst + (2 + half) * kPageTile), &kv_map, 0, vrow, full, policy);
                                bulk_load(smem_u32(dst + 4 * kPageTile + half * kP), p.scales + krow[half], kP, full);
                                bulk_load(smem_u32(dst + 4 * kPageTile + (2 + half) * kP), p.scales + vrow, kP, full);
                            }
                        }
                    }
                    __syncwarp();
                    ++issued[part];
                }
                if (!alive) break;
            }
            if (!alive) break;
            if (lane == 0) mbar_arrive(bar_pdone + 8 * (n % kRing));
        }
        // Loads in flight land before the CTA leaves, as the scheduler's do.
        auto land_ring = [&](uint32_t full, int ring, int x) {
            for (int j = x > ring ? x - ring : 0; j < x; ++j) land(full + 8 * (j % ring), (j / ring) & 1);
        };
        land_ring(QUANT ? bar_rfull : bar_kfull, QUANT ? L::kRaw : L::kKs, issued[0]);
        if (!QUANT) land_ring(bar_vfull, L::kVs, issued[1]);
    } else if (warp < kPrepWarp) {
        // ------------------------------------------------------ products --
        // One warp issues Q K^T of every step, one P V of each slot.
        const bool is_qk = warp == kQkWarp;
        const int s = is_qk ? 0 : warp - kPvWarp;
        const bool issuer = elect_one();
        const int stages = is_qk ? L::kKs : L::kVs;
        int st = 0;       // the tile's stage
        uint32_t ph = 0;  // ... and how often the stages have come round, mod 2
        int items = 0;    // pieces with tiles for the slot so far
        uint32_t k[2] = {0, 0};  // tiles of each slot so far
        const uint32_t tiles = smem_u32(smem + (is_qk ? L::kKv : L::kV));
        for (int n = 0; alive; ++n) {
            const Piece &it = pieces[n % kRing];
            if (!agreed(mbar_wait(bar_piece + 8 * (n % kRing), (n / kRing) & 1, abort_flag, p.status))) break;
            if (it.row < 0) break;
            const int t0 = it.t0, t1 = it.t1, alt = it.alt;
            const int from = it.from(s), t_end = it.end(s), step = it.step();
            const int half = it.q & 1;
            const uint64_t qd = desc_sw128(smem_u32(smem + L::kQ) + half * L::kQBytes);
            if (is_qk && t0 < t1) {
                if ((!alt || half == 0) && !agreed(mbar_wait(bar_qfull, it.q >> 1 & 1, abort_flag, p.status))) break;
                if ((!alt || half == 1) && !agreed(mbar_wait(bar_qfull + 8, it.q >> 2 & 1, abort_flag, p.status))) break;
            }
            items += from < t_end;
            int next = from;  // the slot's next tile
            uint32_t i = it.base;
            // (Nothing in this loop is an operation of the whole warp: its
            // lanes agree behind it.)
            for (int t = t0; t < t1; ++t) {
                // Every tile in turn, another slot's too: a phase is never
                // waited for before the one before it is known to be over.
                if (!mbar_wait((QUANT || !is_qk ? bar_prep : bar_kfull) + 8 * st, ph, abort_flag, p.status)) {
                    alive = false;
                    break;
                }
                if (is_qk) {
                    const uint64_t kd = desc_sw128(tiles + st * L::kTileBytes);
                    // An alternate item's slots have the same Q.
                    for (int slot = alt || t >= t_end ? 1 : 0; slot < 2; ++slot, ++i) {
                        const uint32_t round = i / kBufs, buf = i - round * kBufs;
                        if (round > 0 && !mbar_wait(bar_bfree + 8 * buf, (round & 1) ^ 1, abort_flag, p.status)) {
                            alive = false;
                            break;
                        }
                        fence_after();
                        if (issuer) {
                            const uint64_t q = qd + (alt ? 0 : (slot * L::kQBytes) >> 4);
#pragma unroll
                            for (int kk = 0; kk < kD / 16; ++kk)
                                mma_ss(tmem + col_s(buf), q + ((kk * 32) >> 4), kd + ((kk * 32) >> 4), kIdescQK,
                                       kk > 0 ? 1u : 0u);
                            const int of = alt ? (t - t0) & 1 : slot;
                            const uint32_t turn = of * kBufs + (of ? k[1] : k[0]) % kBufs;
                            mma_commit(bar_sfull + 8 * turn);
                            if (!QUANT && slot == 1) mma_commit(bar_kempty + 8 * st);
                        }
                        if (alt ? (t - t0) & 1 : slot) ++k[1];
                        else ++k[0];
                    }
                    if (!alive) break;
                } else if (t == next && t < t_end) {
                    next += step;
                    const uint32_t buf = static_cast<uint32_t>(it.step_of(s, t)) % kBufs;
                    const uint32_t round = k[0] / kBufs, turn = s * kBufs + k[0] - round * kBufs;
                    ++k[0];
                    if (!mbar_wait(bar_pfull + 8 * turn, round & 1, abort_flag, p.status) ||
                        (t == from && items > 1 && !mbar_wait(bar_ofree + 8 * s, items & 1, abort_flag, p.status))) {
                        alive = false;
                        break;
                    }
                    fence_after();
                    if (issuer) {
                        const uint64_t vd = desc_sw128(tiles + st * L::kTileBytes);
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma_ts(tmem + col_o(s), tmem + col_s(buf) + 8 * kk + (kk >= 4 ? 32 : 0), vd + ((kk * 2048) >> 4),
                                   kIdescPV, (kk > 0 || t != from) ? 1u : 0u);
                        mma_commit(bar_bfree + 8 * buf);
                        mma_commit(bar_pvdone + 8 * turn);
                        mma_commit(bar_empty + 8 * st);
                    }
                } else if (lane == 0) {
                    mbar_arrive(bar_empty + 8 * st);
                }
                if (++st == stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            alive = agreed(alive);
            if (!alive) break;
            if (is_qk && t0 < t1) {
                // Q is free once the products that read it are complete.
                fence_after();
                if (issuer) {
                    mma_commit(bar_qempty + 8 * half);
                    if (!alt) mma_commit(bar_qempty + 8);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_pdone + 8 * (n % kRing));
        }
        // Every product and its signals complete before the CTA leaves.
        fence_after();
        if (issuer) mma_commit(bar_done);
        __syncwarp();
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(bar_done, 0) && global_ns() - t0 < kWaitLimitNs) {
        }
    } else {
        // -------------------------------------------------- preparation --
        const int tid = threadIdx.x - 32 * kPrepWarp;
        int st = 0, rs = 0;
        uint32_t ph = 0, rph = 0;  // rounds of the stages, mod 2
        for (int n = 0; alive; ++n) {
            const Piece &it = pieces[n % kRing];
            if (!agreed(mbar_wait(bar_piece + 8 * (n % kRing), (n / kRing) & 1, abort_flag, p.status))) break;
            if (it.row < 0) break;
            const int piece = it.seq, limit = it.limit, t1 = it.t1;
            Records *rec = recs + piece % kRecords;
            const uint32_t tag = ~static_cast<uint32_t>(piece) << 8;
            const int least = keys_seen(p, it.ctx, it.n, it.tok0);  // keys that every row of the item sees
            for (int t = it.t0; t < t1; ++t) {
                uint8_t *vt = smem + L::kV + st * L::kTileBytes;
                if (QUANT) {
                    const uint8_t *raw = smem + L::kRawOff + rs * L::kRawBytes;
                    alive = agreed(mbar_wait(bar_rfull + 8 * rs, rph, abort_flag, p.status) &&
                                   mbar_wait(bar_empty + 8 * st, ph ^ 1, abort_flag, p.status));
                    if (!alive) break;
                    // 1024 pieces of 16 codes (K's 512, then V's), four a
                    // row; loads of a few of them first.
                    constexpr int kStep = 32 * kPrepWarps, kBatch = 3;
                    for (int c0 = tid; c0 < 1024; c0 += kBatch * kStep) {
                        uint4 w[kBatch];
                        uint32_t sc[kBatch];
#pragma unroll
                        for (int e = 0; e < kBatch; ++e) {
                            const int c = c0 + e * kStep;
                            if (c >= 1024) break;
                            w[e] = *reinterpret_cast<const uint4 *>(raw + c * 16);
                            sc[e] = raw[2 * kTile * kD + (c >> 2)];
                        }
#pragma unroll
                        for (int e = 0; e < kBatch; ++e) {
                            const int c = c0 + e * kStep;
                            if (c >= 1024) break;
                            const uint32_t b = sc[e];
                            const bool is_v = c >= 512;
                            const int row = (c & 511) >> 2, quarter = c & 3;
                            // 2^120 times the scale, in two factors where it
                            // passes bf16's range (rows above 448 * 2^7).
                            const uint32_t e1 = b <= 134u ? b + 120u : 254u;
                            const uint32_t mul = e1 << 7 | e1 << 23;
                            const uint32_t in[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
                            uint32_t o[8];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                o[2 * q] = mul_bf16x2(widen2<0x9180>(in[q]), mul);
                                o[2 * q + 1] = mul_bf16x2(widen2<0xb3a2>(in[q]), mul);
                            }
                            const int key = t * kTile + row;
                            if (b > 134u || (is_v && key >= limit)) {
                                const uint32_t mul2 = (b - 7u) << 7 | (b - 7u) << 23;
                                const bool hidden = is_v && (key >= limit || (b == 255u && key >= least));
#pragma unroll
                                for (int q = 0; q < 8; ++q)
                                    o[q] = hidden ? 0u : b == 255u ? 0x7fff7fffu : mul_bf16x2(o[q], mul2);
                                if (hidden && key < limit) {
                                    for (int d = 0; d < 16; ++d)
                                        atomicMin(&rec->first[2][quarter * 16 + d], tag | (key - least));
                                    rec->piece = piece;
                                }
                            }
                            uint8_t *dst = is_v ? vt : smem + L::kKv + st * L::kTileBytes;
                            *reinterpret_cast<uint4 *>(dst + swz(row, 2 * quarter)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(dst + swz(row, 2 * quarter + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    }
                    fence_proxy_async();
                } else {
                    alive = agreed(mbar_wait(bar_vfull + 8 * st, ph, abort_flag, p.status));
                    if (!alive) break;
                    if ((t + 1) * static_cast<long long>(kTile) > least) {
                        for (int row = tid; row < kTile; row += 32 * kPrepWarps) {
                            const int key = t * kTile + row;
                            if (key < least) continue;
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint4 *at = reinterpret_cast<uint4 *>(vt + swz(row, c));
                                if (key >= limit) {
                                    *at = make_uint4(0, 0, 0, 0);
                                    continue;
                                }
                                const uint4 w = *at;
                                uint32_t v[4] = {w.x, w.y, w.z, w.w};
                                bool bad = false;
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    bad |= (v[q] & 0x7f80u) == 0x7f80u || (v[q] & 0x7f800000u) == 0x7f800000u;
                                if (!bad) continue;
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    const uint32_t e = v[q >> 1] >> (16 * (q & 1)) & 0xffffu;
                                    if ((e & 0x7f80u) != 0x7f80u) continue;
                                    const int kind = e & 0x7fu ? 2 : e >> 15;
                                    atomicMin(&rec->first[kind][8 * c + q], tag | (key - least));
                                    v[q >> 1] &= q & 1 ? 0x0000ffffu : 0xffff0000u;
                                }
                                *at = make_uint4(v[0], v[1], v[2], v[3]);
                                rec->piece = piece;
                            }
                        }
                        fence_proxy_async();
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_prep + 8 * st);
                    if (QUANT) mbar_arrive(bar_rempty + 8 * rs);
                }
                if (++st == L::kVs) {
                    st = 0;
                    ph ^= 1;
                }
                if (QUANT && ++rs == L::kRaw) {
                    rs = 0;
                    rph ^= 1;
                }
            }
            if (!alive) break;
            if (lane == 0) mbar_arrive(bar_pdone + 8 * (n % kRing));
        }
    }

    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kLoadWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    // The kernel this one may have started beside is complete before it is.
    wait_for_stream();
}

// ----------------------------------------------------------------- combine --
//
// Folds the partial results of the items that a cut of the line fell into,
// in the order of their pieces.  CTA (x, y) takes `rows` rows of the x-th such
// item of a pass, the few-rows kernel's first (y < small_y): 16 threads a row
// (4 dims each) times `lanes` piece lanes, lane i folding the pieces i,
// i + lanes, ...; one lane where there are few pieces (a long chunk: many
// rows, two or three pieces), eight where one item spreads over many CTAs.
constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads)
    k3da_chunk_combine_kernel(const __grid_constant__ ChunkParams small, const __grid_constant__ ChunkParams large,
                              int small_y, int small_rows, int large_rows) {
    __shared__ int votes[kCombineThreads / 32];
    __shared__ int owner;
    __shared__ Cut cut;
    __shared__ bool continues[kCtas];  // the CTA's first piece belongs to an item begun before
    __shared__ float4 part[8][32];
    __shared__ float2 part_ml[8][2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool is_small = static_cast<int>(blockIdx.y) < small_y;
    const ChunkParams &p = is_small ? small : large;
    const int y = is_small ? blockIdx.y : blockIdx.y - small_y, rows = is_small ? small_rows : large_rows;
    let_next_start();
    wait_for_stream();
    // The x-th CTA that left an item unfinished.
    static_assert(kCtas <= kCombineThreads, "one CTA a thread");
    // Every cut is read at once: what follows depends on nothing but them.
    Cut mine = {};
    if (tid < kCtas) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.cuts + tid);
        const uint4 c[2] = {src[0], src[1]};
        std::memcpy(&mine, c, sizeof mine);
        continues[tid] = mine.has[0];
    }
    const bool cut_here = tid < kCtas && mine.has[1];
    const unsigned vote = __ballot_sync(kFull, cut_here);
    if (lane == 0) votes[warp] = __popc(vote);
    if (tid == 0) owner = -1;
    __syncthreads();
    int rank = __popc(vote & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) rank += votes[w];
    if (cut_here && rank == static_cast<int>(blockIdx.x)) {
        owner = tid;
        cut = mine;
    }
    __syncthreads();
    const int a = owner;
    if (a < 0 || !cut_fits(cut, a, p.T, p.Hkv, 2 * p.tpt)) return;
    const int pieces = cut.last - a + 1;
    const int lanes = pieces > 8 ? 8 : 1;
    const int dim = tid & 15;
    const int pl = lanes == 8 ? (tid >> 4) & 7 : 0;
    const int per_pass = kCombineThreads / 16 / lanes;
    const int slot_rows = p.tpt * p.G;
    for (int base = 0; base < rows; base += per_pass) {
        const int local = lanes == 8 ? tid >> 7 : tid >> 4;
        const int rho = y * rows + base + local;  // the item's row, slot by slot
        const int s = rho / kSlotRows, in_slot = rho % kSlotRows;
        const int token = s * p.tpt + in_slot / p.G;
        const bool valid = base + local < rows && rho < p.part_rows && in_slot < slot_rows && token < cut.tokens;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (valid) {
            constexpr int kFold = 4;  // pieces whose loads are in flight together
            for (int j = pl; j < pieces; j += lanes * kFold) {
                float2 ml[kFold];
                float4 v[kFold];
#pragma unroll
                for (int q = 0; q < kFold; ++q) {
                    const int i = j + q * lanes;
                    ml[q] = make_float2(-INFINITY, 0.f);
                    v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i >= pieces || (i > 0 && !continues[a + i])) continue;
                    const long long at = (static_cast<long long>(a + i) * 2 + (i == 0 ? 1 : 0)) * p.part_rows + rho;
                    ml[q] = p.part_ml[at];
                    v[q] = reinterpret_cast<const float4 *>(p.part_o + at * kD)[dim];
                }
#pragma unroll
                for (int q = 0; q < kFold; ++q) {
                    const float mt = fmaxf(m, ml[q].x);
                    const float me = mt == -INFINITY ? 0.f : mt;
                    const float f = exp2_approx(m - me), g = exp2_approx(ml[q].x - me);
                    l = l * f + ml[q].y * g;
                    o.x = o.x * f + v[q].x * g;
                    o.y = o.y * f + v[q].y * g;
                    o.z = o.z * f + v[q].z * g;
                    o.w = o.w * f + v[q].w * g;
                    m = mt;
                }
            }
        }
        if (lanes == 8) {
            part[pl][tid & 15 | (tid >> 7) << 4] = o;
            if (dim == 0) part_ml[pl][tid >> 7] = make_float2(m, l);
            __syncthreads();
            if (pl == 0) {
                for (int q = 1; q < 8; ++q) {
                    const float2 ml = part_ml[q][tid >> 7];
                    const float4 v = part[q][tid & 15 | (tid >> 7) << 4];
                    const float mt = fmaxf(m, ml.x);
                    const float me = mt == -INFINITY ? 0.f : mt;
                    const float f = exp2_approx(m - me), g = exp2_approx(ml.x - me);
                    l = l * f + ml.y * g;
                    o.x = o.x * f + v.x * g;
                    o.y = o.y * f + v.y * g;
                    o.z = o.z * f + v.z * g;
                    o.w = o.w * f + v.w * g;
                    m = mt;
                }
            }
            __syncthreads();
        }
        if (valid && pl == 0) {
            const float norm = 1.f / l;
            const long long at = static_cast<long long>(cut.row + token) * p.Hq + cut.head * p.G + in_slot % p.G;
            uint2 w = make_uint2(0, 0);
            if (l != 0.f) w = make_uint2(pack2(o.x * norm, o.y * norm), pack2(o.z * norm, o.w * norm));
            reinterpret_cast<uint2 *>(p.out + at * kD)[dim] = w;
            if (dim == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
    }
}

// -------------------------------------------------------------------- host --

template <bool QUANT>
int launch_kernel(const CUtensorMap &kv_map, const CUtensorMap &q_map, const ChunkParams &prm, cudaStream_t st) {
    if (!allow_smem<QUANT>(reinterpret_cast<const void *>(k3da_chunk_kernel<QUANT>), Smem<QUANT>::kBytes))
        return cuda_failed();
    return launch_beside(k3da_chunk_kernel<QUANT>, dim3(kCtas), threads_of(QUANT), Smem<QUANT>::kBytes, st, kv_map,
                         q_map, prm);
}

int launch_long(const ChunkParams &prm, const void *q, const void *kv_pool, bool quant, cudaStream_t st) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    CUtensorMap kv_map, q_map;
    if (encode == nullptr || !pool_map(encode, &kv_map, kv_pool, prm.num_pages, prm.Hkv, quant, !quant)) return cuda_failed();
    const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(prm.Hq), static_cast<cuuint64_t>(prm.T)};
    const cuuint64_t strides[2] = {kD * 2, static_cast<cuuint64_t>(prm.q_stride) * 2};
    const cuuint32_t box[3] = {kD, static_cast<cuuint32_t>(prm.G), static_cast<cuuint32_t>(prm.tpt)};
    const cuuint32_t estrides[3] = {1, 1, 1};
    if (encode(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estrides,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cuda_failed();
    return quant ? launch_kernel<true>(kv_map, q_map, prm, st) : launch_kernel<false>(kv_map, q_map, prm, st);
}

}  // namespace

extern "C" size_t k3da_chunk_workspace_bytes(int num_tokens, int num_requests, int num_q_heads, int num_kv_heads,
                                             int page_stride) {
    if (num_tokens < 0 || num_requests < 1 || num_requests > kMaxRequests || !heads_ok(num_q_heads, num_kv_heads) ||
        page_stride < 1 || page_stride > kMaxPageStride)
        return 0;
    return kWorkspace;
}

extern "C" int k3da_chunk_attn(void *out, float *lse, const void *q, int64_t q_row_stride, int num_tokens,
                               const void *kv_pool, int cache_dtype, const void *kv_scales, int64_t num_pages,
                               const int32_t *page_table, int page_stride, const int32_t *ctx_lens,
                               const int32_t *cu_seqlens, int num_requests, int num_q_heads, int num_kv_heads,
                               int head_dim, int mask, float softmax_scale, void *workspace,
                               size_t workspace_bytes, int32_t *status, void *stream) {
    const int rc = check_cache(kv_pool, cache_dtype, kv_scales, num_pages, page_table, page_stride, ctx_lens,
                               cu_seqlens, num_requests, num_tokens, num_kv_heads, head_dim, status);
    if (rc != K3DA_OK) return rc;
    if (!heads_ok(num_q_heads, num_kv_heads)) return K3DA_EUNSUPPORTED;
    if (mask != K3DA_MASK_CAUSAL && mask != K3DA_MASK_FULL && mask != K3DA_MASK_CONTEXT) return K3DA_EINVAL;
    if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return K3DA_EINVAL;
    if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(lse, 4)) return K3DA_EINVAL;
    const int64_t width = static_cast<int64_t>(num_q_heads) * kD;
    if (q_row_stride < width || q_row_stride % 8 != 0 || q_row_stride > (1LL << 31)) return K3DA_EINVAL;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < kWorkspace) return K3DA_EWORKSPACE;
    if (num_tokens == 0) return K3DA_OK;
    if (!out || !q) return K3DA_EINVAL;
    const size_t tokens = static_cast<size_t>(num_tokens), ints = sizeof(int32_t);
    const Span spans[] = {{out, tokens * width * 2},
                          {lse, tokens * num_q_heads * sizeof(float)},
                          {workspace, kWorkspace},
                          {q, ((tokens - 1) * q_row_stride + width) * 2},
                          {kv_pool, pool_bytes(num_pages, num_kv_heads, cache_dtype)},
                          {kv_scales, scale_bytes(num_pages, num_kv_heads)},
                          {page_table, table_bytes(num_requests, page_stride)},
                          {ctx_lens, num_requests * ints},
                          {cu_seqlens, (num_requests + 1) * ints},
                          {status, ints}};
    if (written_overlap(spans, 3, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;

    ChunkParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.out = static_cast<__nv_bfloat16 *>(out);
    prm.lse = lse;
    prm.scales = static_cast<const uint8_t *>(kv_scales);
    prm.page_table = page_table;
    prm.ctx_lens = ctx_lens;
    prm.cu_seqlens = cu_seqlens;
    prm.status = status;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    auto parts_at = [](ChunkParams &q, uint8_t *at, int rows) {
        q.part_rows = rows;
        q.cuts = reinterpret_cast<Cut *>(at);
        q.part_ml = reinterpret_cast<float2 *>(at + kCutBytes);
        q.part_o = reinterpret_cast<float *>(at + kCutBytes + static_cast<size_t>(kCtas) * 2 * rows * sizeof(float2));
    };
    parts_at(prm, ws, 2 * kSlotRows);
    prm.q = static_cast<const __nv_bfloat16 *>(q);
    prm.q_stride = q_row_stride;
    prm.num_pages = num_pages;
    prm.page_stride = page_stride;
    prm.R = num_requests;
    prm.T = num_tokens;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.G = num_q_heads / num_kv_heads;
    prm.tpt = kSlotRows / prm.G;
    prm.mask = mask;
    prm.scale_log2 = softmax_scale * 1.4426950408889634f;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool quant = cache_dtype == K3DA_CACHE_E4M3;
    // Which requests are small is known to the kernels alone; that none can
    // be long is known from the number of tokens.  A call whose caches are
    // small, whatever their lengths, is bound by latency: one kernel for all
    // (8 x 6 tokens over up to 2041, 6/1 heads: 13.7 us, with both 15.8; what the
    // small kernel gains on 64 x 8000 keys a head, 80 us with codes and 2 with
    // bf16, comes to those 2 us at 55000 keys of codes, 2 million of bf16).
    const long long heads = static_cast<long long>(num_requests) * num_kv_heads;
    const long long keys = heads * page_stride * kP;
    const bool can_be_long = num_tokens > kSmallRows || num_tokens * prm.G > kSmallRows;
    const bool one_kernel = can_be_long && keys <= 75000;
    prm.pass = one_kernel ? kAll : kLong;
    ChunkParams small = prm;
    small.pass = kSmall;
    parts_at(small, ws + part_bytes(2 * kSlotRows), kSmallRows);
    // The pass that is more likely to have the work goes first: an empty one
    // behind it starts where SMs fall free.
    const bool small_first = num_tokens <= static_cast<long long>(num_requests) * (kSmallRows / prm.G);
    for (int i = 0; i < 2; ++i) {
        const bool is_small = (i == 0) == small_first;
        if (is_small ? one_kernel : !can_be_long) continue;
        (is_small ? small : prm).second = i == 1 && can_be_long && !one_kernel;
        const int launched = is_small ? launch_small(small, kv_pool, quant, st) : launch_long(prm, q, kv_pool, quant, st);
        if (launched != K3DA_OK) return launched;
    }
    // Where all there can be fits one slice, nothing is cut (a token over 300:
    // 7.2 instead of 8.6 us).
    const long long line = keys + heads * (kSmallOverhead + 2 * prm.tpt + kSmallRows);
    if (!can_be_long && line < 2 * kMinSmallSlice) return K3DA_OK;
    // Items a cut can fall into, rows one can have: a grid of about 1200 CTAs
    // over the long chunks' (8 x 8 tokens over long contexts: 102.6 us; with
    // half as many 5 more, with twice as many the same), 600 over the others'.
    const long long items =
        ((static_cast<long long>(num_tokens) + 2 * prm.tpt - 1) / (2 * prm.tpt) + num_requests) * num_kv_heads;
    const unsigned gx = static_cast<unsigned>(items < kCtas ? items : kCtas);
    auto rows_of = [&](int bound, int ctas) {
        const int rows = static_cast<int>((bound * gx + ctas - 1) / ctas);
        return rows < 2 ? 2 : rows;
    };
    const int rows_bound = num_tokens <= prm.tpt ? num_tokens * prm.G : 2 * kSlotRows;
    const int small_rows = rows_of(kSmallRows, 608), rows = rows_of(rows_bound, 1216);
    const int small_y = one_kernel ? 0 : (kSmallRows + small_rows - 1) / small_rows;
    const int y = can_be_long ? (rows_bound + rows - 1) / rows : 0;
    return launch_beside(k3da_chunk_combine_kernel, dim3(gx, static_cast<unsigned>(small_y + y)), kCombineThreads, 0, st,
                         small, prm, small_y, small_rows, rows);
}
