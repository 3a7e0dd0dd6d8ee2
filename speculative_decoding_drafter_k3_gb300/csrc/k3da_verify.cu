// k3da_verify.cu -- probabilities of logits and the verification of drafted
// tokens (sm_103a): k3da_token_probs and k3da_verify.
//
// Drafted tokens are kept by rejection: draft d, drawn from q, stays with
// probability min(1, p(d) / q(d)); where one is rejected the next token is
// drawn from max(p - q, 0), and behind the last draft from p.  What comes out
// is then distributed as p's own tokens.
//
// Drawing is the smallest index whose running sum passes a uniform share of
// the total.  Running sums of rounded numbers depend on their order, and with
// it the token would (in 0.4% of draws from 128,003 words in fp32); so weights are whole multiples of 2^-40 here, summed in
// 64 bits: any split of a row over threads gives the same token.  A weight
// below 2^-40 counts as nothing; a vocabulary of 2^18 words so loses less than
// 2^-22 (of weights that add up to 1; of a difference p - q with a small sum that
// is a larger part).  The share itself has 24 bits, what a uniform fp32 number
// is sure to have: each word is met to 2^-24 of the total, and one of less may never
// be drawn.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "cache_common.cuh"
#include "k3da.h"

namespace {

using namespace k3da_cache;

typedef unsigned long long u64;

constexpr int kMaxVocab = 1 << 22;  // 2^22 weights of at most 2^40: sums stay below 2^63
constexpr long long kMaxRowStride = 1LL << 31;
constexpr int kMaxBlocks = 1 << 24;  // requests of a verification

using k3da_cache::load_here;

__device__ __forceinline__ float load_here(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// ----------------------------------------------------------- probabilities --
//
// Bound by memory: 2 (or 4) bytes in and 4 out for each logit, and each is
// read once.  A row is held in the registers of a cluster of up to 8 CTAs
// (64 logits a thread, packed as they came; of longer rows the last part is,
// and the others come from the L2 again): the largest and the sum of the
// weights below it are first each thread's own, then joined, and between the
// CTAs with one exchange.  Weights are formed twice, for the sum and for the
// result: as fp32 they would take twice the registers, and CTAs of 256
// threads, four on an SM, hide each other's waits (512 threads: 59 us instead of
// 43, three on an SM 48).  301 rows of 128,003 in bf16: 43.7 us, 5.2 TB/s, 0.77 of
// what a copy gets; a CTA's 9.5 us are 2.9 of loading, 1.6 of arithmetic, 3 of
// reducing and waiting for the cluster's others, 1.9 of storing.
//
// Rows begin anywhere (an odd vocabulary).  A thread's 8 logits are those that
// lie on 32 aligned bytes of probs, so that it stores whole sectors; their own 16
// (or 32) bytes are then off by the same step in all of a row, and are put
// together from aligned blocks of two neighbouring lanes.

constexpr int kProbThreads = 256;
constexpr int kFewThreads = 64;  // for vocabularies of up to 1017
constexpr int kMaxCluster = 8;

struct ProbParams {
    float *probs;
    const void *logits;
    const float *temperatures;
    const int32_t *cu_seqlens;
    int32_t *status;
    long long probs_stride, logits_stride;
    int R, T, V;
    int cluster;
};

// Half of what turns a distance below the row's largest logit into a power of
// two, log2(e) / temperature, as the sum of two floats, both above 0: -inf stays
// -inf, and products that leave fp32's range leave it on the same side.  (EXACT:
// used as such; else their sum, rounded once.)  At an infinite temperature the
// longest distance still counts 2^-20.
struct Slope {
    float hi, lo;
};
template <bool EXACT>
__device__ __forceinline__ Slope half_slope(float temperature) {
    constexpr float kHi = 0x1.715470p-1f, kLo = 0x1.94ae0cp-23f;  // log2(e) / 2: hi is so far below it that lo is never below 0
    const float t = fmaxf(temperature, 0x1p-126f), r = __frcp_rn(t);
    const float e = __fmaf_rn(-r, t, 1.0f);  // 1/t = r + r e
    Slope s;
    s.hi = __fmul_rn(kHi, r);
    s.lo = __fadd_rn(__fmaf_rn(kHi, r, -s.hi), __fmaf_rn(s.hi, e, __fmul_rn(kLo, r)));
    s.lo = fmaxf(s.lo, 0x1p-149f);  // (infinity: no number so far)
    s.hi = EXACT ? fmaxf(s.hi, 0x1p-149f) : __fadd_rn(s.hi, s.lo);
    return s;
}

__device__ __forceinline__ float larger(float a, float b) {  // NaN if one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two floats at a time.
typedef u64 Pair;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both_of(Pair v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Square roots of the weights exp((x - top) / temperature) of two logits, for a
// finite `top`: with half the slope the hardware's power of two gives no
// subnormal, and the square rounds those that the result has; its error
// (2^-22) counts twice.  -inf, and a difference that passes fp32's range, give 0.
// What is rounded in front of that: the exponent; the difference, which is exact
// for 16-bit logits of about the same size; and for those the slope.  With fp32
// (EXACT) that is made up for by its low part, an instruction a logit: 16-bit logits
// with it 46.2 us instead of 43.6 (301 rows of 128,003).
template <bool EXACT>
__device__ __forceinline__ Pair roots(Pair x, float top, Slope half) {
    const Pair d = add2(x, pair_of(-top, -top)), hi = pair_of(half.hi, half.hi);
    float2 e = both_of(EXACT ? fma2(d, hi, mul2(d, pair_of(half.lo, half.lo))) : mul2(d, hi));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    return pair_of(e.x, e.y);
}

// A type of logits: 8 of them are kWords words.  two(): the i-th two as
// floats; top(): the largest so far, kept as it came.
template <typename L>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int kWords = 8, kPerWord = 1;
    static constexpr uint32_t kNone = 0xff800000u;  // -inf
    static __device__ __forceinline__ Pair two(const uint32_t *w, int i) {
        return pair_of(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    static __device__ __forceinline__ uint32_t top(uint32_t a, uint32_t b) {
        return __float_as_uint(larger(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float top_of(uint32_t a) { return __uint_as_float(a); }
    static __device__ __forceinline__ uint32_t bits(const float *p) { return __float_as_uint(load_here(p)); }
};
template <>
struct Logits<__nv_bfloat16> {
    static constexpr int kWords = 4, kPerWord = 2;
    static constexpr uint32_t kNone = 0xff80ff80u;
    static __device__ __forceinline__ Pair two(const uint32_t *w, int i) { return pair_of(bf16_lo(w[i]), bf16_hi(w[i])); }
    static __device__ __forceinline__ uint32_t top(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float top_of(uint32_t a) { return larger(bf16_lo(a), bf16_hi(a)); }
    static __device__ __forceinline__ uint32_t bits(const __nv_bfloat16 *p) {
        uint16_t v;
        asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
        return v;
    }
};
template <>
struct Logits<__half> {
    static constexpr int kWords = 4, kPerWord = 2;
    static constexpr uint32_t kNone = 0xfc00fc00u;
    static __device__ __forceinline__ float2 floats(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
    static __device__ __forceinline__ Pair two(const uint32_t *w, int i) {
        const float2 f = floats(w[i]);
        return pair_of(f.x, f.y);
    }
    static __device__ __forceinline__ uint32_t top(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float top_of(uint32_t a) {
        const float2 f = floats(a);
        return larger(f.x, f.y);
    }
    static __device__ __forceinline__ uint32_t bits(const __half *p) {
        uint16_t v;
        asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
        return v;
    }
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const char *p) {
    if constexpr (N == 4) {
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    } else {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    }
}

// N words that begin `shift` bytes into w and next.
template <int N>
__device__ __forceinline__ void realign(uint32_t (&w)[N], const uint32_t (&next)[N], int shift) {
    uint32_t x[2 * N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        x[k] = w[k];
        x[N + k] = next[k];
    }
#pragma unroll
    for (int step = N / 2; step > 0; step /= 2)
#pragma unroll
        for (int k = 0; k < N + step; ++k)
            if (k + step < 2 * N) x[k] = shift & (4 * step) ? x[k + step] : x[k];
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __funnelshift_r(x[k], x[k + 1], 8 * (shift & 3));
}

// Of a part of the row: its largest logit, and the sum of the weights relative
// to that, or, where the temperature is 0, the first place it stands at.
struct Stat {
    float top;
    union {
        float sum;
        int at;
    };
};
__device__ __forceinline__ float finite(float top) { return fmaxf(top, -3.402823466e38f); }
// Bit for bit the same if a and b change places: two lanes that join each
// other's get one result, and so all threads of the row do.  (Contracted, one
// of the products would not be rounded, and equal logits would differ by the
// thread that holds them.)
template <bool EXACT>
__device__ __forceinline__ Stat join(Stat a, Stat b, bool greedy, Slope half) {
    Stat r;
    r.top = larger(a.top, b.top);
    if (greedy) {
        r.at = min(a.top == r.top ? a.at : INT_MAX, b.top == r.top ? b.at : INT_MAX);
        return r;
    }
    const Pair e = roots<EXACT>(pair_of(a.top, b.top), finite(r.top), half);
    const float2 w = both_of(mul2(e, e));
    r.sum = __fadd_rn(__fmul_rn(a.sum, a.top == r.top ? 1.f : w.x), __fmul_rn(b.sum, b.top == r.top ? 1.f : w.y));
    return r;
}

// Every CTA of the cluster gets every CTA's v (index: its rank).
__device__ __forceinline__ void exchange(Stat v, Stat *all, int cluster) {
    if (threadIdx.x < cluster)
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(shared_of(all + cluster_rank(), threadIdx.x)),
                     "r"(__float_as_int(v.top)), "r"(v.at)
                     : "memory");
    cluster_arrive();
    cluster_wait();
}

template <typename L, int K, int THREADS>
__global__ void __launch_bounds__(THREADS, (K * Logits<L>::kWords == 8 ? 5 : 4) * (kProbThreads / THREADS))
    k3da_token_probs_kernel(const __grid_constant__ ProbParams p) {
    using X = Logits<L>;
    constexpr int kWarps = THREADS / 32;
    constexpr int kWords = X::kWords;
    constexpr bool kExact = X::kPerWord == 1;
    __shared__ Stat part[kWarps];
    __shared__ Stat all[kMaxCluster];
    __shared__ float owner[2];  // 1 where the row is some request's, and its temperature
    if (p.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, rank = static_cast<int>(cluster_rank());
    const int t = static_cast<int>(blockIdx.x) / p.cluster;
    const L *in = static_cast<const L *>(p.logits) + t * p.logits_stride;
    float *out = p.probs + t * p.probs_stride;
    // Chunk j is elements 8 j - lead .. 8 j - lead + 7.
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(out) & 31) / 4;
    const int chunks = (p.V + lead + 7) / 8;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(in) - lead * sizeof(L)) & (4 * kWords - 1));
    const int back = shift / static_cast<int>(sizeof(L));
    const int warps = p.cluster * kWarps;
    const int each = (chunks + 32 * warps - 1) / (32 * warps);  // a lane's chunks, K at a time
    const int tiles = (each + K - 1) / K;
    const int e0 = 8 * ((rank * kWarps + (tid >> 5)) * each * 32 + lane) - lead;  // the lane's first element
    if (tid == 0) owner[0] = 0.f;
    __syncthreads();
    wait_for_stream();

    auto inside = [&](int e) { return e >= 0 && e + 8 <= p.V; };
    uint32_t x[K + 1][kWords];
    // A block of the row's aligned memory is read if all of it is the row's.
    // (Lane 0 has the block behind the tile's last one, too.)
    auto load_tile = [&](int tile) {
        const int e = e0 - back + 256 * K * tile, n = each - K * tile;
        const char *at = reinterpret_cast<const char *>(in + e);
#pragma unroll
        for (int k = 0; k <= K; ++k) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) x[k][w] = X::kNone;
            if (((k < K && k < n) || (k <= n && lane == 0 && shift != 0)) && inside(e + 256 * k))
                load_words(x[k], at + 256 * sizeof(L) * k);
        }
    };
    // Then its logits, -inf where none are.
    auto place_tile = [&](int tile) {
        const int e1 = e0 + 256 * K * tile, n = min(K, each - K * tile);
        if (shift != 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint32_t next[kWords];
#pragma unroll
                for (int w = 0; w < kWords; ++w)  // lane 31's next block is lane 0's of the chunks after
                    next[w] = __shfl_sync(kFull, lane == 0 ? x[k + 1][w] : x[k][w], (lane + 1) & 31);
                realign(x[k], next, shift);
            }
        }
        // What reaches over the row's ends, one by one: in the warps that have one.
        const int warp_e = e1 - back - 8 * lane;
        if (warp_e >= 0 && warp_e + 256 * n + 8 <= p.V) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = e1 + 256 * k;
            if (k >= n || (inside(e - back) && (shift == 0 || inside(e - back + 8)))) continue;
#pragma unroll
            for (int w = 0; w < kWords; ++w) x[k][w] = X::kNone;
            if (e >= p.V) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e + i >= 0 && e + i < p.V) {
                    const uint32_t b = X::bits(in + e + i);
                    if (X::kPerWord == 1) x[k][i % kWords] = b;
                    else x[k][i / 2] = i & 1 ? (x[k][i / 2] & 0xffffu) | b << 16 : (x[k][i / 2] & 0xffff0000u) | b;
                }
        }
    };

    load_tile(0);
    // Whose row it is.
    for (int e = tid; e < p.R; e += THREADS) {
        const int a = load_here(p.cu_seqlens + e), b = load_here(p.cu_seqlens + e + 1);
        const float temperature = p.temperatures ? load_here(p.temperatures + e) : 1.0f;
        if (a <= t && t < b) {
            owner[0] = 1.f;
            owner[1] = temperature;
        }
    }
    __syncthreads();
    if (p.cluster > 1) cluster_wait();  // all of the cluster's CTAs run
    if (owner[0] == 0.f) return;        // all CTAs of the row alike
    const bool greedy = !(owner[1] > 0.f);
    const Slope half = half_slope<kExact>(greedy ? 1.0f : owner[1]);

    Stat s;
    s.top = -INFINITY;
    s.at = greedy ? INT_MAX : 0;
    for (int tile = 0; tile < tiles; ++tile) {
        if (tile > 0) load_tile(tile);
        place_tile(tile);
        const int n = each - K * tile;
        uint32_t most = X::kNone;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k < n) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) most = X::top(most, x[k][w]);
            }
        Stat mine;
        mine.top = X::top_of(most);
        if (greedy || mine.top == INFINITY) {
            int count = 0, at = INT_MAX;
#pragma unroll
            for (int k = K - 1; k >= 0; --k)
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    const float2 f = both_of(X::two(x[k], i));
                    const int e = e0 + 256 * (K * tile + k) + 2 * i;
                    if (k < n && f.y == mine.top) ++count, at = e + 1;
                    if (k < n && f.x == mine.top) ++count, at = e;
                }
            if (greedy) mine.at = at;
            else mine.sum = static_cast<float>(count);
        } else {
            const float ref = finite(mine.top);
            Pair sum = pair_of(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k < n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const Pair e = roots<kExact>(X::two(x[k], i), ref, half);
                        sum = fma2(e, e, sum);
                    }
                }
            mine.sum = both_of(sum).x + both_of(sum).y;
        }
        s = tiles == 1 ? mine : join<kExact>(s, mine, greedy, half);
    }
    auto from_lane = [&](int o) {
        Stat y;
        y.top = __shfl_xor_sync(kFull, s.top, o);
        y.at = __shfl_xor_sync(kFull, s.at, o);
        return y;
    };
    for (int o = 16; o > 0; o >>= 1) s = join<kExact>(s, from_lane(o), greedy, half);
    if (lane == 0) part[tid >> 5] = s;
    __syncthreads();
    s = part[lane & (kWarps - 1)];
    for (int o = kWarps / 2; o > 0; o >>= 1) s = join<kExact>(s, from_lane(o), greedy, half);
    if (p.cluster > 1) {
        exchange(s, all, p.cluster);
        s = all[0];
        for (int c = 1; c < p.cluster; ++c) s = join<kExact>(s, all[c], greedy, half);
    }

    const float top = s.top;
    const bool nothing = top == -INFINITY, none = top != top;
    if (p.status && tid == 0 && rank == 0 && (nothing || none)) atomicOr(p.status, K3DA_STATUS_BAD_TOKEN);
    // value(two logits, the first one's index): two results.  The last tile is
    // still there.
    auto store = [&](auto value) {
        for (int tile = tiles - 1; tile >= 0; --tile) {
            if (tile < tiles - 1) {
                load_tile(tile);
                place_tile(tile);
            }
            const int e1 = e0 + 256 * K * tile, n = each - K * tile;
            float *to = out + e1;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int e = e1 + 256 * k;
                if (k >= n || e >= p.V) continue;
                Pair v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = value(X::two(x[k], i), e + 2 * i);
                if (inside(e)) {
                    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(to + 256 * k), "l"(v[0]), "l"(v[1]),
                                 "l"(v[2]), "l"(v[3])
                                 : "memory");
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (e + i >= 0 && e + i < p.V) to[256 * k + i] = i & 1 ? both_of(v[i / 2]).y : both_of(v[i / 2]).x;
                }
            }
        }
    };
    if (!greedy && top < INFINITY && !nothing) {
        const float scale = 1.0f / s.sum;
        const Pair inv = pair_of(scale, scale);
        store([&](Pair f, int) {
            const Pair e = roots<kExact>(f, top, half);
            return mul2(mul2(e, e), inv);
        });
        return;
    }
    // One value at one place, or at every +inf, and another elsewhere.
    const float most = none ? __int_as_float(0x7fffffff) : nothing ? 0.f : greedy ? 1.f : 1.0f / s.sum;
    const float rest = none ? most : 0.f;
    const int at = greedy ? s.at : -1;
    store([&](Pair f, int e) {
        const float2 g = both_of(f);
        return greedy ? pair_of(e == at ? most : rest, e + 1 == at ? most : rest)
                      : pair_of(g.x == top ? most : rest, g.y == top ? most : rest);
    });
}

// ------------------------------------------------------------ verification --
//
// Bound by memory where there are many requests: two rows (p and q) where a
// draft is rejected, one where none is, each read once but for the stretch
// that the token is in.  A cluster of up to 8 CTAs has a request: all of them
// find the row (a chain of four round trips: rows, tokens, probabilities,
// row), each sums a part of the vocabulary, and after one exchange the one
// that has the token narrows its part down.  64 blocks of up to 8 over 128,003
// words: 13.8 us for 46 MB (6.8 at the copy rate); one block of 6 over 32,768: 4.0,
// which is the chain.

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kAhead = 16;  // loads of a lane in flight, of p and of q (8: 14.2 us, 4: 16.6)
constexpr int kLast = 8;    // elements of a thread in the last step

struct VerifyParams {
    void *out_tokens;
    int32_t *num_out;
    const void *tokens;
    const float *target, *draft;
    const float *uniforms;
    const int32_t *cu_seqlens;
    int32_t *status;
    long long target_stride, draft_stride;
    int R, T, V;
    int token_i64;
    int cluster;
};

__device__ __forceinline__ long long token_at(const VerifyParams &p, int row) {
    if (!p.token_i64) return load_here(static_cast<const int32_t *>(p.tokens) + row);
    long long v;
    asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(static_cast<const long long *>(p.tokens) + row));
    return v;
}
__device__ __forceinline__ void put_token(const VerifyParams &p, int row, long long v) {
    if (p.token_i64) static_cast<long long *>(p.out_tokens)[row] = v;
    else static_cast<int32_t *>(p.out_tokens)[row] = static_cast<int32_t>(v);
}

// p - q as a probability: 0 below 0 and for what is no number, at most 1.
__device__ __forceinline__ float above(float p, float q) {
    float r;
    asm("sub.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(p), "f"(q));
    return r;
}

// floor(2^40 x) of x in [0, 1], summed over up to 256 of them: added, rounding
// down, to 2^6, whose last place is 2^-17, x leaves its first 17 places in the
// sum's mantissa, and the rest of x, added to 2^-17, the next 23.  (As a
// conversion to 64 bits it took the fp64 pipe half of the time: 24.5 us instead
// of 17.9 for 64 x 8 rows of 128,003.)
struct Wholes {
    uint32_t high = 0, low = 0;
    __device__ __forceinline__ void add(float x) {
        const float h = __fadd_rd(x, 0x1p6f);
        const float l = __fadd_rd(x - (h - 0x1p6f), 0x1p-17f);
        high += __float_as_uint(h) - 0x42800000u;  // 2^6
        low += __float_as_uint(l) - 0x37000000u;   // 2^-17
    }
    __device__ __forceinline__ u64 sum() const { return (static_cast<u64>(high) << 23) + low; }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__global__ void __launch_bounds__(kVerifyThreads, 4) k3da_verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ u64 part[kVerifyWarps];
    __shared__ u64 all[2][kMaxCluster];
    __shared__ int rejected;
    const int cluster = p.cluster, r = static_cast<int>(blockIdx.x) / cluster;
    if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    wait_for_stream();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = static_cast<int>(cluster_rank());
    const int a = load_here(p.cu_seqlens + r), b = load_here(p.cu_seqlens + r + 1);
    const bool good = a >= 0 && b > a && b <= p.T;
    // The first draft that is rejected; the last row where none is.
    if (tid == 0) rejected = b - a - 1;
    __syncthreads();
    if (cluster > 1) cluster_wait();  // all of the cluster's CTAs run
    if (!good) {
        if (tid == 0 && rank == 0) {
            p.num_out[r] = 0;
            if (a != b && p.status) atomicOr(p.status, K3DA_STATUS_BAD_LENGTH);
        }
        return;
    }
    for (int i = tid; i < b - a - 1; i += kVerifyThreads) {
        const long long d = token_at(p, a + i + 1);
        const float u = load_here(p.uniforms + a + i);
        bool yes = false;
        if (d >= 0 && d < p.V) {
            const float pd = load_here(p.target + (a + i) * p.target_stride + d);
            const float qd = p.draft ? load_here(p.draft + (a + i) * p.draft_stride + d) : 1.0f;
            yes = static_cast<double>(u) * qd < static_cast<double>(pd);  // both sides exact
        } else if (p.status) {
            atomicOr(p.status, K3DA_STATUS_BAD_TOKEN);
        }
        if (!yes) atomicMin(&rejected, i);
    }
    __syncthreads();
    const int kept = rejected;
    const float *pt = p.target + (a + kept) * p.target_stride;
    const float *qt = p.draft && kept < b - a - 1 ? p.draft + (a + kept) * p.draft_stride : nullptr;
    const long long spent = !p.draft && kept < b - a - 1 ? token_at(p, a + kept + 1) : -1;
    const float u = load_here(p.uniforms + b - 1);
    const u64 share = static_cast<u64>(fminf(fmaxf(u, 0.f), 0x0.ffffffp0f) * 0x1p24f);

    // N weights of elements v, v + step, ..., below hi.
    bool residual = kept < b - a - 1;
    auto weights = [&](auto &w, int v, int step, int hi) {
        constexpr int N = sizeof w / sizeof w[0];
        float g[N];
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = v + k * step < hi ? load_here(pt + v + k * step) : 0.f;
        if (residual && qt) {
#pragma unroll
            for (int k = 0; k < N; ++k) g[k] = v + k * step < hi ? load_here(qt + v + k * step) : 0.f;
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) g[k] = residual && v + k * step == spent ? 2.f : 0.f;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = above(w[k], g[k]);
    };
    // Each warp's sum over its eighth of [lo, hi), into part.
    auto eighth = [&](int lo, int hi) { return (hi - lo + 32 * kVerifyWarps - 1) / (32 * kVerifyWarps) * 32; };
    auto sum_eighths = [&](int lo, int hi) {
        const int length = eighth(lo, hi), from = min(hi, lo + warp * length), to = min(hi, from + length);
        u64 sum = 0;
        for (int v = from + lane; v < to; v += 32 * kAhead) {
            float w[kAhead];
            weights(w, v, 32, to);
            Wholes some;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) some.add(w[k]);
            sum += some.sum();
        }
        sum = warp_sum(sum);
        if (lane == 0) part[warp] = sum;
        __syncthreads();
    };
    const int each = (p.V + 32 * cluster - 1) / (32 * cluster) * 32;
    int lo = min(p.V, rank * each), hi = min(p.V, lo + each);
    u64 total, mine, before;
    for (int turn = 0;; ++turn) {
        sum_eighths(lo, hi);
        mine = 0;
        for (int k = 0; k < kVerifyWarps; ++k) mine += part[k];
        total = mine;
        before = 0;
        if (cluster > 1) {
            if (tid < cluster)
                asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(shared_of(&all[turn][rank], tid)), "l"(mine) : "memory");
            cluster_arrive();
            cluster_wait();
            total = 0;
            for (int c = 0; c < cluster; ++c) {
                if (c < rank) before += all[turn][c];
                total += all[turn][c];
            }
        }
        if (total != 0 || !residual) break;
        residual = false;  // nothing is left of p - q: from p itself
        __syncthreads();
    }
    if (rank == 0) {
        for (int i = tid; i < b - a; i += kVerifyThreads)
            if (i != kept) put_token(p, a + i, i < kept ? token_at(p, a + i + 1) : -1);
        if (tid == 0) p.num_out[r] = kept + 1;
        if (tid == 0 && total == 0) {
            put_token(p, a + kept, -1);
            if (p.status) atomicOr(p.status, K3DA_STATUS_BAD_TOKEN);
        }
    }
    const u64 at = __umul64hi(total, share << 40);
    if (total == 0 || at < before || at >= before + mine) return;
    // The eighth that the token is in, its eighth, and so on.
    for (;;) {
        const int length = eighth(lo, hi);
        int k = 0;
        while (k < kVerifyWarps - 1 && before + part[k] <= at) before += part[k++];
        lo += k * length;
        hi = min(hi, lo + length);
        if (hi - lo <= kVerifyThreads * kLast) break;
        __syncthreads();
        sum_eighths(lo, hi);
    }
    float w[kLast];
    weights(w, lo + tid * kLast, 1, hi);
    Wholes all_of_them;
#pragma unroll
    for (int i = 0; i < kLast; ++i) all_of_them.add(w[i]);
    const u64 own = all_of_them.sum();
    u64 run = own;
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(kFull, run, o);
        if (lane >= o) run += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = run;
    __syncthreads();
    for (int k = 0; k < warp; ++k) before += part[k];
    before += run - own;
    if (at < before || at >= before + own) return;
    int k = 0;
#pragma unroll
    for (int i = 0; i < kLast; ++i) {
        Wholes one;
        one.add(w[i]);
        before += one.sum();
        k += before <= at ? 1 : 0;
    }
    put_token(p, a + kept, lo + tid * kLast + k);
}

// -------------------------------------------------------------------- host --

inline size_t row_bytes(int rows, long long stride, int row, int size) {
    return rows == 0 ? 0 : (static_cast<size_t>(rows - 1) * stride + row) * size;
}

inline int check_rows(const int32_t *cu_seqlens, int R, int most, int T, int V, const int32_t *status) {
    if (!cu_seqlens || !aligned_to(cu_seqlens, 4) || !aligned_to(status, 4)) return K3DA_EINVAL;
    if (R < 1 || R > most || T < 0 || V < 1 || V > kMaxVocab) return K3DA_EINVAL;
    return K3DA_OK;
}

// CTAs of a row: as many as its registers take, more where there are few rows.
template <typename L>
int launch_probs(ProbParams &prm, cudaStream_t st) {
    constexpr int kMost = 32 / Logits<L>::kWords;  // chunks that a thread holds
    const int chunks = (prm.V + 14) / 8;
    if (chunks <= 2 * kFewThreads) {  // 8000 rows of 1000 (one request): 16.8 us, 34.8 with 256 threads
        prm.cluster = 1;
        return launch_clusters(k3da_token_probs_kernel<L, 2, kFewThreads>, dim3(static_cast<unsigned>(prm.T)), 1, kFewThreads, st,
                               prm);
    }
    const int rounds = (chunks + kProbThreads - 1) / kProbThreads;  // chunks of a thread of one CTA
    int cluster = 1;
    while (cluster < kMaxCluster && (rounds > kMost * cluster || (rounds > cluster && prm.T * cluster < 2 * 152))) cluster *= 2;
    if (prm.T > INT_MAX / cluster) return K3DA_EINVAL;
    prm.cluster = cluster;
    const dim3 grid(static_cast<unsigned>(prm.T * cluster));
    if (rounds > 2 * cluster)
        return launch_clusters(k3da_token_probs_kernel<L, kMost, kProbThreads>, grid, cluster, kProbThreads, st, prm);
    return launch_clusters(k3da_token_probs_kernel<L, 2, kProbThreads>, grid, cluster, kProbThreads, st, prm);
}

inline bool stride_ok(int64_t stride, int V, int T) {
    return stride >= V && stride <= kMaxRowStride && stride <= (1LL << 48) / (T + 1LL);
}

}  // namespace

extern "C" int k3da_token_probs(float *probs, int64_t probs_row_stride, const void *logits, int logits_dtype,
                                int64_t logits_row_stride, int num_tokens, int vocab, const float *temperatures,
                                const int32_t *cu_seqlens, int num_requests, int32_t *status, void *stream) {
    const int rc = check_rows(cu_seqlens, num_requests, kMaxRequests, num_tokens, vocab, status);
    if (rc != K3DA_OK) return rc;
    if (logits_dtype != K3DA_LOGITS_BF16 && logits_dtype != K3DA_LOGITS_FP16 && logits_dtype != K3DA_LOGITS_FP32)
        return K3DA_EINVAL;
    const int size = logits_dtype == K3DA_LOGITS_FP32 ? 4 : 2;
    if (!aligned_to(probs, 4) || !aligned_to(logits, size) || !aligned_to(temperatures, 4)) return K3DA_EINVAL;
    if (!stride_ok(probs_row_stride, vocab, num_tokens) || !stride_ok(logits_row_stride, vocab, num_tokens)) return K3DA_EINVAL;
    if (num_tokens == 0) return K3DA_OK;
    if (!probs || !logits) return K3DA_EINVAL;
    const size_t ints = sizeof(int32_t);
    const Span spans[] = {{probs, row_bytes(num_tokens, probs_row_stride, vocab, 4)},
                          {logits, row_bytes(num_tokens, logits_row_stride, vocab, size)},
                          {temperatures, num_requests * ints},
                          {cu_seqlens, (num_requests + 1) * ints},
                          {status, ints}};
    if (written_overlap(spans, 1, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    ProbParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.probs = probs;
    prm.logits = logits;
    prm.temperatures = temperatures;
    prm.cu_seqlens = cu_seqlens;
    prm.status = status;
    prm.probs_stride = probs_row_stride;
    prm.logits_stride = logits_row_stride;
    prm.R = num_requests;
    prm.T = num_tokens;
    prm.V = vocab;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (logits_dtype == K3DA_LOGITS_BF16) return launch_probs<__nv_bfloat16>(prm, st);
    if (logits_dtype == K3DA_LOGITS_FP16) return launch_probs<__half>(prm, st);
    return launch_probs<float>(prm, st);
}

extern "C" int k3da_verify(void *out_tokens, int32_t *num_out, const void *tokens, int token_dtype,
                           const float *target_probs, int64_t target_row_stride, const float *draft_probs,
                           int64_t draft_row_stride, const float *uniforms, int num_tokens, int vocab,
                           const int32_t *cu_seqlens, int num_requests, int32_t *status, void *stream) {
    const int rc = check_rows(cu_seqlens, num_requests, kMaxBlocks, num_tokens, vocab, status);
    if (rc != K3DA_OK) return rc;
    if (token_dtype != K3DA_POS_I32 && token_dtype != K3DA_POS_I64) return K3DA_EINVAL;
    const int size = token_dtype == K3DA_POS_I64 ? 8 : 4;
    if (!num_out || !aligned_to(num_out, 4) || !aligned_to(out_tokens, size) || !aligned_to(tokens, size) ||
        !aligned_to(target_probs, 4) || !aligned_to(draft_probs, 4) || !aligned_to(uniforms, 4))
        return K3DA_EINVAL;
    if (!stride_ok(target_row_stride, vocab, num_tokens) ||
        (draft_probs && !stride_ok(draft_row_stride, vocab, num_tokens)))
        return K3DA_EINVAL;
    if (num_tokens > 0 && (!out_tokens || !tokens || !target_probs || !uniforms)) return K3DA_EINVAL;
    const size_t ints = sizeof(int32_t), rows = static_cast<size_t>(num_tokens);
    const size_t requests = static_cast<size_t>(num_requests);
    const Span spans[] = {{out_tokens, rows * size},
                          {num_out, requests * ints},
                          {tokens, rows * size},
                          {target_probs, row_bytes(num_tokens, target_row_stride, vocab, 4)},
                          {draft_probs, row_bytes(num_tokens, draft_row_stride, vocab, 4)},
                          {uniforms, rows * 4},
                          {cu_seqlens, (requests + 1) * ints},
                          {status, ints}};
    if (written_overlap(spans, 2, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    VerifyParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.out_tokens = out_tokens;
    prm.num_out = num_out;
    prm.tokens = tokens;
    prm.target = target_probs;
    prm.draft = draft_probs;
    prm.uniforms = uniforms;
    prm.cu_seqlens = cu_seqlens;
    prm.status = status;
    prm.target_stride = target_row_stride;
    prm.draft_stride = draft_row_stride;
    prm.R = num_requests;
    prm.T = num_tokens;
    prm.V = vocab;
    prm.token_i64 = token_dtype == K3DA_POS_I64;
    // CTAs of a request: as many as fill the SMs (64 requests with half as many
    // CTAs: 17.9 us instead of 13.8), but 4096 words or more for each.
    int cluster = 1;
    while (cluster < kMaxCluster && num_requests * cluster < 4 * 152 && vocab > 4096 * cluster) cluster *= 2;
    prm.cluster = cluster;
    return launch_clusters(k3da_verify_kernel, dim3(static_cast<unsigned>(num_requests * cluster)), cluster, kVerifyThreads,
                           static_cast<cudaStream_t>(stream), prm);
}
