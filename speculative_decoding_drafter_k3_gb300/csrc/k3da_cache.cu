// k3da_cache.cu -- writing a chunk's K and V into the paged cache and reading
// cached tokens back (sm_103a): k3da_kv_append, k3da_kv_append_qknorm and
// k3da_kv_gather.
//
// The cache is the pool the attention calls read ([page][K=0,V=1][kv head]
// [slot][64]), in bf16 or quantised.  A quantised row (one token's K or V of
// one head) is 64 e4m3 codes and one e8m0 byte b: the values are
// code * 2^(b - 127), with 2^(b - 127) the smallest power of two that brings
// the row's largest magnitude to at most 448 (e4m3's largest).  A power of
// two costs a floating-point code nothing but range, makes the scaling and
// the reading back exact (every value is a bf16), and lets each row be
// written as soon as its token is known: no statistics over other tokens.
// A row that holds an infinity or a NaN gets b = 255 (e8m0's NaN): it reads
// back as NaN, and no other row is touched.
//
// Rounding: bf16 inputs are widened exactly, norm and RoPE run in fp32, and
// each value is rounded once, to bf16 or (from fp32) to its e4m3 code.  What
// goes into a bf16 cache as it is keeps its bits, those of a NaN too.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <cstring>

#include "cache_common.cuh"
#include "k3da.h"
#include "rope_table.h"

namespace {

using namespace k3da_cache;

// 32 bytes to 16-byte aligned memory, in one store where `whole` (32-byte
// aligned): two stores of half a sector each cost the L2 twice.
__device__ __forceinline__ void store32(uint4 *dst, uint4 a, uint4 b, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                     "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        dst[0] = a;
        dst[1] = b;
    }
}

// Two bf16 that were widened, as they were.
__device__ __forceinline__ uint32_t bits2(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// -------------------------------------------------------------- quantising --

// e8m0 byte of a row whose largest magnitude has these fp32 bits: 448 is
// 1.75 * 2^8, so the exponent field less 8, one more above 1.75; 255 for a
// row that is not finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7f800000u) return 255u;
    const int b = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return b < 0 ? 0u : static_cast<uint32_t>(b);
}

// Two values, scaled, as e4m3 codes (round to nearest even), the first in
// the low byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 codes16(const float (&x)[16], float mul) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = codes2(x[4 * k] * mul, x[4 * k + 1] * mul) | codes2(x[4 * k + 2] * mul, x[4 * k + 3] * mul) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 2^(b - 127), 2^-127 (a subnormal) included; NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7fffffffu) : b == 0u ? 0x1p-127f : __uint_as_float(b << 23);
}

// Four codes as two pairs of bf16 (exact: code * 2^e has 4 significant bits).
__device__ __forceinline__ uint2 values4(uint32_t c, float mul) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(c));
    float f[4];
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f[0]), "=f"(f[1])
        : "r"(a));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f[2]), "=f"(f[3])
        : "r"(b));
    return make_uint2(pack2(f[0] * mul, f[1] * mul), pack2(f[2] * mul, f[3] * mul));
}

// ------------------------------------------------------------------ append --
//
// Two threads per head row, as in the norm+RoPE cell (and with its
// arithmetic, operation for operation, so appending to a bf16 cache gives
// the bits of that call followed by a plain append): thread hp of a row
// holds the pairs (j, j + 32), 16 hp <= j < 16 hp + 16, read with 16-byte
// loads that are issued before anything they do not depend on: the search
// for the row's request, its page, the angles.  A CTA takes 128 rows' worth
// of whole tokens at once, and the next ones' rows while it works on them.
// Each row is read and written once; the shared-memory reads of cos, sin and
// the weights bound it: 16.8k tokens in 8 requests, 24/4 heads, q out, e4m3:
// 12.8 us where the bytes alone take 8.2; bf16 14.3 (8.7).  Raw, up to 8192
// tokens in each of 4: bf16 4.3 us (2.7), e4m3 4.5 (2.0).
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = kAppendThreads / 2;
constexpr int kAppendTokens = 64;  // most tokens of a CTA
constexpr int kAppendWave = 2 * 152;  // CTAs that run at once

struct AppendParams {
    const __nv_bfloat16 *qkv;
    uint8_t *pool;
    uint8_t *scales;
    __nv_bfloat16 *q_out;
    const int32_t *page_table;
    const int32_t *ctx_lens;
    const int32_t *cu_seqlens;
    const void *positions;
    const __nv_bfloat16 *q_w;
    const __nv_bfloat16 *k_w;
    int32_t *status;
    long long num_pages;
    int page_stride, R, T, Hq, Hkv;
    int rows;            // head rows handled per token: (q,) k and v heads
    int tokens_per_cta;
    int pos_i64;
    float eps;
    float mscale;
    unsigned long long turn_rate[kD / 2];
};

template <bool NORM, bool QUANT>
__global__ void __launch_bounds__(kAppendThreads) k3da_kv_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ float2 trig[NORM ? kAppendTokens * (kD / 2) : 1];
    __shared__ float wsm[NORM ? 2 * kD : 1];
    __shared__ int32_t cu[kMaxRequests + 1];
    __shared__ long long slot[kAppendTokens];  // first row of the token's page and its slot, -1: nothing is written
    __shared__ bool real[kAppendTokens];       // the token is some request's
    // Started beside the end of what is in front; what is behind starts only
    // when these CTAs leave (let in at once, its CTAs took 4 of 13 us).
    wait_for_stream();
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int ntok = min(p.T - t0, p.tokens_per_cta);
    const int heads = p.Hq + 2 * p.Hkv;
    const int skip = heads - p.rows;  // head rows of a token that are left alone (q heads nobody asks for)
    const int hp = tid & 1;

    uint4 a0, a1, b0, b1;
    // The thread's rows: head row h of token tl, kAppendRows further on each
    // time; next_* is the row whose loads are on their way.
    const int step = kAppendRows / p.rows, over = kAppendRows - step * p.rows;
    int next_tl = (tid >> 1) / p.rows, next_h = skip + (tid >> 1) - next_tl * p.rows;
    auto load = [&](int tl, int h) {
        a0 = a1 = b0 = b1 = make_uint4(0, 0, 0, 0);
        if (tl >= ntok) return;
        const uint4 *x = reinterpret_cast<const uint4 *>(p.qkv + (static_cast<long long>(t0 + tl) * heads + h) * kD);
        a0 = x[2 * hp];
        a1 = x[2 * hp + 1];
        b0 = x[4 + 2 * hp];
        b1 = x[4 + 2 * hp + 1];
    };
    load(next_tl, next_h);
    if (NORM) {
        unsigned long long rate = 0;  // read with constant indices: a lane-dependent one would serialise the warp
#pragma unroll
        for (int j = 0; j < kD / 2; ++j)
            if ((tid & 31) == j) rate = p.turn_rate[j];
        for (int e = tid; e < ntok * (kD / 2); e += kAppendThreads) {
            const int t = t0 + (e >> 5);
            const long long pos = p.pos_i64 ? reinterpret_cast<const long long *>(p.positions)[t]
                                            : reinterpret_cast<const int *>(p.positions)[t];
            const unsigned long long turns = static_cast<unsigned long long>(pos) * rate;
            const float half_turns = static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f;
            float sn, cs;
            sincospif(half_turns, &sn, &cs);
            trig[e] = make_float2(__fmul_rn(cs, p.mscale), __fmul_rn(sn, p.mscale));
        }
        if (tid < 2 * kD) wsm[tid] = __bfloat162float(tid < kD ? p.q_w[tid] : p.k_w[tid - kD]);
    }
    for (int e = tid; e <= p.R; e += kAppendThreads) cu[e] = load_here(p.cu_seqlens + e);
    __syncthreads();
    if (tid < ntok) {
        const int t = t0 + tid;
        const int r = request_of(cu, p.R, t);
        long long at = -1;
        const bool mine = t >= cu[r] && t < cu[r + 1];
        if (mine) {
            const long long c = static_cast<long long>(load_here(p.ctx_lens + r)) + (t - cu[r]);
            if (c < t - cu[r] || c >= static_cast<long long>(p.page_stride) * kP) {
                if (p.status) atomicOr(p.status, K3DA_STATUS_BAD_LENGTH);
            } else {
                const long long page = page_of(p.page_table, p.page_stride, p.num_pages, r, static_cast<int>(c));
                if (page >= 0) at = page * 2 * p.Hkv * kP + c % kP;
                else if (p.status) atomicOr(p.status, K3DA_STATUS_BAD_PAGE);
            }
        }
        slot[tid] = at;
        real[tid] = mine;
    }
    __syncthreads();

    for (int base = 0; base < ntok * p.rows; base += kAppendRows) {
        const bool valid = next_tl < ntok;
        const int tl = valid ? next_tl : 0, h = valid ? next_h : heads - 1;
        next_tl += step;
        next_h += over;
        if (next_h >= heads) {
            next_h -= p.rows;
            ++next_tl;
        }
        float lo[16], hi[16];
        {
            const uint32_t av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            const uint32_t bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo[2 * e] = bf16_lo(av[e]);
                lo[2 * e + 1] = bf16_hi(av[e]);
                hi[2 * e] = bf16_lo(bv[e]);
                hi[2 * e + 1] = bf16_hi(bv[e]);
            }
        }
        load(next_tl, next_h);
        if (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = __fmaf_rn(lo[e], lo[e], __fmaf_rn(hi[e], hi[e], ss));
            ss = __fadd_rn(ss, __shfl_xor_sync(kFull, ss, 1));
            if (h < p.Hq + p.Hkv) {
                const float inv = rsqrtf(__fmaf_rn(ss, 1.0f / kD, p.eps));
                const float *w = wsm + (h < p.Hq ? 0 : kD);
                const float2 *tr = trig + tl * (kD / 2);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int jp = 16 * hp + e;
                    const float n_lo = __fmul_rn(__fmul_rn(lo[e], inv), w[jp]);
                    const float n_hi = __fmul_rn(__fmul_rn(hi[e], inv), w[jp + 32]);
                    const float2 cs = tr[jp];
                    lo[e] = __fmaf_rn(n_lo, cs.x, -__fmul_rn(n_hi, cs.y));
                    hi[e] = __fmaf_rn(n_hi, cs.x, __fmul_rn(n_lo, cs.y));
                }
            }
        }
        uint32_t top = 0;  // the row's largest magnitude, as fp32 bits (a NaN's are above all)
        if (QUANT) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                top = max(top, max(__float_as_uint(lo[e]) & 0x7fffffffu, __float_as_uint(hi[e]) & 0x7fffffffu));
            top = max(top, __shfl_xor_sync(kFull, top, 1));
        }
        if (!valid) continue;
        uint4 *dst = nullptr;
        if (h < p.Hq) {
            if (real[tl]) dst = reinterpret_cast<uint4 *>(p.q_out + (static_cast<long long>(t0 + tl) * p.Hq + h) * kD);
        } else if (slot[tl] >= 0) {
            const long long row = slot[tl] + (h - p.Hq) * kP;
            if (QUANT) {
                const uint32_t b = scale_byte(top);
                const float mul = b == 255u ? 0.f : __uint_as_float((254u - b) << 23);  // 2^(127 - b)
                uint4 *codes = reinterpret_cast<uint4 *>(p.pool + row * kD);
                const uint4 zero = make_uint4(0, 0, 0, 0);
                codes[hp] = b == 255u ? zero : codes16(lo, mul);
                codes[2 + hp] = b == 255u ? zero : codes16(hi, mul);
                if (hp == 0) p.scales[row] = static_cast<uint8_t>(b);
            } else {
                dst = reinterpret_cast<uint4 *>(p.pool + row * (kD * 2));
            }
        }
        if (dst != nullptr) {
            const bool whole = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
            uint4 w[4];
            if (!NORM || (!QUANT && h >= p.Hq + p.Hkv)) {
                // As they came, a NaN's bits too: rounding would give them up.
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    w[c] = make_uint4(bits2(lo[8 * c], lo[8 * c + 1]), bits2(lo[8 * c + 2], lo[8 * c + 3]),
                                      bits2(lo[8 * c + 4], lo[8 * c + 5]), bits2(lo[8 * c + 6], lo[8 * c + 7]));
                    w[2 + c] = make_uint4(bits2(hi[8 * c], hi[8 * c + 1]), bits2(hi[8 * c + 2], hi[8 * c + 3]),
                                          bits2(hi[8 * c + 4], hi[8 * c + 5]), bits2(hi[8 * c + 6], hi[8 * c + 7]));
                }
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    w[c] = make_uint4(pack2(lo[8 * c], lo[8 * c + 1]), pack2(lo[8 * c + 2], lo[8 * c + 3]),
                                      pack2(lo[8 * c + 4], lo[8 * c + 5]), pack2(lo[8 * c + 6], lo[8 * c + 7]));
                    w[2 + c] = make_uint4(pack2(hi[8 * c], hi[8 * c + 1]), pack2(hi[8 * c + 2], hi[8 * c + 3]),
                                          pack2(hi[8 * c + 4], hi[8 * c + 5]), pack2(hi[8 * c + 6], hi[8 * c + 7]));
                }
            }
            store32(dst + 2 * hp, w[0], w[1], whole);
            store32(dst + 4 + 2 * hp, w[2], w[3], whole);
        }
    }
}

// ------------------------------------------------------------------ gather --
//
// Four threads per (token, K or V, head) row, 16 dims each: 32 bytes (bf16)
// or 16 codes and the row's scale in, 32 bytes out.  A thread issues the
// loads of all its rows before it stores any.  Bound by memory: 60k tokens,
// 4 heads, e4m3: 18.6 us (the bytes alone 17.1), bf16 27.8 (22.7); 2041
// tokens, 1 head 2.3 us.
constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 256;  // most tokens of a CTA
constexpr int kGatherWave = 4 * 152;  // CTAs that run at once
constexpr int kGatherItems = 4;    // row quarters of a thread in flight

struct GatherParams {
    __nv_bfloat16 *k_out;
    __nv_bfloat16 *v_out;
    const uint8_t *pool;
    const uint8_t *scales;
    const int32_t *page_table;
    const int32_t *starts;
    const int32_t *cu_seqlens;
    int32_t *status;
    long long num_pages;
    int page_stride, R, T, Hkv;
    int tokens_per_cta;
};

template <bool QUANT>
__global__ void __launch_bounds__(kGatherThreads) k3da_kv_gather_kernel(const __grid_constant__ GatherParams p) {
    __shared__ int32_t cu[kMaxRequests + 1];
    __shared__ long long slot[kGatherTokens];  // first row of the token's page and its slot, -1: zeros, -2: the row is left alone
    wait_for_stream();
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int ntok = min(p.T - t0, p.tokens_per_cta);
    for (int e = tid; e <= p.R; e += kGatherThreads) cu[e] = load_here(p.cu_seqlens + e);
    __syncthreads();
    if (tid < ntok) {
        const int t = t0 + tid;
        const int r = request_of(cu, p.R, t);
        long long at = -2;
        if (t >= cu[r] && t < cu[r + 1]) {
            at = -1;
            const long long c = static_cast<long long>(load_here(p.starts + r)) + (t - cu[r]);
            if (c < t - cu[r] || c >= static_cast<long long>(p.page_stride) * kP) {
                if (p.status) atomicOr(p.status, K3DA_STATUS_BAD_LENGTH);
            } else {
                const long long page = page_of(p.page_table, p.page_stride, p.num_pages, r, static_cast<int>(c));
                if (page >= 0) at = page * 2 * p.Hkv * kP + c % kP;
                else if (p.status) atomicOr(p.status, K3DA_STATUS_BAD_PAGE);
            }
        }
        slot[tid] = at;
    }
    __syncthreads();
    // The thread's quarters: token tl's quarter `rest` (K's heads, then V's),
    // kGatherThreads further on each time.
    const int per_token = p.Hkv * 8, half = p.Hkv * 4;
    const int step = kGatherThreads / per_token, over = kGatherThreads - step * per_token;
    int tl = tid / per_token, rest = tid - tl * per_token;
    while (tl < ntok) {
        uint4 x[kGatherItems], y[kGatherItems];
        uint32_t sc[kGatherItems];
        __nv_bfloat16 *dst[kGatherItems];
#pragma unroll
        for (int k = 0; k < kGatherItems; ++k) {
            x[k] = y[k] = make_uint4(0, 0, 0, 0);
            sc[k] = 127u;
            dst[k] = nullptr;
            const long long at = tl < ntok ? slot[tl] : -2;
            if (at != -2) {
                const int in_half = rest < half ? rest : rest - half;
                dst[k] = (rest < half ? p.k_out : p.v_out) + (static_cast<long long>(t0 + tl) * half + in_half) * (kD / 4);
                if (at >= 0) {
                    const long long row = at + (rest >> 2) * kP;
                    const int quarter = rest & 3;
                    if (QUANT) {
                        x[k] = reinterpret_cast<const uint4 *>(p.pool + row * kD)[quarter];
                        sc[k] = p.scales[row];
                    } else {
                        const uint4 *src = reinterpret_cast<const uint4 *>(p.pool + row * (kD * 2)) + 2 * quarter;
                        x[k] = src[0];
                        y[k] = src[1];
                    }
                }
            }
            tl += step;
            rest += over;
            if (rest >= per_token) {
                rest -= per_token;
                ++tl;
            }
        }
#pragma unroll
        for (int k = 0; k < kGatherItems; ++k) {
            if (dst[k] == nullptr) continue;
            if (QUANT) {
                const float mul = scale_of(sc[k]);
                const uint2 v0 = values4(x[k].x, mul), v1 = values4(x[k].y, mul), v2 = values4(x[k].z, mul),
                            v3 = values4(x[k].w, mul);
                x[k] = make_uint4(v0.x, v0.y, v1.x, v1.y);
                y[k] = make_uint4(v2.x, v2.y, v3.x, v3.y);
            }
            store32(reinterpret_cast<uint4 *>(dst[k]), x[k], y[k], (reinterpret_cast<uintptr_t>(dst[k]) & 31) == 0);
        }
    }
}

// -------------------------------------------------------------------- host --

// Tokens of a CTA: as many as its threads take at once, and so many times
// that where the call would fill the SMs more than once (what a CTA does
// before its first row is two dependent loads and a search: with one round of
// 4 tokens a CTA the 12.9 us of append were 19).
inline int tokens_of(int T, int at_once, int most, int wave) {
    if (at_once < 1) at_once = 1;
    const long long ctas = (static_cast<long long>(T) + at_once - 1) / at_once;
    const long long tokens = (ctas + wave - 1) / wave * at_once;
    return static_cast<int>(tokens < most ? tokens : most);
}

// Turn rates of the rotary pairs.  A thread keeps those of the base and YaRN
// that it had last: they take 1 us, a quarter of a small call's host time.
inline void turn_rates(unsigned long long (&rate)[kD / 2], float base, const k3da_yarn *yarn) {
    struct Last {
        float base = 0.f;  // no base is 0
        k3da_yarn yarn;    // factor 0: none
        unsigned long long rate[kD / 2];
    };
    thread_local Last last;
    k3da_yarn y;
    std::memset(&y, 0, sizeof y);
    if (yarn != nullptr) y = *yarn;
    if (last.base != base || std::memcmp(&last.yarn, &y, sizeof y) != 0) {
        double inv_freq[kD / 2];
        k3da_host::rope_frequencies(inv_freq, kD / 2, base, yarn);
        for (int j = 0; j < kD / 2; ++j) last.rate[j] = k3da_host::turn_rate_fixed64(inv_freq[j]);
        last.base = base;
        last.yarn = y;
    }
    std::memcpy(rate, last.rate, sizeof last.rate);
}

int launch_append(void *kv_pool, int cache_dtype, void *kv_scales, int64_t num_pages, const int32_t *page_table,
                  int page_stride, const int32_t *ctx_lens, const int32_t *cu_seqlens, int R, const void *qkv,
                  int T, int Hq, int Hkv, int head_dim, bool norm, const void *positions, int pos_dtype,
                  const void *q_norm_w, const void *k_norm_w, float eps, float rope_base, const k3da_yarn *yarn,
                  void *q_out, int32_t *status, void *stream) {
    const int rc = check_cache(kv_pool, cache_dtype, kv_scales, num_pages, page_table, page_stride, ctx_lens,
                               cu_seqlens, R, T, Hkv, head_dim, status);
    if (rc != K3DA_OK) return rc;
    if (!heads_ok(Hq, Hkv)) return K3DA_EUNSUPPORTED;
    if (T > 0 && !qkv) return K3DA_EINVAL;
    if (!aligned_to(qkv, 16)) return K3DA_EINVAL;
    if (norm) {
        if ((T > 0 && !positions) || !q_norm_w || !k_norm_w) return K3DA_EINVAL;
        if (pos_dtype != K3DA_POS_I32 && pos_dtype != K3DA_POS_I64) return K3DA_EINVAL;
        if (!aligned_to(positions, pos_dtype == K3DA_POS_I64 ? 8 : 4) || !aligned_to(q_norm_w, 2) ||
            !aligned_to(k_norm_w, 2) || !aligned_to(q_out, 16))
            return K3DA_EINVAL;
        if (!(eps >= 0.f) || !std::isfinite(eps) || !(rope_base > 1.f) || !std::isfinite(rope_base)) return K3DA_EINVAL;
        if (yarn != nullptr && !k3da_host::yarn_valid(yarn)) return K3DA_EINVAL;
    }
    if (T == 0) return K3DA_OK;
    // Nothing that is written may overlap what other threads still read, or
    // write.
    const size_t rows = static_cast<size_t>(T), ints = sizeof(int32_t);
    const Span spans[] = {{kv_pool, pool_bytes(num_pages, Hkv, cache_dtype)},
                          {kv_scales, scale_bytes(num_pages, Hkv)},
                          {q_out, rows * Hq * kD * 2},
                          {qkv, rows * (Hq + 2 * Hkv) * kD * 2},
                          {page_table, table_bytes(R, page_stride)},
                          {ctx_lens, R * ints},
                          {cu_seqlens, (R + 1) * ints},
                          {positions, rows * (pos_dtype == K3DA_POS_I64 ? 8 : 4)},
                          {q_norm_w, kD * 2},
                          {k_norm_w, kD * 2},
                          {status, ints}};
    if (written_overlap(spans, 3, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;

    AppendParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.qkv = static_cast<const __nv_bfloat16 *>(qkv);
    prm.pool = static_cast<uint8_t *>(kv_pool);
    prm.scales = static_cast<uint8_t *>(kv_scales);
    prm.q_out = static_cast<__nv_bfloat16 *>(q_out);
    prm.page_table = page_table;
    prm.ctx_lens = ctx_lens;
    prm.cu_seqlens = cu_seqlens;
    prm.positions = positions;
    prm.q_w = static_cast<const __nv_bfloat16 *>(q_norm_w);
    prm.k_w = static_cast<const __nv_bfloat16 *>(k_norm_w);
    prm.status = status;
    prm.num_pages = num_pages;
    prm.page_stride = page_stride;
    prm.R = R;
    prm.T = T;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.rows = 2 * Hkv + (norm && q_out ? Hq : 0);
    prm.tokens_per_cta = tokens_of(T, kAppendRows / prm.rows, kAppendTokens, kAppendWave);
    prm.pos_i64 = pos_dtype == K3DA_POS_I64;
    prm.eps = eps;
    prm.mscale = 1.0f;
    if (norm) {
        turn_rates(prm.turn_rate, rope_base, yarn);
        if (yarn != nullptr) prm.mscale = k3da_host::yarn_mscale(yarn);
    }
    const unsigned ctas = static_cast<unsigned>((static_cast<long long>(T) + prm.tokens_per_cta - 1) / prm.tokens_per_cta);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool quant = cache_dtype == K3DA_CACHE_E4M3;
    if (norm && quant) return launch_beside(k3da_kv_append_kernel<true, true>, dim3(ctas), kAppendThreads, 0, st, prm);
    if (norm) return launch_beside(k3da_kv_append_kernel<true, false>, dim3(ctas), kAppendThreads, 0, st, prm);
    if (quant) return launch_beside(k3da_kv_append_kernel<false, true>, dim3(ctas), kAppendThreads, 0, st, prm);
    return launch_beside(k3da_kv_append_kernel<false, false>, dim3(ctas), kAppendThreads, 0, st, prm);
}

}  // namespace

extern "C" int k3da_kv_append(void *kv_pool, int cache_dtype, void *kv_scales, int64_t num_pages,
                              const int32_t *page_table, int page_stride, const int32_t *ctx_lens,
                              const int32_t *cu_seqlens, int num_requests, const void *qkv, int num_tokens,
                              int num_q_heads, int num_kv_heads, int head_dim, int32_t *status, void *stream) {
    return launch_append(kv_pool, cache_dtype, kv_scales, num_pages, page_table, page_stride, ctx_lens, cu_seqlens,
                         num_requests, qkv, num_tokens, num_q_heads, num_kv_heads, head_dim, false, nullptr, 0,
                         nullptr, nullptr, 0.f, 0.f, nullptr, nullptr, status, stream);
}

extern "C" int k3da_kv_append_qknorm(void *kv_pool, int cache_dtype, void *kv_scales, int64_t num_pages,
                                     const int32_t *page_table, int page_stride, const int32_t *ctx_lens,
                                     const int32_t *cu_seqlens, int num_requests, const void *qkv, int num_tokens,
                                     int num_q_heads, int num_kv_heads, int head_dim, const void *positions,
                                     int pos_dtype, const void *q_norm_w, const void *k_norm_w, float eps,
                                     float rope_base, const k3da_yarn *yarn, void *q_out, int32_t *status,
                                     void *stream) {
    return launch_append(kv_pool, cache_dtype, kv_scales, num_pages, page_table, page_stride, ctx_lens, cu_seqlens,
                         num_requests, qkv, num_tokens, num_q_heads, num_kv_heads, head_dim, true, positions,
                         pos_dtype, q_norm_w, k_norm_w, eps, rope_base, yarn, q_out, status, stream);
}

extern "C" int k3da_kv_gather(void *k_out, void *v_out, const void *kv_pool, int cache_dtype, const void *kv_scales,
                              int64_t num_pages, const int32_t *page_table, int page_stride, const int32_t *starts,
                              const int32_t *cu_seqlens, int num_requests, int num_tokens, int num_kv_heads,
                              int head_dim, int32_t *status, void *stream) {
    const int rc = check_cache(kv_pool, cache_dtype, kv_scales, num_pages, page_table, page_stride, starts,
                               cu_seqlens, num_requests, num_tokens, num_kv_heads, head_dim, status);
    if (rc != K3DA_OK) return rc;
    if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16)) return K3DA_EINVAL;
    if (num_tokens == 0) return K3DA_OK;
    if (!k_out || !v_out) return K3DA_EINVAL;
    const size_t out_bytes = static_cast<size_t>(num_tokens) * num_kv_heads * kD * 2, ints = sizeof(int32_t);
    const Span spans[] = {{k_out, out_bytes},
                          {v_out, out_bytes},
                          {kv_pool, pool_bytes(num_pages, num_kv_heads, cache_dtype)},
                          {kv_scales, scale_bytes(num_pages, num_kv_heads)},
                          {page_table, table_bytes(num_requests, page_stride)},
                          {starts, num_requests * ints},
                          {cu_seqlens, (num_requests + 1) * ints},
                          {status, ints}};
    if (written_overlap(spans, 2, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    GatherParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.k_out = static_cast<__nv_bfloat16 *>(k_out);
    prm.v_out = static_cast<__nv_bfloat16 *>(v_out);
    prm.pool = static_cast<const uint8_t *>(kv_pool);
    prm.scales = static_cast<const uint8_t *>(kv_scales);
    prm.page_table = page_table;
    prm.starts = starts;
    prm.cu_seqlens = cu_seqlens;
    prm.status = status;
    prm.num_pages = num_pages;
    prm.page_stride = page_stride;
    prm.R = num_requests;
    prm.T = num_tokens;
    prm.Hkv = num_kv_heads;
    // Four row quarters a thread for the long calls; one where that leaves
    // SMs without work.
    const long long items = static_cast<long long>(num_tokens) * num_kv_heads * 8;
    const int per_cta = items >= 304LL * kGatherThreads * kGatherItems ? kGatherThreads * kGatherItems : kGatherThreads;
    prm.tokens_per_cta = tokens_of(num_tokens, per_cta / (num_kv_heads * 8), kGatherTokens, kGatherWave);
    const unsigned ctas =
        static_cast<unsigned>((static_cast<long long>(num_tokens) + prm.tokens_per_cta - 1) / prm.tokens_per_cta);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache_dtype == K3DA_CACHE_E4M3)
        return launch_beside(k3da_kv_gather_kernel<true>, dim3(ctas), kGatherThreads, 0, st, prm);
    return launch_beside(k3da_kv_gather_kernel<false>, dim3(ctas), kGatherThreads, 0, st, prm);
}

// ------------------------------------------------------------ packed calls --

namespace {

// The words of a packed call, taken in turn.
struct Words {
    const unsigned char *at;
    bool fits = true;

    template <typename T>
    T word() {
        static_assert(sizeof(T) == 8, "a word");
        T v;
        std::memcpy(&v, at, 8);
        at += 8;
        return v;
    }
    int i() {
        const int64_t v = word<int64_t>();
        fits = fits && v >= INT32_MIN && v <= INT32_MAX;
        return static_cast<int>(v);
    }
    int64_t l() { return word<int64_t>(); }
    float f() { return static_cast<float>(word<double>()); }
    void *p() { return reinterpret_cast<void *>(static_cast<uintptr_t>(word<uint64_t>())); }
    int32_t *ints() { return static_cast<int32_t *>(p()); }
};

// The arguments from kv_pool to num_requests, as every cache call has them.
struct CacheWords {
    void *pool;
    int dtype;
    void *scales;
    int64_t pages;
    int32_t *table;
    int stride;
    int32_t *lens, *cu;
    int R;
    explicit CacheWords(Words &w)
        : pool(w.p()), dtype(w.i()), scales(w.p()), pages(w.l()), table(w.ints()), stride(w.i()), lens(w.ints()),
          cu(w.ints()), R(w.i()) {}
};

}  // namespace

extern "C" int k3da_packed_call(int call, const void *words, int num_words) {
    constexpr int kNumWords[4] = {16, 24, 16, 23};
    if (call < 0 || call > 3 || words == nullptr || num_words != kNumWords[call]) return K3DA_EINVAL;
    Words w{static_cast<const unsigned char *>(words)};
    if (call == K3DA_CALL_KV_APPEND || call == K3DA_CALL_KV_APPEND_QKNORM) {
        const CacheWords c(w);
        void *qkv = w.p();
        const int T = w.i(), hq = w.i(), hkv = w.i(), d = w.i();
        if (call == K3DA_CALL_KV_APPEND) {
            int32_t *status = w.ints();
            void *stream = w.p();
            if (!w.fits) return K3DA_EINVAL;
            return k3da_kv_append(c.pool, c.dtype, c.scales, c.pages, c.table, c.stride, c.lens, c.cu, c.R, qkv, T, hq, hkv,
                                  d, status, stream);
        }
        void *positions = w.p();
        const int pos_dtype = w.i();
        void *q_w = w.p(), *k_w = w.p();
        const float eps = w.f(), base = w.f();
        const k3da_yarn *yarn = static_cast<const k3da_yarn *>(w.p());
        void *q_out = w.p();
        int32_t *status = w.ints();
        void *stream = w.p();
        if (!w.fits) return K3DA_EINVAL;
        return k3da_kv_append_qknorm(c.pool, c.dtype, c.scales, c.pages, c.table, c.stride, c.lens, c.cu, c.R, qkv, T, hq,
                                     hkv, d, positions, pos_dtype, q_w, k_w, eps, base, yarn, q_out, status, stream);
    }
    if (call == K3DA_CALL_KV_GATHER) {
        void *k = w.p(), *v = w.p();
        const CacheWords c(w);
        const int T = w.i(), hkv = w.i(), d = w.i();
        int32_t *status = w.ints();
        void *stream = w.p();
        if (!w.fits) return K3DA_EINVAL;
        return k3da_kv_gather(k, v, c.pool, c.dtype, c.scales, c.pages, c.table, c.stride, c.lens, c.cu, c.R, T, hkv, d,
                              status, stream);
    }
    void *out = w.p();
    float *lse = static_cast<float *>(w.p());
    void *q = w.p();
    const int64_t q_stride = w.l();
    const int T = w.i();
    const CacheWords c(w);
    const int hq = w.i(), hkv = w.i(), d = w.i(), mask = w.i();
    const float scale = w.f();
    void *workspace = w.p();
    const size_t bytes = static_cast<size_t>(w.l());
    int32_t *status = w.ints();
    void *stream = w.p();
    if (!w.fits) return K3DA_EINVAL;
    return k3da_chunk_attn(out, lse, q, q_stride, T, c.pool, c.dtype, c.scales, c.pages, c.table, c.stride, c.lens, c.cu,
                           c.R, hq, hkv, d, mask, scale, workspace, bytes, status, stream);
}
