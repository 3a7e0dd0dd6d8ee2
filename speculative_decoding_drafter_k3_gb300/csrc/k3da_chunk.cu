// k3da_chunk.cu -- attention of ragged chunks of new tokens over the paged
// cache (sm_103a): k3da_chunk_attn.
//
// For row i of request r's chunk and query head h (kv head g = h / (Hq/Hkv)):
//   o = sum_c softmax_c(scale * q . k_c) v_c,   lse = log sum_c exp(scale * q . k_c)
// over the cache tokens c the mask shows: c <= ctx_r + i (causal), all
// ctx_r + n_r (full), or the ctx_r before the chunk (context).  A row that
// sees nothing gets o = 0 and lse = -inf.
//
// One warp per (row, query head): lane l takes the keys l, l + 32, ... with
// a running maximum, sum and output of its own in fp32; the lanes merge at
// the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <cstring>

#include "cache_common.cuh"
#include "k3da.h"

namespace {

using namespace k3da_cache;

struct ChunkParams {
    __nv_bfloat16 *out;
    float *lse;
    const __nv_bfloat16 *q;
    const uint8_t *pool;
    const uint8_t *scales;
    const int32_t *page_table;
    const int32_t *ctx_lens;
    const int32_t *cu_seqlens;
    int32_t *status;
    long long q_stride;
    long long num_pages;
    int page_stride, R, T, Hq, Hkv;
    int mask;
    float scale_log2;
};

constexpr int kWarps = 4;

__device__ __forceinline__ float e4m3_value(uint32_t c) {
    uint32_t h;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(c & 0xffu));
    float f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

template <bool QUANT>
__device__ __forceinline__ float cached(const ChunkParams &p, long long row, int d) {
    if (!QUANT) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.pool)[row * kD + d]);
    const uint32_t b = p.scales[row];
    const float s = b == 255u ? __uint_as_float(0x7fffffffu) : b == 0u ? 0x1p-127f : __uint_as_float(b << 23);
    return e4m3_value(p.pool[row * kD + d]) * s;
}

template <bool QUANT>
__global__ void __launch_bounds__(32 * kWarps) k3da_chunk_simple_kernel(const __grid_constant__ ChunkParams p) {
    __shared__ int32_t cu[kMaxRequests + 1];
    for (int e = threadIdx.x; e <= p.R; e += 32 * kWarps) cu[e] = p.cu_seqlens[e];
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(p.T) * p.Hq) return;
    const int t = static_cast<int>(w / p.Hq), h = static_cast<int>(w % p.Hq);
    const int r = request_of(cu, p.R, t);
    if (t < cu[r] || t >= cu[r + 1]) return;
    const int n = cu[r + 1] - cu[r];
    const int cap = p.page_stride * kP;
    int ctx = p.ctx_lens[r];
    if (ctx < 0 || static_cast<long long>(ctx) + n > cap) {
        if (lane == 0 && p.status) atomicOr(p.status, K3DA_STATUS_BAD_LENGTH);
        ctx = ctx < 0 ? 0 : ctx > cap ? cap : ctx;
    }
    long long limit = p.mask == K3DA_MASK_CAUSAL ? static_cast<long long>(ctx) + (t - cu[r]) + 1
                      : p.mask == K3DA_MASK_FULL ? static_cast<long long>(ctx) + n
                                                 : ctx;
    if (limit > cap) limit = cap;
    const __nv_bfloat16 *q = p.q + t * p.q_stride + h * kD;
    const int g = h / (p.Hq / p.Hkv);
    float m = -INFINITY, l = 0.f, o[kD];
#pragma unroll
    for (int d = 0; d < kD; ++d) o[d] = 0.f;
    for (int c = lane; c < limit; c += 32) {
        const long long page = page_of(p.page_table, p.page_stride, p.num_pages, r, c);
        if (page < 0 && p.status) atomicOr(p.status, K3DA_STATUS_BAD_PAGE);
        const long long krow = ((page * 2) * p.Hkv + g) * kP + c % kP, vrow = krow + static_cast<long long>(p.Hkv) * kP;
        float s = 0.f;
        if (page >= 0)
            for (int d = 0; d < kD; ++d) s += __bfloat162float(q[d]) * cached<QUANT>(p, krow, d);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
        l = l * f + e;
#pragma unroll
        for (int d = 0; d < kD; ++d) o[d] = o[d] * f + (page >= 0 ? e * cached<QUANT>(p, vrow, d) : 0.f);
        m = mn;
    }
    float mt = m;
    for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, x));
    const float f = m == -INFINITY ? 0.f : exp2f(m - mt);
    l *= f;
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(kFull, l, x);
    __nv_bfloat16 *dst = p.out + (static_cast<long long>(t) * p.Hq + h) * kD;
#pragma unroll
    for (int d = 0; d < kD; ++d) {
        float v = f == 0.f ? 0.f : o[d] * f;
        for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(kFull, v, x);
        if (lane == (d & 31)) dst[d] = __float2bfloat16_rn(limit > 0 ? v / l : 0.f);
    }
    if (lane == 0 && p.lse)
        p.lse[static_cast<long long>(t) * p.Hq + h] = limit > 0 ? (mt + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

extern "C" size_t k3da_chunk_workspace_bytes(int num_tokens, int num_requests, int num_q_heads, int num_kv_heads,
                                             int page_stride) {
    if (num_tokens < 0 || num_requests < 1 || num_requests > kMaxRequests || !heads_ok(num_q_heads, num_kv_heads) ||
        page_stride < 1 || page_stride > kMaxPageStride)
        return 0;
    return 256;
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
    if (!workspace || !aligned_to(workspace, 256)) return K3DA_EWORKSPACE;
    if (workspace_bytes < k3da_chunk_workspace_bytes(num_tokens, num_requests, num_q_heads, num_kv_heads, page_stride))
        return K3DA_EWORKSPACE;
    if (num_tokens == 0) return K3DA_OK;
    if (!out || !q) return K3DA_EINVAL;
    const size_t out_bytes = static_cast<size_t>(num_tokens) * width * 2;
    const size_t q_bytes = (static_cast<size_t>(num_tokens - 1) * q_row_stride + width) * 2;
    if (overlap(out, out_bytes, q, q_bytes) ||
        overlap(out, out_bytes, kv_pool, pool_bytes(num_pages, num_kv_heads, cache_dtype)))
        return K3DA_EINVAL;
    ChunkParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.out = static_cast<__nv_bfloat16 *>(out);
    prm.lse = lse;
    prm.q = static_cast<const __nv_bfloat16 *>(q);
    prm.pool = static_cast<const uint8_t *>(kv_pool);
    prm.scales = static_cast<const uint8_t *>(kv_scales);
    prm.page_table = page_table;
    prm.ctx_lens = ctx_lens;
    prm.cu_seqlens = cu_seqlens;
    prm.status = status;
    prm.q_stride = q_row_stride;
    prm.num_pages = num_pages;
    prm.page_stride = page_stride;
    prm.R = num_requests;
    prm.T = num_tokens;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.mask = mask;
    prm.scale_log2 = softmax_scale * 1.4426950408889634f;
    const long long warps = static_cast<long long>(num_tokens) * num_q_heads;
    const unsigned ctas = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache_dtype == K3DA_CACHE_E4M3) k3da_chunk_simple_kernel<true><<<ctas, 32 * kWarps, 0, st>>>(prm);
    else k3da_chunk_simple_kernel<false><<<ctas, 32 * kWarps, 0, st>>>(prm);
    return cudaGetLastError() == cudaSuccess ? K3DA_OK : K3DA_ECUDA;
}
