// cache_common.cuh -- what the paged-cache kernels share (append, gather,
// chunk attention): sizes, the request of a packed row, the cache slot of a
// token, and the host's checks of a cache's arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

#include "k3da.h"

namespace k3da_cache {

constexpr int kD = 64;  // head_dim
constexpr int kP = 64;  // tokens per page
constexpr int kMaxRequests = K3DA_MAX_CHUNK_REQUESTS;
constexpr int kMaxPageStride = 0x7fffffff / kP;  // page_stride * 64 stays an int
constexpr int kMaxGroup = 16;                    // query heads per kv head
constexpr int kMaxKvHeads = 64;
constexpr unsigned kFull = 0xffffffffu;

// Request of packed row t: the last r with cu[r] <= t (cu in shared memory,
// R + 1 entries, rising).  Always in [0, R) whatever cu holds.
__device__ __forceinline__ int request_of(const int32_t *cu, int R, int t) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Loads of what the kernel in front of this one on the stream may write while
// this one is resident already: in the order of the program, behind the wait
// for that kernel.  (A read-only load may be moved in front of it, and
// asks for memory that nobody writes while the kernel is there.  Loads past
// the SM's own cache, ld.global.cg, took 7.5 us instead of 7.1 for 1 token over
// 300: a plan reads some words twice.)
__device__ __forceinline__ int32_t load_here(const int32_t *p) {
    int32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 load_here(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Page of cache token c (inside the row's capacity) of request r, or -1 when
// the table's entry is no page of the pool.
__device__ __forceinline__ long long page_of(const int32_t *page_table, int page_stride, long long num_pages, int r,
                                             int c) {
    const int page = load_here(page_table + static_cast<long long>(r) * page_stride + c / kP);
    return page < 0 || page >= num_pages ? -1 : page;
}

// The kernel in front of this one on the stream is complete, and what it
// wrote can be read.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel behind this one may start (once every CTA has said so or left).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// A runtime call failed: its error is taken back from the thread, where the
// library's other calls would find it behind launches of their own.
inline int cuda_failed() {
    cudaGetLastError();
    return K3DA_ECUDA;
}

// Launches `kernel` as a programmatic dependent: it may start before the
// kernel in front of it on the stream is complete, and waits for that itself
// (wait_for_stream), before it reads or writes anything or, where it only has
// to be complete later, at its end.
template <typename... Params, typename... Args>
inline int launch_beside(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const Args &...args) {
    cudaLaunchConfig_t lc;
    std::memset(&lc, 0, sizeof lc);
    lc.gridDim = grid;
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...) == cudaSuccess ? K3DA_OK : cuda_failed();
}

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Memory a call is given.
struct Span {
    const void *at;  // NULL: not given
    size_t bytes;
};

// One of the first `written` of n spans overlaps another of the n.
inline bool written_overlap(const Span *spans, int written, int n) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < n; ++j)
            if (spans[i].at && spans[j].at && overlap(spans[i].at, spans[i].bytes, spans[j].at, spans[j].bytes)) return true;
    return false;
}

inline bool heads_ok(int hq, int hkv) {
    return hkv >= 1 && hkv <= kMaxKvHeads && hq >= hkv && hq % hkv == 0 && hq / hkv <= kMaxGroup;
}

inline size_t pool_bytes(int64_t num_pages, int hkv, int cache_dtype) {
    return static_cast<size_t>(num_pages) * 2 * hkv * kP * kD * (cache_dtype == K3DA_CACHE_BF16 ? 2 : 1);
}

inline size_t scale_bytes(int64_t num_pages, int hkv) { return static_cast<size_t>(num_pages) * 2 * hkv * kP; }

inline size_t table_bytes(int R, int page_stride) { return static_cast<size_t>(R) * page_stride * sizeof(int32_t); }

// The arguments every cache call has.
inline int check_cache(const void *pool, int cache_dtype, const void *scales, int64_t num_pages,
                       const int32_t *page_table, int page_stride, const int32_t *ctx_lens,
                       const int32_t *cu_seqlens, int R, int num_tokens, int hkv, int head_dim,
                       const int32_t *status) {
    if (!pool || !page_table || !ctx_lens || !cu_seqlens) return K3DA_EINVAL;
    if (cache_dtype != K3DA_CACHE_BF16 && cache_dtype != K3DA_CACHE_E4M3) return K3DA_EINVAL;
    if ((cache_dtype == K3DA_CACHE_E4M3) != (scales != nullptr)) return K3DA_EINVAL;
    if (!aligned_to(pool, 16) || !aligned_to(scales, 16) || !aligned_to(page_table, 4) || !aligned_to(ctx_lens, 4) ||
        !aligned_to(cu_seqlens, 4) || !aligned_to(status, 4))
        return K3DA_EINVAL;
    if (R < 1 || R > kMaxRequests || num_tokens < 0 || page_stride < 1 || page_stride > kMaxPageStride ||
        num_pages < 1)
        return K3DA_EINVAL;
    if (head_dim != kD || hkv < 1 || hkv > kMaxKvHeads) return K3DA_EUNSUPPORTED;
    if (num_pages > ((1LL << 31) - 1) / (2LL * hkv * kP)) return K3DA_EINVAL;
    return K3DA_OK;
}

}  // namespace k3da_cache
