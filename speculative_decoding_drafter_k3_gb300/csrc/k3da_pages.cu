// k3da_pages.cu -- the pages of a cache (sm_103a): who holds which
// (k3da_pages_resize, k3da_pages_fork, k3da_pages_compact) and moving their
// data (k3da_kv_copy).
//
// A page is free when nothing lists it: its count in refs is 0.  There is no
// list of free pages whose order could depend on who came first; whoever
// needs pages gets the lowest free ones, requests in order.  So a call's
// result follows from its inputs alone, counts change by whole numbers whose
// order does not matter, and nothing has to be kept but the counts.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <climits>
#include <cstring>

#include "cache_common.cuh"
#include "k3da.h"

namespace {

using namespace k3da_cache;

constexpr int kThreads = 1024;  // one for each request
constexpr int kWarps = kThreads / 32;
static_assert(kThreads == kMaxRequests, "a thread for each request");

// Reads of what other threads of the kernel wrote (behind a barrier).
__device__ __forceinline__ int32_t load_now(const int32_t *p) {
    int32_t v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void flag(int32_t *status, int bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ int pages_for(int tokens) { return (tokens + (kP - 1)) / kP; }

struct Book {
    int32_t *page_table;
    int32_t *lens;
    int32_t *refs;
    int32_t *status;
    int page_stride, R, num_pages;
};

// Inclusive sum over the block's threads.
__device__ __forceinline__ long long block_scan(long long v, long long *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    long long before = lane < warp ? part[lane] : 0;
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
    __syncthreads();
    return v + before;
}

// The last r with start[r] <= k, for N of them at once (start rises from 0;
// in front of its end there are kMaxRequests of them).
template <int N>
__device__ __forceinline__ void owners_of(int (&r)[N], const long long *start, const long long (&k)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = 0;
#pragma unroll
    for (int step = kMaxRequests / 2; step > 0; step /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (start[r[i] + step] <= k[i]) r[i] += step;
}

// A warp's stretch of refs, and its walk over that: f(page, used) for each
// lane's four pages, 128 a warp at a time, the loads of kAhead steps issued
// before the first is looked at.  Bit k of `used`: page + k is counted; of
// `there`: page + k is in the stretch.
constexpr int kAhead = 4;  // 512 pages

struct Stretch {
    int lo, hi;
};
__device__ __forceinline__ Stretch stretch_of(int num_pages, int part, int parts) {
    const int each = static_cast<int>((num_pages + 128LL * parts - 1) / (128 * parts)) * 128;
    const long long lo = static_cast<long long>(each) * part;
    Stretch s;
    s.lo = static_cast<int>(lo < num_pages ? lo : num_pages);
    s.hi = num_pages - s.lo < each ? num_pages : s.lo + each;
    return s;
}

// What the lane finds from `base` on, in steps of 128 pages.  A count below 0 is
// reported; its page stays out of use.
__device__ __forceinline__ void look(const Book &b, Stretch s, int base, unsigned (&used)[kAhead],
                                     unsigned (&there)[kAhead]) {
    int32_t n[kAhead][4], all = 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int page = base + 128 * i;
        n[i][0] = n[i][1] = n[i][2] = n[i][3] = 0;
        if (page + 4 <= s.hi) {
            asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(n[i][0]), "=r"(n[i][1]), "=r"(n[i][2]), "=r"(n[i][3])
                         : "l"(b.refs + page)
                         : "memory");
        } else {
            for (int k = 0; k < 4; ++k)
                if (page + k < s.hi) n[i][k] = load_now(b.refs + page + k);
        }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        used[i] = there[i] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            all |= n[i][k];
            used[i] |= n[i][k] != 0 ? 1u << k : 0u;
            there[i] |= base + 128 * i + k < s.hi ? 1u << k : 0u;
        }
    }
    if (all < 0) flag(b.status, K3DA_STATUS_BAD_COUNT);
}

// What was found at a stretch's start can be kept (up to 262,144 pages that is
// all there is to see): later walks then read the rest alone.  (compact, 262,144
// pages: 13.8 us instead of 14.9.  resize is not faster by it, and for 512 pages
// 0.5 us slower.)
struct Seen {
    unsigned used[kAhead], there[kAhead];
};
template <typename F>
__device__ __forceinline__ void walk(const Book &b, Stretch s, const Seen *seen, F f) {
    const int lane = threadIdx.x & 31;
    for (int base = s.lo; base < s.hi; base += 128 * kAhead) {
        unsigned used[kAhead], there[kAhead];
        if (seen != nullptr) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                used[i] = seen->used[i];
                there[i] = seen->there[i];
            }
        }
        if (seen == nullptr || base != s.lo) look(b, s, base + 4 * lane, used, there);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (base + 128 * i >= s.hi) break;
            f(base + 128 * i + 4 * lane, used[i], there[i]);
        }
    }
}

// Of the warp's pages, of which `pick` are each lane's: how many are in front
// of the lane's first, and how many in all.
__device__ __forceinline__ int2 places(unsigned pick) {
    const unsigned below = (1u << (threadIdx.x & 31)) - 1;
    int2 r = make_int2(0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const unsigned votes = __ballot_sync(kFull, pick >> k & 1);
        r.x += __popc(votes & below);
        r.y += __popc(votes);
    }
    return r;
}
// Bits of a 4-bit mask whose page (page, page + 1, ...) is at or above `limit`.
__device__ __forceinline__ unsigned from(int page, int limit) {
    const int skip = limit - page;
    return skip <= 0 ? 15u : skip >= 4 ? 0u : 15u << skip & 15u;
}

__device__ __forceinline__ int warp_sum(int v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Stretches go to the cluster's CTAs in turn: what has to be done at the
// pool's start (where free pages are taken from) is shared by all of them.
// Two numbers of every warp of the cluster, everywhere: `all` is [kMaxCluster]
// [kWarps] in each CTA.  A barrier over the cluster.
constexpr int kMaxCluster = 16;
__device__ __forceinline__ int part_of(int rank, int warp, int cluster) { return warp * cluster + rank; }
typedef int2 Counts[kMaxCluster][kWarps];

__device__ __forceinline__ void cluster_barrier(int cluster) {
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}
__device__ __forceinline__ void tell_all(Counts &all, int2 mine, int cluster) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = static_cast<int>(cluster_rank());
    if (cluster == 1) {
        if (lane == 0) all[0][warp] = mine;
    } else if (lane < cluster) {
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(shared_of(&all[rank][warp], lane)), "r"(mine.x),
                     "r"(mine.y)
                     : "memory");
    }
    cluster_barrier(cluster);
}
// Sums over the warps in front of this one, and over all.
__device__ __forceinline__ void sums_of(const Counts &all, int cluster, int2 &before, int2 &total) {
    const int lane = threadIdx.x & 31, me = part_of(static_cast<int>(cluster_rank()), threadIdx.x >> 5, cluster);
    before = total = make_int2(0, 0);
    for (int c = 0; c < cluster; ++c) {
        const int2 n = all[c][lane];
        total.x += n.x;
        total.y += n.y;
        if (part_of(c, lane, cluster) < me) {
            before.x += n.x;
            before.y += n.y;
        }
    }
    before.x = warp_sum(before.x);
    before.y = warp_sum(before.y);
    total.x = warp_sum(total.x);
    total.y = warp_sum(total.y);
}

// CTAs of a cluster: one for each 8192 pages.  More than 8 are not for every
// device (16: resizing 1024 requests over 262,144 pages takes 12.6 us, with 8 16.5;
// compacting them 15.0, with 8 18.7): whether this one runs them is asked once.
template <typename Params>
int cluster_for(void (*kernel)(Params), int64_t num_pages, std::atomic<int> (&runs)[64]) {
    int cluster = 1;
    while (cluster < kMaxCluster && num_pages > 8192LL * cluster) cluster *= 2;
    if (cluster <= 8) return cluster;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device >= 64 ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();
        return 8;
    }
    int known = runs[device].load(std::memory_order_relaxed);  // 0: not asked yet
    if (known == 0) {
        cudaLaunchConfig_t lc;
        std::memset(&lc, 0, sizeof lc);
        lc.gridDim = dim3(kMaxCluster);
        lc.blockDim = dim3(kThreads);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        int at_once = 0;
        const bool yes = cudaOccupancyMaxActiveClusters(&at_once, kernel, &lc) == cudaSuccess && at_once > 0;
        if (!yes) cudaGetLastError();
        known = yes ? kMaxCluster : 8;
        runs[device].store(known, std::memory_order_relaxed);
    }
    return known;
}

// ------------------------------------------------------------------ resize --
//
// Pages are given back first, so that they can be taken in the same call;
// then those who grow are given the free pages, in the order of the requests:
// the k-th free page meets the k-th page that is needed.  Every CTA of the
// cluster works out for itself what each request needs (a thread each); giving
// back and looking for free pages is shared.  Bound by latency: a few bytes
// a page and request, read one after the other.  1024 requests over 262,144
// pages, 32,869 given back and 9,165 taken: 12.8 us (one CTA: 240); 8 requests that
// each grow by 8 tokens, 512 pages: 4.7.

constexpr int kSlots = 2 * kMaxRequests;  // of the table of begun pages
constexpr int kBack = 4;                  // pages that a thread gives back at a time
constexpr int kGive = 4;                  // and gives out

struct ResizeParams {
    Book b;
    const int32_t *new_lens;
    int32_t *copies;
    int cluster;
};

__global__ void __launch_bounds__(kThreads) k3da_pages_resize_kernel(const __grid_constant__ ResizeParams p) {
    __shared__ long long part[kWarps];
    __shared__ long long start[kMaxRequests + 1];  // first page given back, later first page needed, of each request
    __shared__ int32_t first_page[kMaxRequests];   // index in its row of the request's first page that changes hands
    __shared__ int32_t last[kMaxRequests];         // shared page that the request parts from, or -1
    __shared__ uint8_t begun_tokens[kMaxRequests];  // tokens of that page
    __shared__ union {
        struct {
            int32_t key[kSlots], writers[kSlots], lowest[kSlots];  // begun pages: who writes into each
        };
        uint8_t free_pages[kWarps][128 * kAhead];  // a warp's, in order, as places in their 128
    } table;
    __shared__ Counts counts;
    const Book &b = p.b;
    const int cluster = p.cluster;
    if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    wait_for_stream();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = static_cast<int>(cluster_rank());
    const int32_t *row = b.page_table + static_cast<long long>(tid) * b.page_stride;
    int len = 0, now = 0;
    if (tid < b.R) {
        len = load_here(b.lens + tid);
        now = load_here(p.new_lens + tid);
        const int most = b.page_stride * kP;
        if (len < 0 || len > most || now > most) {
            if (rank == 0) flag(b.status, K3DA_STATUS_BAD_LENGTH);
            len = now = 0;
        } else if (now < 0) {
            now = len;
        }
    }
    const int held = pages_for(len), want = pages_for(now);
    // A begun page that the request writes into next.
    int begun = -1, count = 0;
    if (now > len && len % kP) {
        begun = load_here(row + len / kP);
        if (begun < 0 || begun >= b.num_pages) {
            if (rank == 0) flag(b.status, K3DA_STATUS_BAD_PAGE);
            begun = -1;
        }
    }
    if (tid == 0) start[0] = 0;
    last[tid] = -1;
    begun_tokens[tid] = static_cast<uint8_t>(len % kP);
    first_page[tid] = want;
    for (int e = tid; e < kSlots; e += kThreads) {
        table.key[e] = -1;
        table.writers[e] = 0;
        table.lowest[e] = kMaxRequests;
    }
    // Back to the pool.
    start[tid + 1] = block_scan(held > want ? held - want : 0, part);
    __syncthreads();
    if (cluster > 1) cluster_wait();  // all of the cluster's CTAs run
    const long long back = start[kThreads];
    const long long step = static_cast<long long>(cluster) * kThreads;
    for (long long k = static_cast<long long>(rank) * kThreads + tid; k < back; k += kBack * step) {
        int32_t *entry[kBack];
        int page[kBack], old[kBack], r[kBack];
        long long at[kBack];
#pragma unroll
        for (int i = 0; i < kBack; ++i) at[i] = k + i * step;
        owners_of(r, start, at);
#pragma unroll
        for (int i = 0; i < kBack; ++i)
            entry[i] = at[i] < back ? b.page_table + static_cast<long long>(r[i]) * b.page_stride + first_page[r[i]] +
                                          (at[i] - start[r[i]])
                                    : nullptr;
#pragma unroll
        for (int i = 0; i < kBack; ++i) page[i] = entry[i] ? load_here(entry[i]) : 0;
#pragma unroll
        for (int i = 0; i < kBack; ++i) {
            old[i] = 1;
            if (!entry[i]) continue;
            *entry[i] = -1;
            if (page[i] < 0 || page[i] >= b.num_pages) flag(b.status, K3DA_STATUS_BAD_PAGE);
            else old[i] = atomicSub(b.refs + page[i], 1);
        }
#pragma unroll
        for (int i = 0; i < kBack; ++i)
            if (old[i] <= 0) {
                atomicAdd(b.refs + page[i], 1);
                flag(b.status, K3DA_STATUS_BAD_COUNT);
            }
    }
    if (back > 0) {
        __threadfence();
        cluster_barrier(cluster);
    }

    // Copy on write: a begun page that others list too.  Where all who list it
    // write into it now, the first of them keeps it.
    if (begun >= 0) {
        count = load_now(b.refs + begun);
        if (count < 1 && rank == 0) flag(b.status, K3DA_STATUS_BAD_COUNT);
        if (count < 2) begun = -1;
    }
    bool moves = begun >= 0;
    if (__syncthreads_or(moves)) {
        int slot = 0;
        if (moves) {
            const unsigned alike = __match_any_sync(__activemask(), begun);
            if (lane == __ffs(alike) - 1) {
                slot = static_cast<int>(static_cast<uint32_t>(begun) * 2654435761u >> 21);
                static_assert(kSlots == 1 << 11, "bits of a slot");
                for (int old; (old = atomicCAS(&table.key[slot], -1, begun)) != -1 && old != begun;) slot = (slot + 1) % kSlots;
                atomicAdd(&table.writers[slot], __popc(alike));
                atomicMin(&table.lowest[slot], tid);
            }
            slot = __shfl_sync(alike, slot, __ffs(alike) - 1);
        }
        __syncthreads();
        if (moves) {
            moves = table.writers[slot] < count || table.lowest[slot] != tid;
            if (table.writers[slot] > count && rank == 0) flag(b.status, K3DA_STATUS_BAD_COUNT);
        }
        if (moves) last[tid] = begun;
    }
    // What is needed, and what there is.
    const int need = (now > len ? want - held : 0) + (moves ? 1 : 0);
    start[tid + 1] = block_scan(need, part);
    first_page[tid] = moves ? len / kP : held;
    const Stretch mine = stretch_of(b.num_pages, part_of(rank, warp, cluster), cluster * kWarps);
    int free_here = 0;
    walk(b, mine, nullptr, [&](int, unsigned used, unsigned there) { free_here += __popc(there & ~used); });
    tell_all(counts, make_int2(warp_sum(free_here), 0), cluster);
    int2 before, total;
    sums_of(counts, cluster, before, total);
    const long long needed = start[kThreads];
    const bool enough = needed <= total.x;
    if (rank == 0 && tid < b.R) {
        if (now < len || (now > len && enough)) b.lens[tid] = now;
        if (!(moves && enough))
            for (int k = 0; k < 3; ++k) p.copies[k * b.R + tid] = -1;
    }
    if (!enough) {
        if (rank == 0 && tid == 0) flag(b.status, K3DA_STATUS_NO_PAGES);
        return;
    }
    long long next = before.x;  // the stretch's next free page is the next-th of all
    for (int base = mine.lo; base < mine.hi && next < needed; base += 128 * kAhead) {
        unsigned used[kAhead], there[kAhead];
        look(b, mine, base + 4 * lane, used, there);
        int until[kAhead], all = 0;  // free pages of the steps so far
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const unsigned pick = there[i] & ~used[i];
            const int2 place = places(pick);
            int at = all + place.x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (pick >> e & 1) table.free_pages[warp][at++] = static_cast<uint8_t>(4 * lane + e);
            all += place.y;
            until[i] = all;
        }
        __syncwarp();
        for (int first = lane; first < all; first += 32 * kGive) {
            long long k[kGive];
            int r[kGive];
#pragma unroll
            for (int i = 0; i < kGive; ++i) k[i] = next + first + 32 * i;
            owners_of(r, start, k);
#pragma unroll
            for (int i = 0; i < kGive; ++i) {
                const int j = first + 32 * i;
                if (j >= all || k[i] >= needed) continue;
                int page = base + table.free_pages[warp][j];
#pragma unroll
                for (int e = 0; e + 1 < kAhead; ++e) page += j >= until[e] ? 128 : 0;
                const int nth = static_cast<int>(k[i] - start[r[i]]), old = last[r[i]];
                if (old >= 0 && nth == 0) {
                    atomicSub(b.refs + old, 1);
                    p.copies[r[i]] = old;
                    p.copies[b.R + r[i]] = page;
                    p.copies[2 * b.R + r[i]] = begun_tokens[r[i]];
                }
                b.page_table[static_cast<long long>(r[i]) * b.page_stride + first_page[r[i]] + nth] = page;
                b.refs[page] = 1;
            }
        }
        next += all;
    }
}

// -------------------------------------------------------------------- fork --
//
// A CTA for each child: the parent's page ids, one more count on each page.  Bound by
// latency, and by the counts where there are many: 192 forks of 1154 pages 4.5 us.
// A child is some other request's row until its pages are given back, and a
// row that is both parent and child would be read while it is written: both
// are left out.  Which they are follows from the list alone.

constexpr int kForkThreads = 256;
constexpr int kForkEach = 8;  // entries of a thread at a time

struct ForkParams {
    Book b;
    const int32_t *parents;
    const int32_t *children;
    int num_forks;
};

__global__ void __launch_bounds__(kForkThreads) k3da_pages_fork_kernel(const __grid_constant__ ForkParams p) {
    const Book &b = p.b;
    wait_for_stream();
    const int i = blockIdx.x;
    const int parent = load_here(p.parents + i), child = load_here(p.children + i);
    bool bad = parent < 0 || parent >= b.R || child < 0 || child >= b.R;
    for (int k = threadIdx.x; k < p.num_forks; k += kForkThreads) {
        const int other = load_here(p.children + k);
        bad |= other == parent || (k < i && other == child);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag(b.status, K3DA_STATUS_BAD_REQUEST);
        return;
    }
    const int len = load_here(b.lens + parent);
    const bool wrong = len < 0 || len > b.page_stride * kP || load_here(b.lens + child) != 0;
    __syncthreads();  // the child's length is read by all before it is written
    if (wrong) {
        if (threadIdx.x == 0) flag(b.status, K3DA_STATUS_BAD_LENGTH);
        return;
    }
    if (threadIdx.x == 0) b.lens[child] = len;
    const int32_t *from = b.page_table + static_cast<long long>(parent) * b.page_stride;
    int32_t *to = b.page_table + static_cast<long long>(child) * b.page_stride;
    const int held = pages_for(len);
    for (int j = threadIdx.x; j < held; j += kForkEach * kForkThreads) {
        int page[kForkEach];
#pragma unroll
        for (int k = 0; k < kForkEach; ++k) page[k] = j + k * kForkThreads < held ? load_here(from + j + k * kForkThreads) : 0;
#pragma unroll
        for (int k = 0; k < kForkEach; ++k) {
            if (j + k * kForkThreads >= held) continue;
            to[j + k * kForkThreads] = page[k];
            if (page[k] >= 0 && page[k] < b.num_pages) atomicAdd(b.refs + page[k], 1);
            else flag(b.status, K3DA_STATUS_BAD_PAGE);
        }
    }
}

// ----------------------------------------------------------------- compact --
//
// With n live pages, the live ones at n and above change places with the free
// ones below n: the k-th highest goes into the k-th lowest.  A limit on the
// moves so frees the pool's end first.  A cluster counts, lists the moves, and
// leaves in `to` where each page at n and above is afterwards; a second kernel
// moves the counts and rewrites the rows.  (All that it changes of the book it
// changes there: should its launch be refused, rows and counts still belong
// together.)  Bound by latency: counts, n, places and moves follow one
// another with a barrier between each.  262,144 pages, 23,666 moved,
// 276,897 entries of 1024 rows looked at: 13.3 us (one CTA: 153; counts moved by the
// first kernel: 14.0); 512 pages: 5.8.

struct CompactParams {
    Book b;
    int32_t *copies;
    int32_t *num_copies;
    int32_t *to;  // [num_pages]; behind it n and the number of moves
    int max_copies;
    int cluster;
    int rows_too;  // the kernel rewrites the rows itself
};

// Up to so many entries are rewritten by the first kernel itself, an entry a
// thread: 8 rows of 40 entries, 512 pages: 5.7 us instead of 6.1, and a launch less on
// the host.  (Three entries a thread: 64 rows of 40 6.9 us instead of 6.1.)
constexpr int kRowsToo = kThreads;

// A page's count goes with it.  (No page is moved from and to.)
__device__ __forceinline__ void move_count(const Book &b, int from, int to) {
    b.refs[to] = load_now(b.refs + from);
    b.refs[from] = 0;
}

__global__ void __launch_bounds__(kThreads) k3da_pages_compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ Counts counts[2];
    const Book &b = p.b;
    const int cluster = p.cluster;
    if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    wait_for_stream();
    let_next_start();  // the second kernel comes up meanwhile; it waits for this one's end
    const int tid = threadIdx.x, warp = tid >> 5, rank = static_cast<int>(cluster_rank());
    const Stretch mine = stretch_of(b.num_pages, part_of(rank, warp, cluster), cluster * kWarps);
    int2 n = make_int2(0, 0), before, total;
    Seen seen;
    look(b, mine, mine.lo + 4 * (tid & 31), seen.used, seen.there);
    walk(b, mine, &seen, [&](int, unsigned used, unsigned) { n.x += __popc(used); });
    if (cluster > 1) cluster_wait();  // all of the cluster's CTAs run
    tell_all(counts[0], make_int2(warp_sum(n.x), 0), cluster);
    sums_of(counts[0], cluster, before, total);
    const int live = total.x;
    // Live ones at n and above, free ones below.
    n = make_int2(0, 0);
    walk(b, mine, &seen, [&](int page, unsigned used, unsigned there) {
        const unsigned high = from(page, live);
        n.x += __popc(used & high);
        n.y += __popc(there & ~used & ~high);
    });
    n.x = warp_sum(n.x);
    n.y = warp_sum(n.y);
    tell_all(counts[1], n, cluster);
    sums_of(counts[1], cluster, before, total);
    const int moves = min(total.x, p.max_copies);
    int kth_high = total.x - 1 - before.x, kth_low = before.y;  // of the stretch's next one
    int32_t *const from_list = p.copies, *const to_list = p.copies + p.max_copies, *const tokens = to_list + p.max_copies;
    walk(b, mine, &seen, [&](int page, unsigned used, unsigned there) {
        const unsigned high = from(page, live), up = used & high, down = there & ~used & ~high;
        const int base = page - 4 * static_cast<int>(threadIdx.x & 31);
        if (base + 128 > live) {
            // Every page at n and above stays, until its move says otherwise.
            if (there == 15u) {
                if (high) *reinterpret_cast<int4 *>(p.to + page) = make_int4(page, page + 1, page + 2, page + 3);
            } else {
                for (int e = 0; e < 4; ++e)
                    if (there >> e & 1) p.to[page + e] = page + e;
            }
            const int2 a = places(up);
            int i = kth_high - a.x;
            kth_high -= a.y;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (up >> e & 1) {
                    if (i < moves) from_list[i] = page + e;
                    --i;
                }
        }
        if (base < live) {
            const int2 c = places(down);
            int j = kth_low + c.x;
            kth_low += c.y;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (down >> e & 1) {
                    if (j < moves) to_list[j] = page + e;
                    ++j;
                }
        }
    });
    __threadfence();
    cluster_barrier(cluster);
    for (int k = rank * kThreads + tid; k < moves; k += cluster * kThreads) {
        const int x = load_now(from_list + k), y = load_now(to_list + k);
        tokens[k] = kP;
        p.to[x] = y;
        if (p.rows_too) move_count(b, x, y);
    }
    if (rank == 0 && tid == 0) {
        p.num_copies[0] = moves;
        p.to[b.num_pages] = live;
        p.to[b.num_pages + 1] = moves;
    }
    if (!p.rows_too) return;
    __threadfence();
    __syncthreads();
    const int r = tid / b.page_stride, j = tid - r * b.page_stride;
    if (r >= b.R) return;
    const int len = load_here(b.lens + r), page = load_here(b.page_table + tid);
    if (len < 0 || len > b.page_stride * kP) {
        if (j == 0) flag(b.status, K3DA_STATUS_BAD_LENGTH);
    } else if (moves > 0 && j < pages_for(len)) {
        if (page < 0 || page >= b.num_pages) flag(b.status, K3DA_STATUS_BAD_PAGE);
        else if (page >= live) b.page_table[tid] = load_now(p.to + page);
    }
}

constexpr int kRenameThreads = 256;
constexpr int kRenameEach = 4;  // entries of a thread at a time

__global__ void __launch_bounds__(kRenameThreads) k3da_pages_rename_kernel(const __grid_constant__ CompactParams p) {
    const Book &b = p.b;
    wait_for_stream();
    const int len = load_here(b.lens + blockIdx.y);
    const int live = load_here(p.to + b.num_pages), moves = load_here(p.to + b.num_pages + 1);
    const bool good = len >= 0 && len <= b.page_stride * kP;
    if (!good && threadIdx.x == 0) flag(b.status, K3DA_STATUS_BAD_LENGTH);
    if (moves == 0) return;
    for (long long k = (static_cast<long long>(blockIdx.x) * gridDim.y + blockIdx.y) * kRenameThreads + threadIdx.x; k < moves;
         k += static_cast<long long>(gridDim.x) * gridDim.y * kRenameThreads)
        move_count(b, load_here(p.copies + k), load_here(p.copies + p.max_copies + k));
    if (!good) return;
    int32_t *row = b.page_table + static_cast<long long>(blockIdx.y) * b.page_stride;
    const int held = pages_for(len);
    const int step = static_cast<int>(gridDim.x) * kRenameThreads;
    for (long long j = static_cast<long long>(blockIdx.x) * kRenameThreads + threadIdx.x; j < held; j += kRenameEach * step) {
        int page[kRenameEach], to[kRenameEach];
#pragma unroll
        for (int i = 0; i < kRenameEach; ++i) page[i] = j + i * step < held ? load_here(row + j + i * step) : 0;
#pragma unroll
        for (int i = 0; i < kRenameEach; ++i) {
            to[i] = page[i];
            if (page[i] < 0 || page[i] >= b.num_pages) flag(b.status, K3DA_STATUS_BAD_PAGE);
            else if (page[i] >= live) to[i] = load_here(p.to + page[i]);
        }
#pragma unroll
        for (int i = 0; i < kRenameEach; ++i)
            if (to[i] != page[i]) row[j + i * step] = to[i];
    }
}

// -------------------------------------------------------------------- copy --
//
// Bound by memory.  A warp takes one head's K or V of a page: 8 KB (bf16) or
// 4 KB of codes and 64 scales, every load issued before the first store, 32
// bytes a lane where the pool lies on such a boundary.

constexpr int kCopyThreads = 256;
constexpr int kCopyWarps = kCopyThreads / 32;

struct CopyParams {
    uint8_t *pool;
    uint8_t *scales;
    const int32_t *copies;
    const int32_t *num_copies;
    int32_t *status;
    int num_pages, tiles, max_copies;  // tiles: heads' K and V of a page
};

struct Chunk {
    uint32_t w[8];
};
__device__ __forceinline__ Chunk load32(const uint8_t *p, bool whole) {
    Chunk c;
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]), "=r"(c.w[4]), "=r"(c.w[5]), "=r"(c.w[6]),
                       "=r"(c.w[7])
                     : "l"(p));
    } else {
        const uint4 x = load_here(reinterpret_cast<const uint4 *>(p)), y = load_here(reinterpret_cast<const uint4 *>(p) + 1);
        c.w[0] = x.x, c.w[1] = x.y, c.w[2] = x.z, c.w[3] = x.w, c.w[4] = y.x, c.w[5] = y.y, c.w[6] = y.z, c.w[7] = y.w;
    }
    return c;
}
__device__ __forceinline__ void store32(uint8_t *p, const Chunk &c, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(c.w[0]), "r"(c.w[1]),
                     "r"(c.w[2]), "r"(c.w[3]), "r"(c.w[4]), "r"(c.w[5]), "r"(c.w[6]), "r"(c.w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(c.w[4], c.w[5], c.w[6], c.w[7]);
    }
}

template <bool QUANT>
__global__ void __launch_bounds__(kCopyThreads) k3da_kv_copy_kernel(const __grid_constant__ CopyParams p) {
    constexpr int kRow = QUANT ? kD : kD * 2;   // bytes of a token's row
    constexpr int kEach = kP * kRow / (32 * 32);  // 32-byte chunks of a lane
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    int n = p.max_copies;
    if (p.num_copies) n = min(n, load_here(p.num_copies));
    const bool whole = (reinterpret_cast<uintptr_t>(p.pool) & 31) == 0;
    const long long step = static_cast<long long>(gridDim.x) * kCopyWarps, items = static_cast<long long>(n) * p.tiles;
    for (long long it = static_cast<long long>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); it < items; it += step) {
        const int i = static_cast<int>(it / p.tiles), tile = static_cast<int>(it - static_cast<long long>(i) * p.tiles);
        const int from = load_here(p.copies + i), to = load_here(p.copies + static_cast<long long>(p.max_copies) + i),
                  tokens = load_here(p.copies + 2LL * p.max_copies + i);
        if (from == -1) continue;
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
            if (lane == 0) flag(p.status, K3DA_STATUS_BAD_PAGE);
            continue;
        }
        if (tokens < 0 || tokens > kP) {
            if (lane == 0) flag(p.status, K3DA_STATUS_BAD_LENGTH);
            continue;
        }
        const long long src_row = (static_cast<long long>(from) * p.tiles + tile) * kP;
        const long long dst_row = (static_cast<long long>(to) * p.tiles + tile) * kP;
        const uint8_t *src = p.pool + src_row * kRow;
        uint8_t *dst = p.pool + dst_row * kRow;
        const int bytes = tokens * kRow;
        Chunk c[kEach];
        uint8_t s[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if ((k * 32 + lane) * 32 < bytes) c[k] = load32(src + (k * 32 + lane) * 32, whole);
        if (QUANT)
            for (int k = 0; k < 2; ++k)
                if (k * 32 + lane < tokens) s[k] = *(p.scales + src_row + k * 32 + lane);
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if ((k * 32 + lane) * 32 < bytes) store32(dst + (k * 32 + lane) * 32, c[k], whole);
        if (QUANT)
            for (int k = 0; k < 2; ++k)
                if (k * 32 + lane < tokens) p.scales[dst_row + k * 32 + lane] = s[k];
    }
}

// -------------------------------------------------------------------- host --

inline int check_book(const int32_t *page_table, int page_stride, const int32_t *lens, int R, const int32_t *refs,
                      int64_t num_pages, const int32_t *status) {
    if (!page_table || !lens || !refs) return K3DA_EINVAL;
    if (!aligned_to(page_table, 4) || !aligned_to(lens, 4) || !aligned_to(refs, 16) || !aligned_to(status, 4))
        return K3DA_EINVAL;
    if (R < 1 || R > kMaxRequests || page_stride < 1 || page_stride > kMaxPageStride) return K3DA_EINVAL;
    if (num_pages < 1 || num_pages > INT_MAX / (2 * kP)) return K3DA_EINVAL;
    return K3DA_OK;
}

inline Book book_of(int32_t *page_table, int page_stride, int32_t *lens, int R, int32_t *refs, int64_t num_pages,
                    int32_t *status) {
    Book b;
    b.page_table = page_table;
    b.lens = lens;
    b.refs = refs;
    b.status = status;
    b.page_stride = page_stride;
    b.R = R;
    b.num_pages = static_cast<int>(num_pages);
    return b;
}

constexpr size_t kInt = sizeof(int32_t);

}  // namespace

extern "C" int k3da_pages_resize(int32_t *page_table, int page_stride, int32_t *lens, int num_requests, int32_t *refs,
                                 int64_t num_pages, const int32_t *new_lens, int32_t *copies, int32_t *status,
                                 void *stream) {
    const int rc = check_book(page_table, page_stride, lens, num_requests, refs, num_pages, status);
    if (rc != K3DA_OK) return rc;
    if (!new_lens || !copies || !aligned_to(new_lens, 4) || !aligned_to(copies, 4)) return K3DA_EINVAL;
    const Span spans[] = {{page_table, table_bytes(num_requests, page_stride)},
                          {lens, num_requests * kInt},
                          {refs, static_cast<size_t>(num_pages) * kInt},
                          {copies, 3 * num_requests * kInt},
                          {new_lens, num_requests * kInt},
                          {status, kInt}};
    if (written_overlap(spans, 4, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    ResizeParams prm;
    prm.b = book_of(page_table, page_stride, lens, num_requests, refs, num_pages, status);
    prm.new_lens = new_lens;
    prm.copies = copies;
    static std::atomic<int> runs[64];
    prm.cluster = cluster_for(k3da_pages_resize_kernel, num_pages, runs);
    return launch_clusters(k3da_pages_resize_kernel, dim3(static_cast<unsigned>(prm.cluster)), prm.cluster, kThreads,
                           static_cast<cudaStream_t>(stream), prm);
}

extern "C" int k3da_pages_fork(int32_t *page_table, int page_stride, int32_t *lens, int num_requests, int32_t *refs,
                               int64_t num_pages, const int32_t *parents, const int32_t *children, int num_forks,
                               int32_t *status, void *stream) {
    const int rc = check_book(page_table, page_stride, lens, num_requests, refs, num_pages, status);
    if (rc != K3DA_OK) return rc;
    if (num_forks < 0 || num_forks > kMaxRequests || !aligned_to(parents, 4) || !aligned_to(children, 4)) return K3DA_EINVAL;
    if (num_forks == 0) return K3DA_OK;
    if (!parents || !children) return K3DA_EINVAL;
    const Span spans[] = {{page_table, table_bytes(num_requests, page_stride)},
                          {lens, num_requests * kInt},
                          {refs, static_cast<size_t>(num_pages) * kInt},
                          {parents, num_forks * kInt},
                          {children, num_forks * kInt},
                          {status, kInt}};
    if (written_overlap(spans, 3, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    ForkParams prm;
    prm.b = book_of(page_table, page_stride, lens, num_requests, refs, num_pages, status);
    prm.parents = parents;
    prm.children = children;
    prm.num_forks = num_forks;
    return launch_beside(k3da_pages_fork_kernel, dim3(static_cast<unsigned>(num_forks)), kForkThreads, 0,
                         static_cast<cudaStream_t>(stream), prm);
}

extern "C" size_t k3da_compact_workspace_bytes(int64_t num_pages) {
    if (num_pages < 1 || num_pages > INT_MAX / (2 * kP)) return 0;
    return (static_cast<size_t>(num_pages) + 2) * kInt;
}

extern "C" int k3da_pages_compact(int32_t *page_table, int page_stride, int32_t *lens, int num_requests, int32_t *refs,
                                  int64_t num_pages, int32_t *copies, int max_copies, int32_t *num_copies,
                                  void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
    const int rc = check_book(page_table, page_stride, lens, num_requests, refs, num_pages, status);
    if (rc != K3DA_OK) return rc;
    if (!copies || !num_copies || !aligned_to(copies, 4) || !aligned_to(num_copies, 4) || max_copies < 1)
        return K3DA_EINVAL;
    const size_t need = k3da_compact_workspace_bytes(num_pages);
    if (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need) return K3DA_EWORKSPACE;
    const Span spans[] = {{page_table, table_bytes(num_requests, page_stride)},
                          {refs, static_cast<size_t>(num_pages) * kInt},
                          {copies, 3 * static_cast<size_t>(max_copies) * kInt},
                          {num_copies, kInt},
                          {workspace, need},
                          {lens, num_requests * kInt},
                          {status, kInt}};
    if (written_overlap(spans, 5, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    CompactParams prm;
    prm.b = book_of(page_table, page_stride, lens, num_requests, refs, num_pages, status);
    prm.copies = copies;
    prm.num_copies = num_copies;
    prm.to = static_cast<int32_t *>(workspace);
    prm.max_copies = max_copies;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static std::atomic<int> runs[64];
    prm.cluster = cluster_for(k3da_pages_compact_kernel, num_pages, runs);
    prm.rows_too = prm.cluster == 1 && static_cast<long long>(num_requests) * page_stride <= kRowsToo;
    const int first = launch_clusters(k3da_pages_compact_kernel, dim3(static_cast<unsigned>(prm.cluster)), prm.cluster, kThreads,
                                      st, prm);
    if (first != K3DA_OK || prm.rows_too) return first;
    // A thread for kRenameEach entries, up to what the SMs hold at once.
    const int across = (page_stride + kRenameThreads * kRenameEach - 1) / (kRenameThreads * kRenameEach), most = 8 * 152 / num_requests + 1;
    return launch_beside(k3da_pages_rename_kernel, dim3(static_cast<unsigned>(across < most ? across : most),
                                                        static_cast<unsigned>(num_requests)),
                         kRenameThreads, 0, st, prm);
}

extern "C" int k3da_kv_copy(void *kv_pool, int cache_dtype, void *kv_scales, int64_t num_pages, int num_kv_heads,
                            int head_dim, const int32_t *copies, int max_copies, const int32_t *num_copies,
                            int32_t *status, void *stream) {
    if (!kv_pool || (cache_dtype != K3DA_CACHE_BF16 && cache_dtype != K3DA_CACHE_E4M3) ||
        (cache_dtype == K3DA_CACHE_E4M3) != (kv_scales != nullptr))
        return K3DA_EINVAL;
    if (!aligned_to(kv_pool, 16) || !aligned_to(kv_scales, 16) || !aligned_to(copies, 4) || !aligned_to(num_copies, 4) ||
        !aligned_to(status, 4))
        return K3DA_EINVAL;
    if (num_pages < 1 || max_copies < 0 || (max_copies > 0 && !copies)) return K3DA_EINVAL;
    if (head_dim != kD || num_kv_heads < 1 || num_kv_heads > kMaxKvHeads) return K3DA_EUNSUPPORTED;
    if (num_pages > ((1LL << 31) - 1) / (2LL * num_kv_heads * kP)) return K3DA_EINVAL;
    if (max_copies == 0) return K3DA_OK;
    const Span spans[] = {{kv_pool, pool_bytes(num_pages, num_kv_heads, cache_dtype)},
                          {kv_scales, scale_bytes(num_pages, num_kv_heads)},
                          {copies, 3 * static_cast<size_t>(max_copies) * kInt},
                          {num_copies, kInt},
                          {status, kInt}};
    if (written_overlap(spans, 2, sizeof spans / sizeof spans[0])) return K3DA_EINVAL;
    CopyParams prm;
    std::memset(&prm, 0, sizeof prm);
    prm.pool = static_cast<uint8_t *>(kv_pool);
    prm.scales = static_cast<uint8_t *>(kv_scales);
    prm.copies = copies;
    prm.num_copies = num_copies;
    prm.status = status;
    prm.num_pages = static_cast<int>(num_pages);
    prm.tiles = 2 * num_kv_heads;
    prm.max_copies = max_copies;
    // A warp for each tile: 8191 pages of 4 heads in codes take 81.8 us (two CTAs
    // on an SM that go round 84.4, four 89.5, eight 85.7).  Where only the device
    // knows how long the list is, most of such a grid could have nothing to do:
    // then it is two on an SM.
    const long long ctas = (static_cast<long long>(max_copies) * prm.tiles + kCopyWarps - 1) / kCopyWarps;
    const long long most = num_copies ? 2 * 152 : INT_MAX;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache_dtype == K3DA_CACHE_E4M3) return launch_beside(k3da_kv_copy_kernel<true>, grid, kCopyThreads, 0, st, prm);
    return launch_beside(k3da_kv_copy_kernel<false>, grid, kCopyThreads, 0, st, prm);
}
