// chunk_cut.h -- what a CTA of the chunk attention leaves for the combine
// kernel, and what the combine asks of it before it uses it as an index; which
// pages need a mask.  (No CUDA here: tested on the host.)
#pragma once

#ifdef __CUDACC__
#define K3DA_HOST_DEVICE __host__ __device__
#else
#define K3DA_HOST_DEVICE
#endif

namespace k3da_chunk {

constexpr int kCtas = 152;  // slices of the line at most: one CTA an SM

// part 0: the piece the CTA began with belongs to an item begun before; part
// 1: the item it ended with goes on in later CTAs, up to `last`.
struct Cut {
    int has[2];
    int row;     // first row of the item that goes on
    int tokens;  // its tokens
    int head;    // its kv head
    int last;
    int pad[2];
};
static_assert(sizeof(Cut) == 32, "cuts are 32 bytes");

// CTA `owner`'s cut names CTAs, rows and a head that there are, in a call of
// `rows` rows and `heads` kv heads whose items have at most `most` tokens.
// Every CTA writes its cut whatever becomes of its waits; nothing that it
// might hold leads the combine out of bounds.
K3DA_HOST_DEVICE inline bool cut_fits(const Cut &cut, int owner, int rows, int heads, int most) {
    return cut.last >= owner && cut.last < kCtas && cut.tokens >= 0 && cut.tokens <= most && cut.row >= 0 &&
           cut.row <= rows && cut.tokens <= rows - cut.row && cut.head >= 0 && cut.head < heads;
}

// A page whose first key is `first` has keys that not all of the rows see,
// who see `least` keys at least.  (The last page of the longest table ends 64
// keys before 2^31: a tile's second page begins there, and first + 64 is no
// int.)
K3DA_HOST_DEVICE inline bool page_masked(int first, int least) { return least - first < 64; }

}  // namespace k3da_chunk
