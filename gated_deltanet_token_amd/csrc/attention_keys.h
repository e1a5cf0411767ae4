// Which keys a row of the paged attention sees, and where its tiles of keys
// begin: integer arithmetic on lengths up to 2^31 - 1, shared by the kernels
// and, as plain C++, by the checks on the host.
#pragma once

#ifdef __HIPCC__
#include <hip/hip_runtime.h>

#define GDN_KEYS_FN __host__ __device__ __forceinline__
#else
#define GDN_KEYS_FN inline
#endif

namespace gdn {

GDN_KEYS_FN int key_min(int a, int b) { return a < b ? a : b; }

// one request's part in a call, as the kernels see it
struct Request {
    int begin, n;       // its first token, and how many
    int len;            // keys, as seq_lens says (>= 0)
    int L;              // keys within the block table's row
};

// The keys [jb, je) that token i of the request sees, 0 <= jb <= L and je <= L.
// (A window of a request that is longer than its row may begin past the row:
// it is cut too, so that tiles never begin past key L, which is 1,024 short of
// 2^31 - 1 at most.  Uncut, the tiles of a wave further on begin past 2^31 - 1,
// which is below key 0.)
GDN_KEYS_FN void key_range(int causal, int window, const Request &r, int i, int &jb, int &je) {
    const int upto = r.len - r.n + i + 1;            // its position + 1
    je = causal ? key_min(r.L, upto) : r.L;
    jb = window > 0 && upto > window ? key_min(upto - window, r.L) : 0;
}

// The splits of a row tile's keys [lo, hi): split i takes the keys of [i C,
// (i + 1) C), the last one all that follow.
struct Splits {
    int first, last;    // those that have keys (last < first: none)
};
GDN_KEYS_FN Splits splits_of(int lo, int hi, int chunk, int n) {
    Splits s;
    s.first = key_min(lo / chunk, n - 1);
    s.last = hi > lo ? key_min((hi - 1) / chunk, n - 1) : s.first - 1;
    return s;
}

// the first of a wave's tiles of `tile` keys (a power of two) that are taken in
// turns from key k_lo on
GDN_KEYS_FN int first_tile(int k_lo, int tile, int wave) { return (k_lo & ~(tile - 1)) + wave * tile; }

}  // namespace gdn
