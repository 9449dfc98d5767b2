// paged.cuh -- what the kernels that read the paged FP8 KV cache in place
// share: the view of the cache, the position -> slot map, the visibility rule
// and the host-side checks of the arguments.
#pragma once

#include <cmath>

#include "common.cuh"

namespace {

using namespace fp8q;

constexpr int kPagedMaxRow = 8192;   // H * Dh per token, the cache's own limit
// max_blocks * block_size: positions, and the ends of the tiles that hold
// them, stay below 2^31
constexpr int64_t kPagedMaxContext = 0x7FFF0000ll;

// n / d for 0 <= n < 2^31, d fixed for a launch: multiply and shift (Granlund
// and Montgomery's round-up form), because the table lookup of every position
// divides by the page size.
struct FastDiv {
    uint32_t mul, shift, d;
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};
inline FastDiv make_fastdiv(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {(uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s, d};
}

// A K scale as it multiplies a logit: an infinite one is a NaN, as the elements of q . k that it makes infinite are of
// both signs.
__device__ __forceinline__ float k_factor(float d) { return fmaf(d, 0.0f, d); }

// The cache as one launch sees it.  Slot ids fit 31 bits (checked on the
// host); byte offsets are formed in 64 bits.
struct PagedView {
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *lens;
    int64_t max_blocks;
    FastDiv bs;
    int num_blocks, H, Dh, cap;   // cap = max_blocks * block_size, at most kPagedMaxContext
    int window, sinks;            // window == 0: none

    __device__ __forceinline__ int length(int64_t b) const {
        const int n = lens[b];
        return n < 0 ? 0 : (n > cap ? cap : n);
    }
    // slot of position j of sequence b, or -1 when its page id is not a page
    __device__ __forceinline__ int slot(int64_t b, int j) const {
        const uint32_t pg = bs.div((uint32_t)j);
        const int32_t blk = table[b * max_blocks + pg];
        if (blk < 0 || blk >= num_blocks) return -1;
        return (int)((uint32_t)blk * bs.d + ((uint32_t)j - pg * bs.d));
    }
    // first position of the window of the query at position p
    __device__ __forceinline__ int window_begin(int p) const {
        return window > 0 && p + 1 > window ? p + 1 - window : 0;
    }
};

}  // namespace

namespace {

inline fp8_status paged_cache_shape(int64_t H, int64_t Dh, int64_t block_size, int64_t num_blocks) {
    if (H < 1 || Dh < 8 || Dh % 8 || Dh > kPagedMaxRow || H > kPagedMaxRow || H * Dh > kPagedMaxRow)
        return FP8_ERR_SHAPE;
    if (block_size < 1 || block_size > 0x7FFFFFFFll || num_blocks < 0 || num_blocks > 0x7FFFFFFFll ||
        block_size * num_blocks > 0x7FFFFFFFll)
        return FP8_ERR_SHAPE;
    return FP8_OK;
}

inline PagedView make_paged_view(const uint8_t *kc, const float *ks, const uint8_t *vc, const float *vs, int64_t H,
                                 int64_t Dh, int64_t block_size, int64_t num_blocks, const int32_t *table,
                                 const int32_t *lens, int64_t max_blocks, int64_t window, int64_t sinks) {
    PagedView v;
    v.kc = kc; v.ks = ks; v.vc = vc; v.vs = vs;
    v.table = table; v.lens = lens; v.max_blocks = max_blocks;
    v.bs = make_fastdiv((uint32_t)block_size);
    v.num_blocks = (int)num_blocks; v.H = (int)H; v.Dh = (int)Dh;
    const int64_t lim = 0x7FFFFFFFll;
    v.cap = (int)(max_blocks * block_size);
    v.window = (int)(window > lim ? 0 : window);   // a window of 2^31 or more hides nothing
    v.sinks = (int)(sinks > lim ? lim : sinks);
    return v;
}

}  // namespace
