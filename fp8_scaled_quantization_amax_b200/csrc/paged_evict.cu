// paged_evict.cu -- eviction from the paged FP8 KV cache by accumulated
// attention weight.
//
// Two launches.  k_evict_select: a CTA per (sequence, KV head) finds the
// threshold mass by a radix selection on order-preserving integer keys (four
// passes of eight bits) and lists the kept positions in ascending order.
// k_evict_copy: the kept rows' codes and scales go to the new pages.
#include "paged.cuh"

using namespace fp8q;

namespace {

constexpr int kSel = 512;

struct EvictArgs {
    const float *mass;
    int64_t ld_mass;
    const int32_t *dst_table;
    int64_t dst_max_blocks;
    int budget, sinks, recent;
    int32_t *kept;
    float *mass_out;
    int64_t ld_out;
    int32_t *lens_out;
};

// Larger float <-> larger key; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t mass_key(float m) {
    if (isnan(m)) m = -INFINITY;
    const uint32_t u = __float_as_uint(m + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSel)
k_evict_select(PagedView pv, EvictArgs a) {
    __shared__ uint32_t hist[256], sh[3], wsum[2][kSel / 32];
    const int64_t row = blockIdx.x, b = row / pv.H;
    const int n = pv.length(b), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float *m = a.mass + row * a.ld_mass;
    int32_t *kept = a.kept + row * a.budget;
    float *mo = a.mass_out + row * a.ld_out;
    auto mass_at = [&](int j) { return j < a.ld_mass ? m[j] : 0.0f; };
    if (n <= a.budget) {
        for (int j = tid; j < a.budget; j += kSel) kept[j] = j < n ? j : -1;
        for (int64_t j = tid; j < a.ld_out; j += kSel) mo[j] = j < n ? mass_at((int)j) : 0.0f;
        return;
    }
    for (int64_t j = (int64_t)a.budget + tid; j < a.ld_out; j += kSel) mo[j] = 0.0f;
    const int lo = a.sinks, hi = n - a.recent;            // the positions to choose from
    uint32_t need = (uint32_t)(a.budget - a.sinks - a.recent), prefix = 0;
    for (int shift = 24; need > 0 && shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = lo + tid; j < hi; j += kSel) {
            const uint32_t k = mass_key(mass_at(j));
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t left = need, d = 255;
            while (hist[d] < left) left -= hist[d--];     // the counts sum to at least `need`
            sh[0] = d;
            sh[1] = left;
        }
        __syncthreads();
        prefix |= sh[0] << shift;
        need = sh[1];
        __syncthreads();
    }
    // keys above `prefix` are kept, and the first `need` that equal it
    const bool choose = a.budget > a.sinks + a.recent;
    uint32_t out = 0, ties = 0;
    for (int j0 = 0; j0 < n; j0 += kSel) {
        const int j = j0 + tid;
        bool k = j < n && (j < lo || j >= hi), tie = false;
        if (choose && j >= lo && j < hi) {
            const uint32_t key = mass_key(mass_at(j));
            k = key > prefix;
            tie = key == prefix;
        }
        const uint32_t tb = __ballot_sync(0xFFFFFFFFu, tie);
        if (lane == 0) wsum[0][warp] = __popc(tb);
        __syncthreads();
        uint32_t before = ties, all = 0;
        for (int w = 0; w < kSel / 32; ++w) {
            if (w < warp) before += wsum[0][w];
            all += wsum[0][w];
        }
        if (tie && before + __popc(tb & ((1u << lane) - 1u)) < need) k = true;
        ties += all;
        const uint32_t kb = __ballot_sync(0xFFFFFFFFu, k);
        if (lane == 0) wsum[1][warp] = __popc(kb);
        __syncthreads();
        uint32_t at = out;
        all = 0;
        for (int w = 0; w < kSel / 32; ++w) {
            if (w < warp) at += wsum[1][w];
            all += wsum[1][w];
        }
        at += __popc(kb & ((1u << lane) - 1u));
        if (k && at < (uint32_t)a.budget) {
            kept[at] = j;
            if (at < a.ld_out) mo[at] = mass_at(j);
        }
        out += all;
        __syncthreads();
    }
}

// One thread per 8 codes of K and of V of a kept row.
__global__ void __launch_bounds__(256)
k_evict_copy(PagedView pv, EvictArgs a, uint8_t *kc, float *ks, uint8_t *vc, float *vs) {
    const int64_t b = blockIdx.y;
    const int C = pv.H * pv.Dh / 8, G = pv.Dh / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        const int n = pv.length(b);
        a.lens_out[b] = n < a.budget ? n : a.budget;
    }
    if (i >= (int64_t)a.budget * C) return;
    const int r = (int)(i / C), c = (int)(i % C), h = c / G;
    const int j = a.kept[(b * pv.H + h) * a.budget + r];
    if (j < 0) return;
    const uint32_t pg = pv.bs.div((uint32_t)r);
    if (pg >= a.dst_max_blocks) return;
    const int32_t blk = a.dst_table[b * a.dst_max_blocks + pg];
    if (blk < 0 || blk >= pv.num_blocks) return;
    const int64_t dst = (int64_t)blk * pv.bs.d + (r - pg * pv.bs.d), src = pv.slot(b, j);
    const uint2 z = make_uint2(0u, 0u);
    reinterpret_cast<uint2 *>(kc)[dst * C + c] = src >= 0 ? reinterpret_cast<const uint2 *>(kc)[src * C + c] : z;
    reinterpret_cast<uint2 *>(vc)[dst * C + c] = src >= 0 ? reinterpret_cast<const uint2 *>(vc)[src * C + c] : z;
    if (c % G == 0) {
        ks[dst * pv.H + h] = src >= 0 ? ks[src * pv.H + h] : 0.0f;
        vs[dst * pv.H + h] = src >= 0 ? vs[src * pv.H + h] : 0.0f;
    }
}

}  // namespace

using namespace fp8q_host;

extern "C" fp8_status fp8_paged_kv_evict(uint8_t *k_cache, float *k_scale, uint8_t *v_cache, float *v_scale, int64_t H,
                                         int64_t Dh, int64_t block_size, int64_t num_blocks,
                                         const int32_t *block_table, const int32_t *seq_lens, int64_t B,
                                         int64_t max_blocks, const float *mass, int64_t ld_mass,
                                         const int32_t *dst_table, int64_t dst_max_blocks, int64_t budget,
                                         int64_t sinks, int64_t recent, int32_t *kept, float *mass_out,
                                         int64_t ld_out, int32_t *lens_out, void *stream) {
    fp8_status st = paged_cache_shape(H, Dh, block_size, num_blocks);
    if (st != FP8_OK) return st;
    if (B < 0 || B > 65535 || max_blocks < 0 || dst_max_blocks < 0 || ld_mass < 0) return FP8_ERR_SHAPE;
    if (budget < 1 || budget > 0x7FFFFFFFll || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks ||
        ld_out < 0)
        return FP8_ERR_SHAPE;
    if (max_blocks > kPagedMaxContext / block_size || dst_max_blocks > kPagedMaxContext / block_size)
        return FP8_ERR_SHAPE;
    const int64_t blocks = (budget * (H * Dh / 8) + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return FP8_ERR_SHAPE;
    if (B == 0) return FP8_OK;
    if (!seq_lens || !kept || !lens_out || (ld_out > 0 && !mass_out) || (ld_mass > 0 && !mass)) return FP8_ERR_INVALID_ARG;
    if ((max_blocks > 0 && !block_table) || (dst_max_blocks > 0 && !dst_table)) return FP8_ERR_INVALID_ARG;
    if (num_blocks > 0 && (!k_cache || !k_scale || !v_cache || !v_scale)) return FP8_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return FP8_ERR_ALIGNMENT;
    int sms;
    st = check_device(&sms);
    if (st != FP8_OK) return st;
    const PagedView pv = make_paged_view(k_cache, k_scale, v_cache, v_scale, H, Dh, block_size, num_blocks,
                                         block_table, seq_lens, max_blocks, 0, 0);
    const EvictArgs a = {mass, ld_mass, dst_table, dst_max_blocks, (int)budget, (int)sinks, (int)recent,
                         kept, mass_out, ld_out, lens_out};
    cudaStream_t s = as_stream(stream);
    k_evict_select<<<dim3((unsigned)(B * H)), kSel, 0, s>>>(pv, a);
    k_evict_copy<<<dim3((unsigned)blocks, (unsigned)B), 256, 0, s>>>(pv, a, k_cache, k_scale, v_cache, v_scale);
    return cudaPeekAtLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}
