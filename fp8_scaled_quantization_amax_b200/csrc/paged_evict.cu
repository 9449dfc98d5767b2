// paged_evict.cu -- eviction from the paged FP8 KV cache by accumulated
// attention weight.
//
// Two launches.
//
// k_evict_select: a CTA per (sequence, KV head) finds the mass of the last kept
// token by a radix selection on order-preserving integer keys, eight bits a pass
// (a warp adds equal digits up before its one shared atomic: accumulated weights
// are full of zeros and of equal exponents), ending early when a digit's tokens
// are all kept.  Then one pass in order of position: a token's place among the
// kept is (sure ones before it) + min(ties before it, ties kept), one block scan
// of both counts per 4096 positions.  Rows of up to 4096 tokens stay in
// registers between the passes, longer ones come from L1 and L2 again.
//
// k_evict_copy: bound by HBM (2 * (Dh + 4) bytes read and written per kept row,
// K and V).  A CTA takes some positions of one sequence with all their heads, so
// that its writes are whole token rows; it looks the rows' slots up once, into
// shared memory, and then copies 16 bytes per thread and load, eight loads in
// flight.
//
// Measured on a B200 with L2 flushed: 16 sequences x 32 heads of 128, 8192
// tokens to 4096: selection 47 us, copy 212 us (1.1 GB read and written, 5.4
// TB/s).  Selection by 1024 threads instead of 512: 10 - 15 us slower there.
#include <algorithm>

#include "paged.cuh"

using namespace fp8q;

namespace {

constexpr int kSel = 512, kPer = 8, kSpan = kSel * kPer;   // threads; positions of a thread, of a round

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

// Adds one to hist[digit] for every lane with on, one atomic per digit of the warp.
__device__ __forceinline__ void count_digit(uint32_t *hist, uint32_t digit, bool on) {
    const uint32_t who = __match_any_sync(0xFFFFFFFFu, on ? digit : 256u);
    if (on && (threadIdx.x & 31) == (uint32_t)(__ffs(who) - 1)) atomicAdd(&hist[digit], (uint32_t)__popc(who));
}

__global__ void __launch_bounds__(kSel, 4)
k_evict_select(const PagedView pv, const EvictArgs a) {
    __shared__ uint32_t hist[256], s_digit, s_left, s_count;
    __shared__ uint64_t s_warp[kSel / 32];
    const int64_t row = blockIdx.x, b = row / pv.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int n = pv.length(b);
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
    const int rounds = (int)(((int64_t)n + kSpan - 1) / kSpan);
    const bool whole_vectors = (reinterpret_cast<uintptr_t>(m) & 15) == 0;
    float v[kPer];                                        // masses of this thread's positions in the round
    auto load = [&](int round) {
        const int j0 = round * kSpan + tid * kPer;        // below 2^31: lengths end 2^16 before it
        if (whole_vectors && j0 + kPer <= n && j0 + kPer <= a.ld_mass) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(m + j0 + i);
                v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = j0 + i < n ? mass_at(j0 + i) : 0.0f;
    };
    load(0);
    uint32_t need = (uint32_t)(a.budget - a.sinks - a.recent), prefix = 0;
    const bool choose = need > 0;
    bool sharp = false;                                   // keys from `prefix` on are kept, no ties
    for (int shift = 24; need > 0 && !sharp && shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int r = 0; r < rounds; ++r) {
            if (rounds > 1) load(r);
            const int j0 = r * kSpan + tid * kPer;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t k = mass_key(v[i]);
                const bool on = j0 + i >= lo && j0 + i < hi && (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)));
                if (__any_sync(0xFFFFFFFFu, on)) count_digit(hist, (k >> shift) & 255u, on);
            }
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: digits 255 - 8 l downwards; the counts sum to at least `need`
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
            uint32_t before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, before, o);
                if (lane >= o) before += y;
            }
            before -= sum;
            if (before < need && need <= before + sum) {
                uint32_t left = need - before, i = 0;
                while (c[i] < left) left -= c[i++];
                s_digit = 255u - 8u * lane - i;
                s_left = left;
                s_count = c[i];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_left;
        sharp = s_count == need && prefix > 0;            // the whole digit is kept
    }
    if (sharp) {                                          // "above prefix - 1", and no ties
        prefix -= 1;
        need = 0;
    }
    uint64_t base = 0;                                    // sure ones, and ties in the upper half, so far
    for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
        const int j0 = r * kSpan + tid * kPer;
        uint32_t sure = 0, tie = 0;                       // bits of this thread's positions
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = j0 + i;
            const uint32_t k = mass_key(v[i]);
            const bool in = j >= lo && j < hi;
            if (j < n && (!in || (choose && k > prefix))) sure |= 1u << i;
            if (choose && in && k == prefix) tie |= 1u << i;
        }
        uint64_t x = (uint64_t)__popc(sure) | (uint64_t)__popc(tie) << 32;
        const uint64_t own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        uint64_t at = base + x - own;
        for (int w = 0; w < kSel / 32; ++w) {
            if (w < warp) at += s_warp[w];
            base += s_warp[w];
        }
        uint32_t ns = (uint32_t)at, nt = (uint32_t)(at >> 32);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool t = (tie >> i) & 1u, k = ((sure >> i) & 1u) || (t && nt < need);
            const uint32_t to = ns + min(nt, need);
            if (k && to < (uint32_t)a.budget) {
                kept[to] = j0 + i;
                if (to < a.ld_out) mo[to] = v[i];
            }
            ns += (sure >> i) & 1u;
            nt += t;
        }
    }
}

// V: 16 or 8 bytes.  Dynamic shared memory: source slots [positions][H], target
// slots [positions].
template <typename V>
__global__ void __launch_bounds__(256)
k_evict_copy(const PagedView pv, const EvictArgs a, uint8_t *kc, float *ks, uint8_t *vc, float *vs, int positions,
             FastDiv chunks, FastDiv heads) {
    extern __shared__ int s_src[];
    const int64_t b = blockIdx.y;
    const int H = pv.H, p0 = (int)blockIdx.x * positions, tid = threadIdx.x;
    pdl_wait();
    if (blockIdx.x == 0 && tid == 0) {
        const int n = pv.length(b);
        a.lens_out[b] = n < a.budget ? n : a.budget;
    }
    const int count = min(positions, a.budget - p0), rows = count * H;
    // slot that row (r, h) comes from: -1 no page (zeros), -2 nothing to copy; a warp reads consecutive r of one head
    for (int h = tid >> 5; h < H; h += 8)
        for (int r = tid & 31; r < count; r += 32) {
            const int j = a.kept[(b * H + h) * a.budget + p0 + r];
            s_src[r * H + h] = j < 0 ? -2 : pv.slot(b, j);
        }
    int *s_dst = s_src + positions * H;                   // -1: no page
    for (int r = tid; r < count; r += 256) {
        const uint32_t p = (uint32_t)(p0 + r), pg = pv.bs.div(p);
        const int32_t blk = pg < a.dst_max_blocks ? a.dst_table[b * a.dst_max_blocks + pg] : -1;
        s_dst[r] = blk < 0 || blk >= pv.num_blocks ? -1 : (int)((uint32_t)blk * pv.bs.d + (p - pg * pv.bs.d));
    }
    __syncthreads();
    const int C = (int)chunks.d, total = rows * C;
    const V *kin = reinterpret_cast<const V *>(kc), *vin = reinterpret_cast<const V *>(vc);
    V *kout = reinterpret_cast<V *>(kc), *vout = reinterpret_cast<V *>(vc);
    constexpr int U = 4;
    for (int x0 = tid; x0 < total; x0 += 256 * U) {
        V k[U], v[U];
        int64_t to[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int x = x0 + 256 * i;
            to[i] = -1;
            k[i] = v[i] = V{};
            if (x >= total) continue;
            const int q = (int)chunks.div((uint32_t)x), c = x - q * C, r = (int)heads.div((uint32_t)q), h = q - r * H;
            const int s = s_src[q], d = s_dst[r];
            if (s == -2 || d < 0) continue;
            to[i] = (int64_t)d * (H * C) + (h * C + c);
            if (s >= 0) {
                const int64_t from = (int64_t)s * (H * C) + (h * C + c);
                k[i] = kin[from];
                v[i] = vin[from];
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (to[i] >= 0) {
                kout[to[i]] = k[i];
                vout[to[i]] = v[i];
            }
    }
    for (int q = tid; q < rows; q += 256) {
        const int r = (int)heads.div((uint32_t)q), h = q - r * H, s = s_src[q];
        const int64_t d = s_dst[r];
        if (s == -2 || d < 0) continue;
        ks[d * H + h] = s >= 0 ? ks[(int64_t)s * H + h] : 0.0f;
        vs[d * H + h] = s >= 0 ? vs[(int64_t)s * H + h] : 0.0f;
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
    if (budget < 1 || budget > kPagedMaxContext || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks ||
        ld_out < 0)
        return FP8_ERR_SHAPE;
    if (max_blocks > kPagedMaxContext / block_size || dst_max_blocks > kPagedMaxContext / block_size)
        return FP8_ERR_SHAPE;
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
    cudaError_t e = pdl_launch(k_evict_select, dim3((unsigned)(B * H)), dim3(kSel), 0, s, pv, a);
    if (e != cudaSuccess) return FP8_ERR_CUDA;
    // rows per CTA: enough CTAs for every SM to hold several, at most 1024 rows each
    const int64_t want = std::min<int64_t>(1024, std::max<int64_t>(64, B * budget * H / (8 * (int64_t)sms)));
    const int positions = (int)std::min<int64_t>(budget, std::max<int64_t>(1, want / H));
    const dim3 grid((unsigned)((budget + positions - 1) / positions), (unsigned)B);
    const size_t smem = (size_t)positions * (H + 1) * 4;  // at most 2048 slots: 8 KiB
    const int bytes = Dh % 16 ? 8 : 16;
    const FastDiv chunks = make_fastdiv((uint32_t)(Dh / bytes)), heads = make_fastdiv((uint32_t)H);
    if (bytes == 16)
        e = pdl_launch(k_evict_copy<uint4>, grid, dim3(256), smem, s, pv, a, k_cache, k_scale, v_cache, v_scale,
                       positions, chunks, heads);
    else
        e = pdl_launch(k_evict_copy<uint2>, grid, dim3(256), smem, s, pv, a, k_cache, k_scale, v_cache, v_scale,
                       positions, chunks, heads);
    return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}
