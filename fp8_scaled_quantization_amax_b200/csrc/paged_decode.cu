// paged_decode.cu -- attention of one new token per sequence over the paged
// FP8 KV cache.
//
// Per KV head the work is S^T = K Q^T (positions x query heads of the group),
// a softmax over the positions and O^T = V^T P^T.  Every K and V byte is used
// once per group of query heads, so the kernel is bound by reading the cache:
// what it has to reach is the HBM rate, and what stands against that is the
// instructions spent on each byte.  Hence:
//   * a warp owns one KV head and 32 positions at a time.  Its K and V tiles
//     come by TMA into a ring in shared memory (boxes of 8, 16 or 32 rows of one
//     head, whatever divides the page size; pages of another size take
//     cp.async into the same layout), with no other warp to wait for;
//   * the copied bytes are matrix fragments as they lie: any permutation of
//     the head elements is allowed in K Q^T when Q is permuted alike (lane t of
//     a row takes whole 16-byte chunks), and any permutation of V's columns
//     only permutes the rows of O^T, so nothing is transposed but V's pairs of
//     positions (one byte permute per four codes);
//   * E4M3 and E5M2 codes are exact in fp16 (one conversion per two codes), so
//     the products run as mma.m16n8k16 on fp16 with fp32 sums (N = 8 query
//     heads fits a group; the tensor rate is not the bound).  The rows' scales
//     multiply the logits and the weights, in fp32, per position;
//   * Q's rows are brought to [2^14, 2^15) by a power of two before they become
//     fp16, which is then exact for every element above 2^-24 of the row's
//     largest; the weights times V's scales are normalised by a running power
//     of two of each query head, so that fp16 holds them to 2^-11 down to 2^-19
//     of the largest product (a large scale that hardly weighs does not count);
//   * the maximum is only moved when a logit passes it by 2^6 (one vote per
//     tile instead of shuffles); weights stay below 2^6, far inside fp16.
//
// Split: the tiles of all (sequence, block of heads) are laid end to end and
// every CTA takes an equal, contiguous run of them, whatever the lengths (they
// are only known on the device).  A CTA that covers all of a row's tiles
// writes its result; otherwise it leaves (O, max, sum) in the workspace and
// k_decode_join adds the parts in the order of the CTAs.  At most two parts
// per CTA, so the workspace does not grow with the batch.
//
// Measured on a B200 with L2 flushed: 32 sequences of up to 8192 tokens, 32
// heads of 128, 1.12 GB in 202 - 205 us (5.5 TB/s, 0.85 of a copy); one of 131072
// tokens, 8 heads with 8 query heads each, 277 MB in 60 - 62 us, 12 of those before
// the first and after the last tile.  Tiles by TMA instead of cp.async: 306 -> 235
// us and 118 -> 97 us when they came in; pages of 100 take 236 - 247 us today.
#include <algorithm>
#include <atomic>

#include "paged_attn.cuh"

using namespace fp8q;

namespace {

constexpr int kTile = 32;                    // positions per warp and step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.0e38f;           // before the first logit; below every finite logit that matters
constexpr float kLazy = 6.0f;                // log2 of how far a logit may pass the maximum in use
constexpr int kMaxUnit = 120;                // log2 of the largest power of two on the weights: 2^kLazy of them are finite

struct DecodeArgs {
    const __nv_bfloat16 *q;
    int64_t ld_q;
    int box;                 // rows per TMA box: 8, 16 or 32
    int B, G, GC, HB;        // query heads per KV head; chunks of them; (virtual) heads per CTA
    float scale;
    __nv_bfloat16 *out;
    float *lse;              // [B, Hq]
    float *part;             // two parts per CTA
    int2 *span;              // [B, rows]: first and last CTA of each row with tiles
    float *logits;           // weights' scratch [B, H * GC, vis_max, 8 * NT] (log2 units), or nullptr
    int64_t vis_max;
    float *mass;
    int64_t ld_mass;
    float decay;
};

// A warp's ring of UNITS tile halves: K of 32 positions, then V of the same,
// each with its 32 scales (and, K, the mask of live positions).  Three halves
// keep two (8 KiB at a head size of 128) in flight per warp, which at 16 warps
// is 134 KiB per SM, more than the HBM rate needs at its latency.
template <int DH, int NT>
struct Cfg {
    static constexpr int WARPS = (DH <= 128 && NT == 1) ? 16 : 8;   // 128 registers a thread, or 255
    static constexpr int UNIT = 32 * DH, AUX = 128 + 16;
    static constexpr int UNITS = DH == 64 ? 6 : DH == 128 ? (NT == 1 ? 3 : 6) : 3;
    static constexpr int AUX_OFF = WARPS * UNITS * UNIT, BAR_OFF = AUX_OFF + WARPS * UNITS * AUX;
    static constexpr size_t SMEM = 1024 + BAR_OFF + WARPS * UNITS * 8;
    static constexpr int COLS = 8 * NT;                  // query heads per chunk
    static_assert(UNITS * UNIT >= COLS * DH * 4, "the warps' results are merged in the pipeline's memory");
};

// copies BYTES, or writes zeros when !live
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool live) {
    const int n = live ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Visible positions of the one query of sequence b: [0, sinks) and [begin, n).
// Its tiles hold 32 aligned positions each: those of the sinks, then those of
// the window, without the ones that are already there.
struct Visible {
    int begin, sinks, n, sink_tiles, first_tile, tiles;
    __device__ __forceinline__ int position(int tile) const {   // first of a tile
        return (tile < sink_tiles ? tile : first_tile + (tile - sink_tiles)) * kTile;
    }
    __device__ __forceinline__ bool sees(int j) const { return j < n && (j >= begin || j < sinks); }
};
__device__ __forceinline__ Visible visible_of(const PagedView &pv, int64_t b) {
    Visible v;
    v.n = pv.length(b);
    v.begin = pv.window_begin(v.n - 1);
    v.sinks = min(pv.sinks, v.begin);
    v.first_tile = v.begin / kTile;
    v.sink_tiles = min((int)(((uint32_t)v.sinks + kTile - 1) / kTile), v.first_tile);
    v.tiles = v.sink_tiles + (int)(((uint32_t)v.n + kTile - 1) / kTile) - v.first_tile;
    return v;
}

// Tiles of WT * 32 positions laid end to end: rows (b, hb) with b slowest, as
// many tiles in each row of a sequence as its visible positions fill.
__device__ __forceinline__ int tiles_of(const PagedView &pv, int64_t b, int WT) {
    return (visible_of(pv, b).tiles + WT - 1) / WT;
}
__device__ int64_t block_scan(int64_t v, int64_t *buf, int64_t *total) {   // exclusive
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    int64_t base = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) base += buf[w];
        all += buf[w];
    }
    *total = all;
    return base + x - v;
}
// Block-wide: the tiles of all sequences.
__device__ int64_t count_tiles(const PagedView &pv, int B, int WT, int rows, int64_t *buf) {
    int64_t all = 0, total;
    for (int i = threadIdx.x; i < B; i += blockDim.x) all += (int64_t)tiles_of(pv, i, WT) * rows;
    block_scan(all, buf, &total);
    return total;
}

// First tile of CTA c of n when `total` tiles are dealt out evenly.
__device__ __forceinline__ int64_t deal(int64_t total, int64_t n, int64_t c) { return total * c / n; }

// TMA: boxes of a.box rows, which divides the page size; otherwise cp.async.
template <int FMT, int DH, int NT, bool TMA>
__global__ void __launch_bounds__(Cfg<DH, NT>::WARPS * 32, 1)
k_decode(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedView pv,
         const DecodeArgs a) {
    using C = Cfg<DH, NT>;
    constexpr int kWarps = C::WARPS;
    constexpr int KC = DH / 64;              // 16-byte chunks of a K row per lane
    constexpr int VB = DH / 8;               // V bytes of a position per lane
    constexpr int KS = DH / 16;              // k steps of K Q^T
    constexpr int MI = DH / 16;              // row blocks of O^T
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint32_t s_abort;
    __shared__ int64_t scan_buf[kWarps], s_before;
    __shared__ int s_b;
    __shared__ float s_m[kWarps][C::COLS], s_l[kWarps][C::COLS];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int WT = kWarps / a.HB;            // warps that share a head, a tile of positions each
    const int hw = warp / WT, wt = warp % WT;
    const int VH = pv.H * a.GC, rows = VH / a.HB;
    const uint32_t data = smem_u32(smem) + (uint32_t)(warp * C::UNITS * C::UNIT);
    const uint32_t aux = smem_u32(smem) + (uint32_t)(C::AUX_OFF + warp * C::UNITS * C::AUX);
    const uint32_t bars = smem_u32(smem) + (uint32_t)(C::BAR_OFF + warp * C::UNITS * 8);
    if (TMA && lane == 0) {
        for (int u = 0; u < C::UNITS; ++u) mbar_init(bars + 8 * u, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (warp == 0) {
            s_abort = 0u;
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
        }
    }
    pdl_wait();
    pdl_trigger();

    // the first of this CTA's tiles: its sequence, and the tiles before that
    int64_t total;
    int64_t mine = 0;
    if (a.B <= kWarps * 32) {
        if (threadIdx.x < a.B) mine = (int64_t)tiles_of(pv, threadIdx.x, WT) * rows;
    } else {
        total = count_tiles(pv, a.B, WT, rows, scan_buf);
    }
    int64_t pre = 0;
    if (a.B <= kWarps * 32) pre = block_scan(mine, scan_buf, &total);
    const int64_t ncta = min((int64_t)gridDim.x, total);
    if ((int64_t)blockIdx.x >= ncta) return;
    int64_t at = deal(total, ncta, blockIdx.x);
    const int64_t end = deal(total, ncta, blockIdx.x + 1);
    for (int64_t b0 = 0, base = 0;; b0 += kWarps * 32) {
        if (a.B > kWarps * 32) {
            const int64_t bb = b0 + threadIdx.x;
            mine = bb < a.B ? (int64_t)tiles_of(pv, bb, WT) * rows : 0;
            int64_t all;
            pre = base + block_scan(mine, scan_buf, &all);
            base += all;
        } else {
            base = total;
        }
        if (at >= pre && at < pre + mine) {
            s_b = (int)(b0 + threadIdx.x);
            s_before = pre;
        }
        if (at < base) break;                 // at < total: some round ends here
    }
    __syncthreads();
    int b = s_b;
    Visible vis = visible_of(pv, b);
    int nt = (vis.tiles + WT - 1) / WT;
    int row = (int)((at - s_before) / nt), tile = (int)((at - s_before) % nt);

    const uint32_t row_bytes = (uint32_t)(pv.H * pv.Dh);
    // Byte of a unit where chunk c (16 bytes) of row r lies: 128-byte rows (two
    // blocks of them for 256), 64-byte rows, in TMA's swizzle of the same width.
    auto at_chunk = [](int r, int c) -> uint32_t {
        if (DH == 64) return (uint32_t)(r * 64 + ((c ^ (r >> 1)) & 3) * 16);
        return (uint32_t)((c >> 3) * 4096 + r * 128 + ((c ^ r) & 7) * 16);
    };
    // chunk of a K row that lane t takes as its c-th: even and odd rows then meet different banks
    auto k_chunk = [](int t, int c) { return DH == 64 ? t : (c >> 1) * 8 + 2 * t + (c & 1); };
    int fill = 0, read = 0;                   // units of the ring to copy into and to read
    uint32_t phase = 0;                       // parity of the unit to read
    bool dead = false;                        // a wait of this warp ran out: nothing more is copied or computed

    while (true) {
        const int tile_end = (int)min((int64_t)nt, tile + (end - at));
        const int vh = row * a.HB + hw, h = vh / a.GC, chunk = vh % a.GC;

        float o[NT][MI][4], m[NT][2], l[NT][2], vs[NT][2];   // O^T is held times the power of two vs
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][i][e] = 0.0f;
            m[x][0] = m[x][1] = kNoMax;
            l[x][0] = l[x][1] = 0.0f;
            vs[x][0] = vs[x][1] = pow2i(kMaxUnit);
        }

        const uint8_t *kh = pv.kc + (int64_t)h * pv.Dh + 16 * t, *vhp = pv.vc + (int64_t)h * pv.Dh + 16 * t;
        const float *ksh = pv.ks + h, *vsh = pv.vs + h;
        const int ntile = tile_end - tile;
        // The tile whose copies come next: this lane's position in it, its slot and whether it is visible.  The
        // page id is loaded half a tile before it is looked at.
        int fetch = tile, j = 0, blk = -1, slot = -1;
        bool live = false;
        auto look_up = [&] {
            const int i = fetch * WT + wt;
            j = i < vis.tiles ? vis.position(i) + lane : vis.n;
            blk = j < vis.n ? __ldg(pv.table + (int64_t)b * pv.max_blocks + pv.bs.div((uint32_t)j)) : -1;
        };
        auto look_at = [&] {
            slot = blk >= 0 && blk < pv.num_blocks
                       ? (int)((uint32_t)blk * pv.bs.d + ((uint32_t)j - pv.bs.div((uint32_t)j) * pv.bs.d))
                       : -1;
            live = slot >= 0 && vis.sees(j);
        };
        // K or V of that tile into the next unit
        auto issue = [&](const CUtensorMap *map, const uint8_t *codes, const float *scales, bool is_k) {
            if (fetch < tile_end && !dead) {  // the same for all lanes
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, live);
                const uint32_t dst = data + (uint32_t)(fill * C::UNIT), ax = aux + (uint32_t)(fill * C::AUX);
                if constexpr (TMA) {
                    const uint32_t bar = bars + 8 * fill;
                    if (lane == 0) mbar_expect_tx(bar, C::UNIT);
                    if ((lane & (a.box - 1)) == 0) {
                        // a box without a visible row starts past the last slot: zeros, and nothing is read
                        const bool any = (mask >> lane) & (0xFFFFFFFFu >> (32 - a.box));
                        const int z = any && slot >= 0 ? slot : (int)(pv.bs.d * (uint32_t)pv.num_blocks);
                        tma_load_3d(dst + (uint32_t)(lane * (DH == 64 ? 64 : 128)), map, bar, 0, h, z);
                        if (DH == 256) tma_load_3d(dst + 4096u + (uint32_t)(lane * 128), map, bar, 128, h, z);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = __shfl_sync(0xFFFFFFFFu, live ? slot : -1, g + 8 * r);
                        const uint8_t *src = codes + (uint64_t)(uint32_t)max(s, 0) * row_bytes;
#pragma unroll
                        for (int c = 0; c < KC; ++c)
                            cp_async<16>(dst + at_chunk(g + 8 * r, t + 4 * c), src + 64 * c,
                                         s >= 0 && 16 * (t + 4 * c) < pv.Dh);
                    }
                }
                cp_async<4>(ax + 4 * lane, scales + (uint64_t)(uint32_t)max(slot, 0) * (uint32_t)pv.H, live);
                if (is_k && lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(ax + 128), "r"(mask) : "memory");
                fill = fill + 1 == C::UNITS ? 0 : fill + 1;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto issue_k = [&] {
            look_at();
            issue(&tmK, kh, ksh, true);
        };
        auto issue_v = [&] {
            issue(&tmV, vhp, vsh, false);
            ++fetch;
            look_up();
        };
        auto next_read = [&] {
            if (++read == C::UNITS) {
                read = 0;
                phase ^= 1u;
            }
        };
        // The copies of the unit to read have landed.  Where that wait runs out the warp waits (again with a limit) for
        // every copy it has in flight, so that none lands in memory that has another use by then.
        auto landed = [&]() -> bool {
            if constexpr (TMA) {
                if (__all_sync(0xFFFFFFFFu, wait_bar(bars + 8 * read, phase, &s_abort, kErrProducer))) return true;
                dead = true;
                uint32_t at_phase = phase;
                for (int u = read, left = fill > read ? fill - read : fill - read + C::UNITS; left > 0; --left) {
                    wait_bar_drain(bars + 8 * u, at_phase);
                    if (++u == C::UNITS) {
                        u = 0;
                        at_phase ^= 1u;
                    }
                }
                __syncwarp();
                return false;
            }
            return true;
        };
        look_up();
        // the ring's last unit is filled when the one that was read before it is done with
#pragma unroll
        for (int u = 0; u < C::UNITS - 1; ++u) {
            if (u % 2 == 0) issue_k(); else issue_v();
        }

        // ---- Q: this warp's chunk of the group, as fp16 fragments
        uint32_t qf[NT][KS][2];
        float cf[NT][2];                      // logit factor (log2 units) of columns 2t, 2t + 1
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int gi = chunk * C::COLS + x * 8 + g;
            const __nv_bfloat16 *qp = a.q + (int64_t)b * a.ld_q + (int64_t)(h * a.G + gi) * pv.Dh;
            uint4 w[KC][2];
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int d0 = 16 * k_chunk(t, c);
                const bool live = gi < a.G && d0 < pv.Dh;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[c][e] = live ? *reinterpret_cast<const uint4 *>(qp + d0 + 8 * e) : make_uint4(0, 0, 0, 0);
                    uint32_t bad = 0;
                    mx = amax_exact8(mx, w[c][e], bad);       // finite elements only
                }
            }
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int ex = max((int)(mx >> 7), 14) - 127;     // exponent of the row's largest, at least 2^-113
            const float up = pow2i(14 - ex);
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint32_t ww[8] = {w[c][0].x, w[c][0].y, w[c][0].z, w[c][0].w,
                                        w[c][1].x, w[c][1].y, w[c][1].z, w[c][1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qf[x][c * 4 + i][e] = pack_f16x2(bf_lo(ww[2 * i + e]) * up, bf_hi(ww[2 * i + e]) * up);
            }
            const float f = a.scale * kLog2e * pow2i(ex) * 0x1p-14f;
            cf[x][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * t);
            cf[x][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4);
        }

        for (int k = 0; k < ntile && !dead; ++k) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::UNITS - 2) : "memory");
            __syncwarp();                     // the other lanes' copies; and the unit read before is done with
            if constexpr (C::UNITS % 2) issue_k(); else issue_v();
            uint32_t un = data + (uint32_t)(read * C::UNIT), ax = aux + (uint32_t)(read * C::AUX), seen;
            if (!landed()) break;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(seen) : "r"(ax + 128));

            // ---- S^T = K Q^T, 16 positions at a time
            float s[2][NT][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int x = 0; x < NT; ++x) s[y][x][0] = s[y][x][1] = s[y][x][2] = s[y][x][3] = 0.0f;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint4 k0 = lds128(un + at_chunk(16 * y + g, k_chunk(t, c)));
                    const uint4 k1 = lds128(un + at_chunk(16 * y + g + 8, k_chunk(t, c)));
                    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a0, a1, a2, a3;
                        to_f16x4<FMT>(w0[i], a0, a2);
                        to_f16x4<FMT>(w1[i], a1, a3);
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            mma16816(s[y][x], a0, a1, a2, a3, qf[x][c * 4 + i][0], qf[x][c * 4 + i][1]);
                    }
                }
            }
            // ---- logits in log2 units; what is not visible becomes -inf
            bool up = false;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float dk0 = k_factor(lds_f(ax + 4 * (16 * y + g)));
                const float dk1 = k_factor(lds_f(ax + 4 * (16 * y + g + 8)));
#pragma unroll
                for (int x = 0; x < NT; ++x) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[y][x][e] *= dk0 * cf[x][e];
                        s[y][x][2 + e] *= dk1 * cf[x][e];
                    }
                }
            }
            if (seen != 0xFFFFFFFFu) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        if (!((seen >> (16 * y + g)) & 1u)) s[y][x][0] = s[y][x][1] = -INFINITY;
                        if (!((seen >> (16 * y + g + 8)) & 1u)) s[y][x][2] = s[y][x][3] = -INFINITY;
                    }
            }
            if (a.logits) {
                const int i0 = (tile + k) * WT + wt;
                float *lp = a.logits + (((int64_t)b * VH + vh) * a.vis_max + (int64_t)i0 * kTile + g) * C::COLS + 2 * t;
                if (i0 < vis.tiles) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            *reinterpret_cast<float2 *>(lp + 8 * y * C::COLS + 8 * x) =
                                make_float2(s[y / 2][x][2 * (y & 1)], s[y / 2][x][2 * (y & 1) + 1]);
                }
            }
            float mx[NT][2];
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[x][e] = fmaxf(fmaxf(s[0][x][e], s[0][x][2 + e]), fmaxf(s[1][x][e], s[1][x][2 + e]));
                    up |= mx[x][e] > m[x][e] + kLazy;
                }
            if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(m[x][e], mx[x][e]);
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
                        // what O^T holds shrinks by 2^dm: its power of two grows by as many whole steps as the
                        // maximum passes, which come to within one of it however often it moves
                        const float dm = m[x][e] - v;
                        const int was = (int)(__float_as_uint(vs[x][e]) >> 23) - 127;
                        const int now = min(kMaxUnit, was + (int)fminf(floorf(v) - floorf(m[x][e]), 1000.0f));
                        m[x][e] = v;
                        l[x][e] *= exp2_fast(dm);
                        vs[x][e] = pow2i(now);
                        const float al = exp2_fast(dm + (float)(now - was));
#pragma unroll
                        for (int i = 0; i < MI; ++i) {
                            o[x][i][e] *= al;
                            o[x][i][2 + e] *= al;
                        }
                    }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[y][x][e] = exp2_fast(s[y][x][e] - m[x][e & 1]);
                        l[x][e & 1] += s[y][x][e];
                    }
            next_read();

            asm volatile("cp.async.wait_group %0;" ::"n"(C::UNITS - 2) : "memory");
            __syncwarp();
            if constexpr (C::UNITS % 2) issue_v(); else issue_k();
            un = data + (uint32_t)(read * C::UNIT);
            ax = aux + (uint32_t)(read * C::AUX);
            if (!landed()) break;
            // ---- weights times V's scales, under the power of two that keeps them in fp16
            float dv[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) dv[y] = lds_f(ax + 4 * (8 * y + g));
            const float dmax = fmaxf(fmaxf(fabsf(dv[0]), fabsf(dv[1])), fmaxf(fabsf(dv[2]), fabsf(dv[3])));
            float vmax = vs[0][0];
#pragma unroll
            for (int x = 0; x < NT; ++x) vmax = fmaxf(vmax, fmaxf(vs[x][0], vs[x][1]));
            if (__any_sync(0xFFFFFFFFu, dmax * vmax >= 512.0f && dmax < INFINITY)) {   // else below 2^9 2^kLazy = 2^15
                // the largest product of each query head, to [2^6, 2^7) where it is more: scales up to four times
                // as large do not come here again
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = 0.0f;             // times 2^-16, which keeps it finite
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float w = fabsf(s[y / 2][x][2 * (y & 1) + e] * (dv[y] * 0x1p-16f));
                            top = fmaxf(top, w < INFINITY ? w : 0.0f);
                        }
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const int was = (int)(__float_as_uint(vs[x][e]) >> 23) - 127;
                        const int now = min(was, -10 - ((int)(__float_as_uint(top) >> 23) - 127));
                        const float r = exp2_fast((float)(now - was));
                        vs[x][e] = pow2i(now);
#pragma unroll
                        for (int i = 0; i < MI; ++i) {
                            o[x][i][e] *= r;
                            o[x][i][2 + e] *= r;
                        }
                    }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        pb[y][x][e] = transpose8x8(pack_f16x2(s[y][x][2 * e] * vs[x][0] * dv[2 * y + e],
                                                              s[y][x][2 * e + 1] * vs[x][1] * dv[2 * y + e]));
            // ---- O^T += V^T P^T.  A weight of zero does not hide what a slot that is not visible holds (it
            // may be a NaN code): such rows of a box become zeros, each by the lane that reads it next.
            if (TMA && seen != 0xFFFFFFFFu) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = 2 * t + (e & 1) + 4 * (e & 2) + 4 * (e & 4);
                    if (!((seen >> r) & 1u)) {
                        if constexpr (VB == 8) {
                            asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(un + at_chunk(r, g >> 1) + 8 * (g & 1)),
                                         "r"(0) : "memory");
                        } else {
#pragma unroll
                            for (int c = 0; c < VB / 16; ++c)
                                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(un + at_chunk(r, 8 * c + g)),
                                             "r"(0) : "memory");
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the unit's next copy comes by TMA
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int c = 0; c < (VB + 15) / 16; ++c) {
                    uint32_t v[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 16 * y + 2 * t + (e & 1) + 4 * (e & 2);
                        if constexpr (VB == 8) {
                            const uint2 w = lds64(un + at_chunk(r, g >> 1) + 8 * (g & 1));
                            v[e][0] = w.x; v[e][1] = w.y;
                        } else {
                            const uint4 w = lds128(un + at_chunk(r, 8 * c + g));
                            v[e][0] = w.x; v[e][1] = w.y; v[e][2] = w.z; v[e][3] = w.w;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < (VB == 8 ? 2 : 4); ++w)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t sel = hf ? 0x7362u : 0x5140u;
                            const uint32_t xx = __byte_perm(v[0][w], v[1][w], sel);
                            const uint32_t yy = __byte_perm(v[2][w], v[3][w], sel);
                            uint32_t a0, a1, a2, a3;
                            to_f16x4<FMT>(xx, a0, a1);
                            to_f16x4<FMT>(yy, a2, a3);
#pragma unroll
                            for (int x = 0; x < NT; ++x)
                                mma16816(o[x][c * 8 + w * 2 + hf], a0, a1, a2, a3, pb[y][x][0], pb[y][x][1]);
                        }
                }
            next_read();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");

        // ---- this run of tiles is done: result, or a part of one
        // o[..][i] holds the head elements dh_of(i) and the next one
        auto dh_of = [&](int i) { return VB == 8 ? 8 * g + 2 * i : 128 * (i >> 3) + 16 * g + 2 * (i & 7); };
        float inv[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                inv[x][e] = 1.0f / vs[x][e];
                float v = l[x][e];
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
                l[x][e] = v;
            }
        const bool whole = tile == 0 && tile_end == nt;
        if (tile == 0 && threadIdx.x == 0) {
            // CTA c holds the tiles [total * c / ncta, total * (c + 1) / ncta): the one with tile x is the largest c
            // with total * c / ncta <= x, that is c <= (x * ncta + ncta - 1) / total
            const int64_t last = whole ? blockIdx.x : ((at + nt - 1) * ncta + ncta - 1) / total;
            a.span[(int64_t)b * rows + row] = make_int2(blockIdx.x, (int)last);
        }
        float *part = a.part + ((int64_t)blockIdx.x * 2 + (tile == 0 ? 1 : 0)) * a.HB * C::COLS * (DH + 2);
        // column c of head hw: DH sums, then (max, sum) behind all columns' sums
        float *part_ml = part + (int64_t)a.HB * C::COLS * DH;
        if (WT == 1) {
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = 8 * x + 2 * t + e, gi = chunk * C::COLS + col;
                    if (gi >= a.G) continue;
                    if (whole) {
                        const float r = l[x][e] == 0.0f ? 0.0f : inv[x][e] / l[x][e];
                        const int64_t orow = (int64_t)b * pv.H * a.G + h * a.G + gi;
                        if (g == 0) a.lse[orow] = l[x][e] == 0.0f ? -INFINITY : (m[x][e] + log2f(l[x][e])) * kLn2;
                        __nv_bfloat16 *op = a.out + orow * pv.Dh;
#pragma unroll
                        for (int c = 0; c < VB / 8; ++c)
                            if (dh_of(4 * c) < pv.Dh) {
                                uint4 w;
                                w.x = pack_bf16x2(o[x][4 * c][e] * r, o[x][4 * c][2 + e] * r);
                                w.y = pack_bf16x2(o[x][4 * c + 1][e] * r, o[x][4 * c + 1][2 + e] * r);
                                w.z = pack_bf16x2(o[x][4 * c + 2][e] * r, o[x][4 * c + 2][2 + e] * r);
                                w.w = pack_bf16x2(o[x][4 * c + 3][e] * r, o[x][4 * c + 3][2 + e] * r);
                                *reinterpret_cast<uint4 *>(op + dh_of(4 * c)) = w;
                            }
                    } else {
                        const int pc = hw * C::COLS + col;
                        if (g == 0) *reinterpret_cast<float2 *>(part_ml + 2 * pc) = make_float2(m[x][e], l[x][e]);
                        float *pp = part + (int64_t)pc * DH;
#pragma unroll
                        for (int i = 0; i < MI; i += 2)
                            *reinterpret_cast<float4 *>(pp + dh_of(i)) =
                                make_float4(o[x][i][e] * inv[x][e], o[x][i][2 + e] * inv[x][e],
                                            o[x][i + 1][e] * inv[x][e], o[x][i + 1][2 + e] * inv[x][e]);
                    }
                }
        } else {
            __syncthreads();                  // every warp's copies have landed and been read
            float *mine = reinterpret_cast<float *>(smem + (size_t)warp * C::UNITS * C::UNIT);
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = 8 * x + 2 * t + e;
                    if (g == 0) {
                        s_m[warp][col] = m[x][e];
                        s_l[warp][col] = l[x][e];
                    }
#pragma unroll
                    for (int i = 0; i < MI; ++i)
                        *reinterpret_cast<float2 *>(mine + col * DH + dh_of(i)) =
                            make_float2(o[x][i][e] * inv[x][e], o[x][i][2 + e] * inv[x][e]);
                }
            __syncthreads();
            // four elements per thread and step
            for (int idx = threadIdx.x; idx < a.HB * C::COLS * (DH / 4); idx += kWarps * 32) {
                const int d = idx % (DH / 4) * 4, pc = idx / (DH / 4), col = pc % C::COLS, hh = pc / C::COLS;
                const int vh2 = row * a.HB + hh, gi = vh2 % a.GC * C::COLS + col;
                if (gi >= a.G) continue;
                float mx = kNoMax;
                for (int w = 0; w < WT; ++w) mx = fmaxf(mx, s_m[hh * WT + w][col]);
                float sum = 0.0f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int w = 0; w < WT; ++w) {
                    const float al = exp2_fast(s_m[hh * WT + w][col] - mx);
                    const float4 v = *reinterpret_cast<const float4 *>(
                        smem + (size_t)(hh * WT + w) * C::UNITS * C::UNIT + (size_t)(col * DH + d) * 4);
                    sum = fmaf(s_l[hh * WT + w][col], al, sum);
                    acc.x = fmaf(v.x, al, acc.x); acc.y = fmaf(v.y, al, acc.y);
                    acc.z = fmaf(v.z, al, acc.z); acc.w = fmaf(v.w, al, acc.w);
                }
                if (whole) {
                    const int64_t orow = (int64_t)b * pv.H * a.G + vh2 / a.GC * a.G + gi;
                    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
                    if (d == 0) a.lse[orow] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
                    if (d < pv.Dh)
                        *reinterpret_cast<uint2 *>(a.out + orow * pv.Dh + d) =
                            make_uint2(pack_bf16x2(acc.x * r, acc.y * r), pack_bf16x2(acc.z * r, acc.w * r));
                } else {
                    if (d == 0) *reinterpret_cast<float2 *>(part_ml + 2 * pc) = make_float2(mx, sum);
                    *reinterpret_cast<float4 *>(part + (int64_t)pc * DH + d) = acc;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();                  // before the next run's copies
        }

        at += tile_end - tile;
        if (at >= end) break;
        tile = 0;
        if (++row == rows) {
            row = 0;
            do {
                ++b;                          // at < end <= total: another sequence with tiles follows
                vis = visible_of(pv, b);
            } while (vis.tiles == 0);
            nt = (vis.tiles + WT - 1) / WT;
        }
    }
}

// Joins the parts of the rows that more than one CTA worked on, and writes the
// results of queries that see nothing.  One CTA per (sequence, query head, 32
// head elements): 8 lanes read 128 bytes of a part, so a warp has 4 parts in
// each of 10 loads and one round takes a row that 160 CTAs have a part of.
constexpr int kJoinWarps = 4;
template <int DH, int COLS>
__global__ void __launch_bounds__(kJoinWarps * 32)
k_decode_join(const PagedView pv, const DecodeArgs a) {
    constexpr int SL = DH / 32, R = 4 * kJoinWarps, U = 10;
    __shared__ float4 s_acc[R][8];
    __shared__ float s_sum[R], s_max[R];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> 3, q4 = lane & 7, r = warp * 4 + sub;
    const int Hq = pv.H * a.G, sl = (int)(blockIdx.x % SL), b = (int)(blockIdx.x / SL / Hq);
    const int hq = (int)(blockIdx.x / SL % Hq), h = hq / a.G, gi = hq % a.G;
    const int rows = pv.H * a.GC / a.HB, vh = h * a.GC + gi / COLS, row = vh / a.HB;
    const int pc = (vh % a.HB) * COLS + gi % COLS;
    const int64_t orow = (int64_t)b * Hq + hq;
    pdl_wait();
    const int2 span = a.span[(int64_t)b * rows + row];          // not looked at where the row has no tiles
    if (visible_of(pv, b).tiles == 0) {
        if (threadIdx.x < 32 && 32 * sl + lane < pv.Dh) a.out[orow * pv.Dh + 32 * sl + lane] = __float2bfloat16(0.0f);
        if (threadIdx.x == 0 && sl == 0) a.lse[orow] = -INFINITY;
        return;
    }
    if (span.x == span.y || 32 * sl >= pv.Dh) return;
    // the row's tile 0 is in the first CTA, whose part is the second of its two; the others' is their first
    const int64_t stride = (int64_t)a.HB * COLS * (DH + 2), ml = (int64_t)a.HB * COLS * DH + 2 * pc;
    float mx = kNoMax, sum = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = span.x + r; cb <= span.y; cb += U * R) {
        float2 v[U];
        float4 o[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = min(cb + i * R, span.y);
            const float *p = a.part + (2 * (int64_t)c + (c == span.x ? 1 : 0)) * stride;
            v[i] = *reinterpret_cast<const float2 *>(p + ml);
            o[i] = *reinterpret_cast<const float4 *>(p + (int64_t)pc * DH + 32 * sl + 4 * q4);
        }
        float nm = mx;
#pragma unroll
        for (int i = 0; i < U; ++i) nm = fmaxf(nm, cb + i * R <= span.y ? v[i].x : kNoMax);
        const float al = exp2_fast(mx - nm);
        mx = nm;
        sum *= al;
        acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (cb + i * R > span.y) break;
            const float be = exp2_fast(v[i].x - nm);
            sum = fmaf(v[i].y, be, sum);
            acc.x = fmaf(o[i].x, be, acc.x); acc.y = fmaf(o[i].y, be, acc.y);
            acc.z = fmaf(o[i].z, be, acc.z); acc.w = fmaf(o[i].w, be, acc.w);
        }
    }
    s_acc[r][q4] = acc;
    if (q4 == 0) {
        s_max[r] = mx;
        s_sum[r] = sum;
    }
    __syncthreads();
    if (warp > 0) return;
    mx = s_max[0];
#pragma unroll
    for (int w = 1; w < R; ++w) mx = fmaxf(mx, s_max[w]);
    sum = 0.0f;
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < R; ++w) {
        const float al = exp2_fast(s_max[w] - mx);
        sum = fmaf(s_sum[w], al, sum);
        x = fmaf(reinterpret_cast<const float *>(s_acc[w])[lane], al, x);
    }
    if (32 * sl + lane < pv.Dh) a.out[orow * pv.Dh + 32 * sl + lane] = __float2bfloat16(sum == 0.0f ? 0.0f : x / sum);
    if (lane == 0 && sl == 0) a.lse[orow] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// mass of the visible positions from the logits and the joined lse.  One
// thread per (sequence, KV head, visible index); the heads of the group in order.
template <int COLS>
__global__ void __launch_bounds__(256)
k_decode_mass(const PagedView pv, const DecodeArgs a) {
    const int b = (int)blockIdx.z, h = (int)blockIdx.y, VH = pv.H * a.GC;
    pdl_wait();
    const Visible vis = visible_of(pv, b);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)vis.tiles * kTile;
         i += (int64_t)gridDim.x * 256) {
        const int j = vis.position((int)(i / kTile)) + (int)(i % kTile);
        if (!vis.sees(j) || j >= a.ld_mass || pv.slot(b, j) < 0) continue;
        float sum = 0.0f;
        for (int c = 0; c < a.GC; ++c) {
            const float *lp = a.logits + (((int64_t)b * VH + h * a.GC + c) * a.vis_max + i) * COLS;
            const float *ls = a.lse + (int64_t)b * pv.H * a.G + h * a.G + c * COLS;
            for (int e = 0; e < COLS && c * COLS + e < a.G; ++e) sum += exp2_fast(lp[e] - ls[e] * kLog2e);
        }
        float *o = a.mass + ((int64_t)b * pv.H + h) * a.ld_mass + j;
        *o = a.decay == 0.0f ? sum : a.decay * *o + sum;
    }
}

}  // namespace

using namespace fp8q_host;

namespace {

struct DecodePlan {
    int DH, NT, G, GC, HB, ctas, sms;
    size_t part_bytes, span_bytes, lse_bytes, logit_bytes;
    size_t total() const { return part_bytes + span_bytes + lse_bytes + logit_bytes; }
};

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Groups of up to 8 query heads take one column block, larger ones two (16
// heads per pass over K and V; a head size of 256 has registers for one).
// 16 x 8192 tokens, 8 KV heads of 128, 9, 16 and 32 query heads each: 85, 93 and
// 153 us; with one block and more passes 89, 97 and 167 (heads of 64: 69 and 75),
// when that was chosen; 1 - 2 % more today.
// A CTA's warps share out the largest power of two of heads that divides their
// number, so that no warp is idle; the warps left per head take turns at its
// tiles.
// max_context: positions of a sequence that the call may look at.
DecodePlan decode_plan(int64_t B, int64_t Hq, int64_t H, int64_t Dh, int64_t max_context, bool weights, int sms) {
    DecodePlan p;
    p.G = (int)(Hq / H);
    p.DH = Dh <= 64 ? 64 : Dh <= 128 ? 128 : 256;
    p.NT = p.G > 8 && p.DH <= 128 ? 2 : 1;
    p.GC = (p.G + 8 * p.NT - 1) / (8 * p.NT);
    const int64_t VH = H * p.GC;
    const int warps = p.DH <= 128 && p.NT == 1 ? 16 : 8;      // Cfg::WARPS
    for (p.HB = warps; VH % p.HB; p.HB /= 2) {}
    p.sms = p.ctas = sms;
    p.part_bytes = round256((size_t)p.ctas * 2 * p.HB * 8 * p.NT * (p.DH + 2) * 4);
    p.span_bytes = round256((size_t)(B * (VH / p.HB)) * 8);
    p.lse_bytes = round256((size_t)(B * Hq) * 4);
    const size_t tiles = (size_t)((max_context + kTile - 1) / kTile);
    p.logit_bytes = weights ? round256((size_t)(B * VH) * tiles * kTile * 8 * p.NT * 4) : 0;
    return p;
}

// Dynamic shared memory above 48 KiB is granted per kernel and device, once.
template <typename K>
cudaError_t grant_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);     // check_device() admits ordinals below 64
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// 3-D map over codes [slots, H, Dh]: boxes of `rows` slots of one head, 64 or
// 128 bytes wide (a head size in between reads zeros behind its end).
bool make_map_paged(CUtensorMap *map, const void *codes, const PagedView &pv, int DH, int rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)pv.Dh, (cuuint64_t)pv.H, (cuuint64_t)pv.bs.d * (cuuint64_t)pv.num_blocks};
    cuuint64_t strides[2] = {(cuuint64_t)pv.Dh, (cuuint64_t)pv.Dh * (cuuint64_t)pv.H};
    cuuint32_t box[3] = {DH == 64 ? 64u : 128u, 1, (cuuint32_t)rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(codes), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, DH == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int DH, int NT, bool TMA>
cudaError_t launch_main(const PagedView &pv, const DecodeArgs &a, const DecodePlan &p, cudaStream_t s) {
    using C = Cfg<DH, NT>;
    static std::atomic<uint64_t> granted{0};
    cudaError_t e = grant_smem(k_decode<FMT, DH, NT, TMA>, C::SMEM, granted);
    if (e != cudaSuccess) return e;
    CUtensorMap tk = {}, tv = {};
    if (TMA && (!make_map_paged(&tk, pv.kc, pv, DH, a.box) || !make_map_paged(&tv, pv.vc, pv, DH, a.box)))
        return cudaErrorInvalidValue;
    return pdl_launch(k_decode<FMT, DH, NT, TMA>, dim3(p.ctas), dim3(C::WARPS * 32), C::SMEM, s, tk, tv, pv, a);
}

template <int FMT, int DH, int NT>
cudaError_t launch_decode(const PagedView &pv, const DecodeArgs &a, const DecodePlan &p, cudaStream_t s) {
    using C = Cfg<DH, NT>;
    // pages that 8 rows do not divide, and a pool without pages, have no boxes
    cudaError_t e = pv.bs.d % 8 == 0 && pv.num_blocks > 0 ? launch_main<FMT, DH, NT, true>(pv, a, p, s)
                                                          : launch_main<FMT, DH, NT, false>(pv, a, p, s);
    if (e != cudaSuccess) return e;
    e = pdl_launch(k_decode_join<DH, C::COLS>, dim3((unsigned)(a.B * (int64_t)pv.H * a.G * (DH / 32))),
                   dim3(kJoinWarps * 32), 0, s, pv, a);
    if (e != cudaSuccess || !a.logits) return e;
    // eight CTAs per SM in all, or one per (sequence, head) where there are more of those
    const int64_t pairs = (int64_t)a.B * pv.H, want = std::max<int64_t>(1, 8 * (int64_t)p.sms / pairs);
    const unsigned steps = (unsigned)std::min<int64_t>((a.vis_max + 255) / 256, want);
    return pdl_launch(k_decode_mass<C::COLS>, dim3(std::max(steps, 1u), pv.H, a.B), dim3(256), 0, s, pv, a);
}

}  // namespace

extern "C" fp8_status fp8_paged_attention_workspace_size(int64_t B, int64_t Hq, int64_t H, int64_t Dh,
                                                         int64_t max_context, int weights, int64_t tokens,
                                                         size_t *bytes) {
    if (!bytes) return FP8_ERR_INVALID_ARG;
    if (max_context < 0 || max_context > kPagedMaxContext) return FP8_ERR_SHAPE;
    fp8_status st = attn_shape(0x7FFFFFFFFFFFll, tokens, B, Hq, H, Dh, 1, 0, 0, 0, 0);
    if (st != FP8_OK) return st;
    if (tokens > 0) return prefill_workspace(tokens, B, Hq, H, Dh, bytes);
    int sms;
    st = check_device(&sms);
    if (st != FP8_OK) return st;
    *bytes = decode_plan(B, Hq, H, Dh, max_context, weights != 0, sms).total();
    return FP8_OK;
}

extern "C" fp8_status fp8_paged_attention_decode(
    const void *q_bf16, int64_t ld_q, int64_t B, int64_t Hq, const uint8_t *k_cache, const float *k_scale,
    const uint8_t *v_cache, const float *v_scale, int64_t H, int64_t Dh, int64_t block_size, int64_t num_blocks,
    fp8_format fmt, const int32_t *block_table, const int32_t *seq_lens, int64_t max_blocks, int64_t window,
    int64_t sinks, float softmax_scale, void *out_bf16, float *lse, float *mass, int64_t ld_mass, float mass_decay,
    void *workspace, size_t workspace_bytes, void *stream) {
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return FP8_ERR_INVALID_ARG;
    fp8_status st = attn_shape(ld_q, B, B, Hq, H, Dh, block_size, num_blocks, max_blocks, window, sinks);
    if (st != FP8_OK) return st;
    if (B * Hq * (Dh <= 64 ? 2 : Dh <= 128 ? 4 : 8) > 0x7FFFFFFFll) return FP8_ERR_SHAPE;   // the join's CTAs
    if (mass && ld_mass < 0) return FP8_ERR_SHAPE;
    if (!std::isfinite(softmax_scale) || (mass && !std::isfinite(mass_decay))) return FP8_ERR_INVALID_ARG;
    if (B == 0) return FP8_OK;
    st = attn_pointers(q_bf16, ld_q, k_cache, k_scale, v_cache, v_scale, num_blocks, block_table, seq_lens, max_blocks,
                       out_bf16, workspace);
    if (st != FP8_OK) return st;
    int sms;
    st = check_device(&sms);
    if (st != FP8_OK) return st;
    const PagedView pv = make_paged_view(k_cache, k_scale, v_cache, v_scale, H, Dh, block_size, num_blocks,
                                         block_table, seq_lens, max_blocks, window, sinks);
    int64_t context = max_blocks * block_size;
    // whole tiles: at most one begun for the sinks and two for the window
    if (pv.window > 0) context = std::min<int64_t>(context, (int64_t)pv.window + pv.sinks + 3 * kTile);
    const DecodePlan p = decode_plan(B, Hq, H, Dh, context, mass != nullptr, sms);
    if (!workspace || workspace_bytes < p.total()) return FP8_ERR_INVALID_ARG;
    uint8_t *ws = (uint8_t *)workspace;
    DecodeArgs a = {};
    a.q = (const __nv_bfloat16 *)q_bf16;
    a.ld_q = ld_q;
    a.B = (int)B;
    a.G = p.G;
    a.GC = p.GC;
    a.HB = p.HB;
    a.scale = softmax_scale;
    a.box = block_size % 32 == 0 ? 32 : block_size % 16 == 0 ? 16 : 8;
    a.out = (__nv_bfloat16 *)out_bf16;
    a.part = (float *)ws;
    a.span = (int2 *)(ws + p.part_bytes);
    a.lse = lse ? lse : (float *)(ws + p.part_bytes + p.span_bytes);
    if (mass && ld_mass > 0 && context > 0) {
        a.logits = (float *)(ws + p.part_bytes + p.span_bytes + p.lse_bytes);
        a.vis_max = (context + kTile - 1) / kTile * kTile;
        a.mass = mass;
        a.ld_mass = ld_mass;
        a.decay = mass_decay;
    }
    cudaStream_t s = as_stream(stream);
    cudaError_t e;
#define FP8Q_DECODE(DH, NT) \
    e = fmt == FP8_E4M3 ? launch_decode<FP8_E4M3, DH, NT>(pv, a, p, s) : launch_decode<FP8_E5M2, DH, NT>(pv, a, p, s)
    if (p.DH == 64 && p.NT == 1) FP8Q_DECODE(64, 1);
    else if (p.DH == 64) FP8Q_DECODE(64, 2);
    else if (p.DH == 128 && p.NT == 1) FP8Q_DECODE(128, 1);
    else if (p.DH == 128) FP8Q_DECODE(128, 2);
    else FP8Q_DECODE(256, 1);
#undef FP8Q_DECODE
    return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

// This file's device error word (fp8_device_error reads it with the others').
fp8_status fp8q_decode_device_error(uint32_t *out, int clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof(v)) != cudaSuccess) return FP8_ERR_CUDA;
    *out = v;
    if (clear) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_gemm_error, &z, sizeof(z)) != cudaSuccess) return FP8_ERR_CUDA;
    }
    return FP8_OK;
}
