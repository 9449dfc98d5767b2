// paged_prefill.cu -- causal attention of several new tokens per sequence over
// the paged FP8 KV cache (a prompt, a chunk of one, a few drafted tokens).
//
// The query heads of a KV head and the new tokens form the rows of one matrix
// product: row (token, head of the group), 256 rows to a unit of work in two
// 128-row tiles, so every K and V tile that is read and converted serves 256
// rows.  Per tile of 128 positions, on tcgen05:
//   S = Q K^T   both operands fp16 in shared memory, S in TMEM;
//   softmax     a thread per row, S in its registers; P back to TMEM as fp16;
//   O += P V    P from TMEM, V from shared memory, O stays in TMEM.
// E4M3 and E5M2 codes are exact in fp16.  K's row scales multiply the columns
// of S in fp32 (in the multiply-add that subtracts the reference); V's are
// multiplied into the fp16 V (rounded to fp16 as a factor and as a product,
// 2^-11 each: in P they would cost a multiply and a shared load per weight),
// against a running power of two of the largest scale so far.  Where the scales
// of a run are too far apart for that, V is the codes and the scales multiply P,
// each row by a power of two of its own (8192 tokens: 2260 instead of 700 us).
// Q is brought to [2^14, 2^15) by a power of two of the row tile, or of each row
// where rows are more than 2^15 apart (1110 us).  The softmax reference is set to 2^7 below a
// maximum and only moves when a tile's weights sum to 2^15, so neither the
// maximum of a tile is looked for nor O rescaled but seldom, and weights are
// exact to 2^-11 down to 2^-21 of the largest in fp16.
//
// Warp roles: warp 0 issues the MMAs; warps 2 and 3 look up the tiles' slots and
// scales, warp 1 copies their codes (TMA boxes of 8 rows or more of one head where
// the page size allows it, cp.async otherwise); warpgroup 3 converts them to the
// fp16 tiles; warpgroups 1 and 2 are the softmax of the two row tiles (and load
// Q, rescale O, write results).  The tensor core alternates between the row tiles, so one
// tile's softmax runs under the other's products.
//
// Split: k_prefill_plan lists the row blocks of all sequences and deals the
// (row block, head, position tile) triples, laid end to end, to the CTAs in
// runs of equal cost.  A unit that one CTA covers is written at once; the others
// leave (O, reference, sum) in the workspace and k_prefill_join adds the parts in
// the order of the CTAs.
//
// Measured on a B200, 32 query heads over 8 KV heads of 128: 8192 tokens 700 -
// 720 us (765 - 785 TFLOP/s), tensor pipe 39 % busy, MUFU 39 %, issue slots 46 %.
// What bounds it is the chain of a row tile: softmax of 128 columns 2100 - 2600
// cycles (128 exponentials of 8 cycles each and what they wait for), P to TMEM
// 300, P V and the next S 1500 with their waits; two row tiles in turn take 4400 -
// 5000 cycles, where the tensor core needs 2048 (16 MMAs of 64 cycles for each) and
// the exponentials 2048 as well.  The softmax threads and the look-up warps spill
// (1240 bytes stored, 590 loaded in the code; 2.4 of 322 million warp instructions
// executed are loads of spilled registers).  How the code lies in the instruction
// cache, which four roles share, moves the time by 3 % either way.  A unit costs
// 13000 - 17000 cycles more, for Q and the results.  Codes by TMA instead of
// cp.async (pages that 8 does not divide): 700 against 1000 us.
//
// What a row must not see is kept out of it whatever it holds: S is masked by
// selection; V rows of slots that are no live position are written as zeros;
// and since a weight of zero does not hide a NaN or infinity in V, such values
// in tiles that only part of the rows see are written as zeros as well, and
// added to the rows that do see them at the end.  A V scale or a query row of
// others decides at most which of the two ways above is taken.
#include <algorithm>
#include <atomic>

#include "paged_attn.cuh"

using namespace fp8q;

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.0e38f;    // the reference before the first logit
constexpr float kBelow = 7.0f;        // log2 of how far under the maximum a reference is set
constexpr float kMaxSum = 32768.0f;   // a row's weights of one tile sum to less, so that none passes 2^15

struct PrefillArgs {
    const __nv_bfloat16 *q;
    int64_t ld_q;
    const int64_t *q_off;
    int64_t T;
    int B, G, ctas, box;
    FastDiv gdiv;             // by G
    int64_t max_blocks;       // row blocks that the workspace has room for
    float scale;
    __nv_bfloat16 *out;
    float *lse;               // or nullptr
    float *part;              // two parts per CTA
    int4 *split;              // per CTA: {row block, head, last CTA} of the unit that it began and others go on with
    int64_t *hdr;             // {cost in all}
    int64_t *first_block;     // [B] row blocks before each sequence
    int2 *block;              // {sequence, row block of it}
    longlong2 *start;         // per CTA: {row block, cost before it}
};

template <int DH>
struct Pre {
    static constexpr int MT = DH <= 128 ? 2 : 1;          // 128-row tiles of a unit
    static constexpr int KT = DH <= 128 ? 128 : 64;       // positions per tile
    static constexpr int ROWS = 128 * MT;
    static constexpr int QB = 128 * DH * 2, KVB = KT * DH * 2;   // bytes of a Q tile, of a K or V tile in fp16
    static constexpr int RAW = KT * DH;                   // and in codes
    static constexpr int RING = 3;                        // buffers of each kind: K, V, K, V, ... in turn
    static constexpr int META = 8;                        // tiles whose scales and masks are kept
    static constexpr int OFF_KV = MT * QB, OFF_RAW = OFF_KV + RING * KVB, OFF_M = OFF_RAW + RING * RAW;
    static constexpr int M_DK = 0, M_DV = KT * 4, M_SLOT = KT * 8, M_LIVE = KT * 12, M_MAX = M_LIVE + 16,
                         M_MIN = M_MAX + 4, M_EXP = M_MAX + 8, M_BYTES = M_MAX + 16;
    static constexpr int OFF_BAR = OFF_M + META * M_BYTES;
    static constexpr int NBARS = 4 * RING + 4 * MT + 1 + META;
    static constexpr size_t SMEM = 1024 + OFF_BAR + NBARS * 8;
    static constexpr int S_COL = KT, O_COL = 256;         // TMEM: S of tile i at i * S_COL, O at O_COL + i * DH
    static constexpr int VC_E4M3 = 6, VC_E5M2 = -1;       // code * scale * 2^(VC - exponent of the largest) < 2^16
    // V holds its scales while the exponents of a run's stay this close together.  E4M3: the factor is then 2^(6 - 11)
    // or more and its product with the smallest code 2^-14, fp16's smallest normal.  E5M2 (codes down to 2^-16): the
    // product is off by 2^-25 at most, 2^-16 of its own scale.  A weight below 2^-14 is off by 2^-25 too, which large
    // scales must not make count.
    static constexpr int SPREAD_E4M3 = 11, SPREAD_E5M2 = 8;
};
constexpr int kNoScale = -1000;       // exponent of V's scales, and of O's unit, before the first scale: O is zero
constexpr int kWide = 0x40000000;     // in place of a tile's unit: the scales multiply the weights instead

constexpr int kThreads = 512;
// registers per thread: launch pool 128 * 512; MMA warpgroup, softmax, converter
constexpr int kRegsLaunch = 128, kRegsMma = 56, kRegsSoft = 176, kRegsConv = 104;
static_assert(128 * kRegsMma + 256 * kRegsSoft + 128 * kRegsConv <= kThreads * kRegsLaunch, "register split");

// ------------------------------------------------------------- the units --
// Rows [rho0, rho1) of sequence b (row = token * G + head of the group) and
// the position tiles that some row sees: those of the first positions that
// stay visible, then the window's.
struct Unit {
    int64_t t0;                       // q row of the sequence's first token
    int n, count, rho0, rho1, pmin, pmax, first_tile, sink_tiles, tiles;
};
template <int ROWS, int KT>
__device__ __forceinline__ Unit unit_of(const PagedView &pv, const PrefillArgs &a, int b, int mb) {
    Unit u;
    const int64_t o0 = max((int64_t)0, min(a.T, a.q_off[b])), o1 = max(o0, min(a.T, a.q_off[b + 1]));
    u.t0 = o0;
    u.count = (int)(o1 - o0);
    u.n = pv.length(b);
    u.rho0 = mb * ROWS;
    u.rho1 = min(u.rho0 + ROWS, u.count * a.G);
    const int p0 = u.n - u.count;
    u.pmin = p0 + (int)a.gdiv.div((uint32_t)u.rho0);
    u.pmax = p0 + (int)a.gdiv.div((uint32_t)(u.rho1 - 1));
    if (u.pmax < 0) {                 // no row sees anything: one tile, all masked
        u.first_tile = u.sink_tiles = 0;
        u.tiles = 1;
        return u;
    }
    u.first_tile = pv.window_begin(max(u.pmin, 0)) / KT;
    u.sink_tiles = min((min(pv.sinks, u.pmax + 1) + KT - 1) / KT, u.first_tile);
    u.tiles = u.sink_tiles + u.pmax / KT - u.first_tile + 1;
    return u;
}
template <int KT>
__device__ __forceinline__ int tile_pos(const Unit &u, int t) {
    return (t < u.sink_tiles ? t : u.first_tile + t - u.sink_tiles) * KT;
}
// every row sees every position of the tile at j0 (as far as the pages are there)
template <int KT>
__device__ __forceinline__ bool tile_full(const PagedView &pv, const Unit &u, int j0) {
    return u.pmin >= 0 && j0 + KT - 1 <= u.pmin && (j0 >= pv.window_begin(u.pmax) || j0 + KT <= pv.sinks);
}

// A unit costs its tiles and this many more, for Q and the results.  Laid end to
// end in cost, a unit's first kUnitCost places hold no tile.  At 3, 4, 5, 6, 8:
//   8192 tokens, 8 x 4 heads of 128     743   697  704  711  726 us
//   2 x 5000 tokens, the same           638   596  594  599  618
//   2048 tokens, the same                96    98  100  100  105
//   16000 tokens, 8 heads of 64         579   583  586  589  596
//   8192 tokens, 4 x 4 heads of 256    1143  1024  930  889  901
// and a few tokens over a long cache, or chunks with a window, within 4 %.
constexpr int kUnitCost = 5;

constexpr int kPlanThreads = 1024;
__device__ int64_t plan_scan(int64_t v, int64_t *buf, int64_t *total) {   // exclusive, block-wide
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    int64_t w = buf[lane], s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xFFFFFFFFu, s, 31);
    return __shfl_sync(0xFFFFFFFFu, s - w, warp) + x - v;
}

// One CTA: the row blocks of every sequence, their tiles, and where each CTA of
// the attention kernel starts.
template <int ROWS, int KT>
__global__ void __launch_bounds__(kPlanThreads)
k_prefill_plan(const PagedView pv, const PrefillArgs a) {
    __shared__ int64_t buf[32], place[kPlanThreads];
    pdl_wait();
    pdl_trigger();
    int64_t base = 0, all;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int64_t blocks = 0;
        if (b < a.B) {
            const int64_t o0 = max((int64_t)0, min(a.T, a.q_off[b])), o1 = max(o0, min(a.T, a.q_off[b + 1]));
            blocks = ((o1 - o0) * a.G + ROWS - 1) / ROWS;
        }
        const int64_t pre = base + plan_scan(blocks, buf, &all);
        if (b < a.B) a.first_block[b] = pre;
        base += all;
    }
    const int64_t nb = min(base, a.max_blocks);   // more only if q_offsets decrease somewhere
    __syncthreads();                  // first_block is read by the whole CTA
    auto tiles_at = [&](int64_t i, int2 *who) -> int64_t {
        if (i >= nb) return 0;
        int lo = 0, hi = a.B - 1;     // the last sequence whose blocks begin at or before i
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (a.first_block[mid] <= i) lo = mid; else hi = mid - 1;
        }
        *who = make_int2(lo, (int)(i - a.first_block[lo]));
        return (int64_t)(unit_of<ROWS, KT>(pv, a, lo, who->y).tiles + kUnitCost) * pv.H;
    };
    int64_t sum = 0, total;
    int2 who = make_int2(0, 0);
    int64_t mine = 0;
    for (int64_t i = threadIdx.x; i < nb; i += kPlanThreads) sum += mine = tiles_at(i, &who);
    plan_scan(sum, buf, &total);
    if (threadIdx.x == 0) a.hdr[0] = total;
    const int64_t n = min((int64_t)a.ctas, total);
    base = 0;
    for (int64_t i0 = 0; i0 < nb; i0 += kPlanThreads) {
        const int64_t i = i0 + threadIdx.x;
        if (nb > kPlanThreads || i >= nb) mine = tiles_at(i, &who);
        const int64_t pre = base + plan_scan(mine, buf, &all);
        if (i < nb) a.block[i] = who;
        // a thread per CTA: its first place, total * c / n, and the row block that holds it, if it is one of these
        place[threadIdx.x] = pre;
        __syncthreads();
        const int blocks = (int)min((int64_t)kPlanThreads, nb - i0);
        for (int64_t c = threadIdx.x; c < n; c += kPlanThreads) {
            const int64_t at = total * c / n;
            if (at < base || at >= base + all) continue;
            int lo = 0, hi = blocks - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (place[mid] <= at) lo = mid; else hi = mid - 1;
            }
            a.start[c] = make_longlong2(i0 + lo, place[lo]);
        }
        base += all;
        __syncthreads();              // the next blocks' places go there
    }
}

// The runs of one CTA: consecutive tiles of one unit.
template <int ROWS, int KT>
struct Runs {
    const PagedView &pv;
    const PrefillArgs &a;
    int64_t at, end, total, ncta;     // places of the CTA; in all; CTAs with any
    int2 who;
    Unit u;
    int bi, h, v, tile, len, span;    // row block, head, place in the unit; tiles [tile, tile + len) of it; places

    __device__ __forceinline__ Runs(const PagedView &pv_, const PrefillArgs &a_) : pv(pv_), a(a_) {
        total = a.hdr[0];
        ncta = min((int64_t)a.ctas, total);
        at = end = 0;
        len = span = 0;
        if ((int64_t)blockIdx.x >= ncta) return;
        at = total * blockIdx.x / ncta;
        end = total * (blockIdx.x + 1) / ncta;
        const longlong2 s = a.start[blockIdx.x];
        bi = (int)s.x;
        who = a.block[bi];
        u = unit_of<ROWS, KT>(pv, a, who.x, who.y);
        const int places = u.tiles + kUnitCost;
        h = (int)((at - s.y) / places);
        v = (int)((at - s.y) % places);
        settle();
    }
    __device__ __forceinline__ void cut() {
        span = (int)min((int64_t)(u.tiles + kUnitCost - v), end - at);
        tile = max(0, v - kUnitCost);
        len = max(0, v + span - kUnitCost) - tile;
    }
    __device__ __forceinline__ void step() {
        at += span;
        v = 0;
        if (at < end && ++h == pv.H) {
            h = 0;
            who = a.block[++bi];
            u = unit_of<ROWS, KT>(pv, a, who.x, who.y);
        }
    }
    __device__ __forceinline__ void settle() {          // to a run with tiles
        while (at < end) {
            cut();
            if (len > 0) return;
            step();
        }
        len = 0;
    }
    __device__ __forceinline__ void next() {
        step();
        settle();
    }
    __device__ __forceinline__ bool live() const { return len > 0; }
    __device__ __forceinline__ bool whole() const { return tile == 0 && len == u.tiles; }
    // CTA that holds the unit's last place: the largest c with total * c / ncta <= place
    __device__ __forceinline__ int last_cta() const {
        const int64_t place = at - v + u.tiles + kUnitCost - 1;
        return (int)((place * ncta + ncta - 1) / total);
    }
};

// --------------------------------------------------------------- PTX glue --
// Bounded wait, as wait_bar(), for warps that share their scheduler with others that work: a try sleeps up to
// 20 us unless the phase completes, and nobody waits again after a wait that ran out.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, uint32_t code) {
    if (try_wait_long(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!try_wait_long(bar, parity)) {
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kTimeoutNs) {
            atomicOr(&g_gemm_error, code);
            *abort_flag = 1u;
            return false;
        }
    }
    return true;
}
// Bounded wait until the count at addr has reached n (n <= 0: at once).
__device__ __forceinline__ void wait_progress(uint32_t addr, uint32_t n, volatile uint32_t *abort_flag) {
    uint64_t t0 = 0;
    while (true) {
        uint32_t v;
        asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
        if ((int)(v - n) >= 0 || *abort_flag) return;
        if (t0 == 0) t0 = globaltimer();
        else if (globaltimer() - t0 > kTimeoutNs) {
            atomicOr(&g_gemm_error, kErrProducer);
            *abort_flag = 1u;
            return;
        }
        __nanosleep(200);
    }
}
__device__ __forceinline__ void arrive_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The MMA warp runs as a whole and one elected lane (`leader`) issues: with the
// descriptors in a branch of lane 0 alone an MMA took 270 cycles to issue, four
// times as long as it runs.  A descriptor is its low word (the address moves)
// and a constant high word.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t l;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(l));
    return l;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t acc,
                                       uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
// A predicate here too: in a branch of its own the leader would fall behind lanes that already wait for what it is
// to commit.
__device__ __forceinline__ void st_release_one(uint32_t addr, uint32_t v, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q st.release.cta.shared::cta.u32 [%0], %1;\n\t}" ::"r"(addr),
        "r"(v), "r"(leader)
        : "memory");
}
// 32 lanes x 16 columns from registers; tmem_st_wait() before they are read
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t addr, uint32_t *o) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]), "=r"(o[8]),
          "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld8_async(uint32_t addr, uint32_t *o) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// waits for the loads in flight; the registers of this array cannot be read above it
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pack_ff(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// bytes of four codes that are NaN or (E5M2) infinite: 0x80 in each such byte
template <int FMT>
__device__ __forceinline__ uint32_t nonfinite4(uint32_t c) {
    return ((c & 0x7F7F7F7Fu) + (FMT == FP8_E4M3 ? 0x01010101u : 0x04040404u)) & 0x80808080u;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void st_shared_u32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Low and high words of the shared-memory descriptors, 128-byte swizzle.  K-major
// (Q, K): rows of 64 elements, 8 rows 1 KiB apart.  MN-major (V: a row per
// position, 64 head elements of 128 bytes per block): 8 positions 1 KiB apart,
// blocks `block` bytes apart.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t block) {
    return ((addr >> 4) & 0x3FFFu) | (block ? (block >> 4) << 16 : 1u << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride; sm_100 version; 128-byte swizzle
// kind::f16: fp32 sums, A and B fp16
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// bits below x of a 32-bit word
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u; }

// ----------------------------------------------------------------- kernel --
// TMA: boxes of a.box rows, which divides the page size; otherwise cp.async.
template <int FMT, int DH, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
k_prefill(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedView pv,
          const PrefillArgs a) {
    using P = Pre<DH>;
    constexpr int MT = P::MT, KT = P::KT, ROWS = P::ROWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // s_poison: something was taken out of V (for good: later results of this CTA look again for nothing)
    __shared__ uint32_t s_tmem, s_abort, s_poison;
    __shared__ uint2 s_q[MT][4];      // largest and smallest row exponent of Q, per softmax warp
    __shared__ uint32_t s_progress;   // tiles whose weights all softmax warps have handed over
    __shared__ float4 s_factor[MT][2][KT / 4];   // column factors of a row tile's softmax, two tiles
    __shared__ float s_ones[KT];      // in their place where the products have been multiplied by them
    volatile uint32_t *abort_flag = &s_abort;
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    const uint32_t bar0 = sb + P::OFF_BAR;
    constexpr int RING = P::RING;
    auto rfull = [&](uint32_t i) { return bar0 + 8 * (i % RING); };              // codes of unit i = 2 tile + (V ? 1 : 0)
    auto rempty = [&](uint32_t i) { return bar0 + 8 * (RING + i % RING); };
    auto ffull = [&](uint32_t i) { return bar0 + 8 * (2 * RING + i % RING); };   // the same in fp16
    auto fempty = [&](uint32_t i) { return bar0 + 8 * (3 * RING + i % RING); };
    auto phase = [](uint32_t i) { return (i / RING) & 1u; };
    auto qfull = [&](int i) { return bar0 + 8 * (4 * RING + i); };
    auto sfull = [&](int i) { return bar0 + 8 * (4 * RING + MT + i); };
    auto pfull = [&](int i) { return bar0 + 8 * (4 * RING + 2 * MT + i); };
    auto pvdone = [&](int i) { return bar0 + 8 * (4 * RING + 3 * MT + i); };
    const uint32_t drain = bar0 + 8 * (4 * RING + 4 * MT);
    auto mfull = [&](uint32_t k) { return bar0 + 8 * (4 * RING + 4 * MT + 1 + k % P::META); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(rfull(i), TMA ? 1 : 32);
            mbar_init(rempty(i), 128);
            mbar_init(ffull(i), 128);
            mbar_init(fempty(i), 1);
        }
        for (int i = 0; i < MT; ++i) {
            mbar_init(qfull(i), 128);
            mbar_init(pfull(i), 128);
            mbar_init(sfull(i), 1);
            mbar_init(pvdone(i), 1);
        }
        for (int i = 0; i < P::META; ++i) mbar_init(mfull(i), 32);
        mbar_init(drain, 1);
        s_abort = s_poison = s_progress = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < KT) s_ones[threadIdx.x] = 1.0f;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();

    Runs<ROWS, KT> run(pv, a);
    if (threadIdx.x == 128) a.split[blockIdx.x] = make_int4(-1, 0, 0, 0);   // the thread that writes the other value

    if (wg == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
        if (warp == 0) {
            const uint32_t leader = elect_one();
            // ------------------------------------------------------ MMAs --
            constexpr uint32_t id_s = idesc_f16(128, KT, false), id_o = idesc_f16(128, DH, true);
            uint32_t kc = 0, pc[2] = {0, 0}, qc[2] = {0, 0};   // tiles so far; P tiles; runs
            bool ok = true;
            for (; ok && run.live(); run.next()) {
                const int len = run.len, tiles_m = run.u.rho1 - run.u.rho0 > 128 ? MT : 1;
                // Step k: P V of tile k, then S of tile k + 1, for each row tile.  The loops stay rolled: four roles
                // share an instruction cache.
#pragma unroll 1
                for (int k = -1; ok && k < len; ++k) {
                    const uint32_t vi = 2 * kc + 1, ki = k < 0 ? 2 * kc : 2 * kc + 2;   // V of tile k, K of tile k + 1
                    if (k >= 0) ok = wait_for(ffull(vi), phase(vi), abort_flag, kErrMma);
                    else for (int i = 0; ok && i < tiles_m; ++i) ok = wait_for(qfull(i), qc[i]++ & 1u, abort_flag, kErrMma);
#pragma unroll 1
                    for (int i = 0; ok && i < tiles_m; ++i) {
                        if (k >= 0) {
                            const uint32_t par = (i ? pc[1]++ : pc[0]++) & 1u;
                            ok = wait_for(pfull(i), par, abort_flag, kErrMma);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t vd = desc_lo(sb + P::OFF_KV + vi % RING * P::KVB, KT * 128);
#pragma unroll 2
                            for (int s = 0; s < KT / 16; ++s)
                                mma_ts(tmem + P::O_COL + i * DH, tmem + i * P::S_COL + 8 * s, vd + 128 * s, kDescHi, id_o,
                                       (k | s) ? 1u : 0u, leader);
                            commit_one(pvdone(i), leader);
                        }
                        if (k + 1 < len) {
                            if (i == 0) ok = wait_for(ffull(ki), phase(ki), abort_flag, kErrMma);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t qd = desc_lo(sb + i * P::QB, 0);
                            const uint32_t kd = desc_lo(sb + P::OFF_KV + ki % RING * P::KVB, 0);
#pragma unroll 2
                            for (int s = 0; s < DH / 16; ++s)       // 64 elements to a swizzled block
                                mma_ss(tmem + i * P::S_COL, qd + (s >> 2) * (128 * 128 >> 4) + 2 * (s & 3), kDescHi,
                                       kd + (s >> 2) * (KT * 128 >> 4) + 2 * (s & 3), kDescHi, id_s, s ? 1u : 0u, leader);
                            commit_one(sfull(i), leader);
                        }
                    }
                    if (!ok) break;
                    if (k >= 0) {
                        commit_one(fempty(vi), leader);
                        st_release_one(smem_u32(&s_progress), ++kc, leader);
                    }
                    if (k + 1 < len) commit_one(fempty(ki), leader);
                }
            }
            commit_one(drain, leader);
            wait_bar_drain(drain, 0u);
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------- codes of the tiles, K and V in turn --
            uint32_t kc = 0, issued = 0;
            bool ok = true;                   // after a wait that ran out nothing more is copied
            for (; ok && run.live(); run.next()) {
                for (int k = 0; ok && k < run.len; ++k, ++kc) {
                    ok = wait_for(mfull(kc), (kc / P::META) & 1u, abort_flag, kErrProducer);
                    const uint32_t slots = sb + P::OFF_M + (kc % P::META) * P::M_BYTES + P::M_SLOT;
                    for (uint32_t i = 2 * kc; ok && i < 2 * kc + 2; ++i) {
                        ok = wait_for(rempty(i), phase(i) ^ 1u, abort_flag, kErrProducer) && !*abort_flag;
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        issued = i + 1;
                        const uint32_t dst = sb + P::OFF_RAW + i % RING * P::RAW;
                        if constexpr (TMA) {
                            if (lane == 0) mbar_expect_tx(rfull(i), P::RAW);
                            // lane l: the box at row l * box; one without a slot starts past the last: zeros
                            const int r = lane * a.box;
                            if (r < KT) {
                                const int s = (int)ld_shared_u32(slots + 4 * r);
                                const int z = s >= 0 ? s : (int)(pv.bs.d * (uint32_t)pv.num_blocks);
                                tma_load_3d(dst + (uint32_t)r * DH, i & 1 ? &tmV : &tmK, rfull(i), 0, run.h, z);
                            }
                        } else {
                            const uint8_t *codes = (i & 1 ? pv.vc : pv.kc) + run.h * pv.Dh;
                            constexpr int CH = DH / 16;
                            for (int x = lane; x < KT * CH; x += 32) {
                                const int s = (int)ld_shared_u32(slots + 4 * (x / CH)), c = x % CH;
                                const int n = s >= 0 && 16 * c < pv.Dh ? 16 : 0;
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * x),
                                             "l"(codes + (uint64_t)(uint32_t)max(s, 0) * (uint32_t)(pv.H * pv.Dh) +
                                                 (n ? 16 * c : 0)),
                                             "r"(n)
                                             : "memory");
                            }
                            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(rfull(i)) : "memory");
                        }
                    }
                }
            }
            if constexpr (!TMA) asm volatile("cp.async.wait_all;" ::: "memory");
            // copies that the converter may not have waited for end before the CTA does
            if (TMA && *abort_flag)
                for (uint32_t i = issued > RING ? issued - RING : 0; i < issued; ++i) wait_bar_drain(rfull(i), phase(i));
            __syncwarp();
        } else {
            // ------------------------- slots, scales and masks of tiles ---
            // Warps 2 and 3 take turns, a few tiles ahead: a tile's look-up is two dependent loads, which nothing
            // behind it could hide.
            uint32_t kc = 0;
            for (; run.live(); run.next()) {
                const Unit &u = run.u;
                const int h = run.h;
                for (int k = 0; k < run.len; ++k, ++kc) {
                    if ((kc & 1) != (uint32_t)(warp & 1)) continue;
                    // Nobody reads tile kc - META any more: a count, because a parity only tells a phase from its
                    // neighbours and this warp may come much later than the phase it would wait for.
                    wait_progress(smem_u32(&s_progress), kc + 1 - P::META, abort_flag);
                    uint8_t *m = smem + P::OFF_M + (kc % P::META) * P::M_BYTES;
                    const int j0 = tile_pos<KT>(u, run.tile + k);
                    int s[KT / 32];
                    float dk[KT / 32], dv[KT / 32];
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i) {
                        const int j = j0 + 32 * i + lane;
                        s[i] = j < u.n && j <= u.pmax ? pv.slot(run.who.x, j) : -1;
                    }
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i) {
                        dk[i] = s[i] >= 0 ? pv.ks[(int64_t)s[i] * pv.H + h] : 0.0f;
                        dv[i] = s[i] >= 0 ? pv.vs[(int64_t)s[i] * pv.H + h] : 0.0f;
                    }
                    uint32_t mx = 0, mn = 0xFFFFFFFFu;        // of the finite scales; of those that are not zero
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i) {
                        reinterpret_cast<float *>(m + P::M_DK)[32 * i + lane] = k_factor(dk[i]) * fabsf(a.scale) * kLog2e;
                        reinterpret_cast<float *>(m + P::M_DV)[32 * i + lane] = dv[i];
                        reinterpret_cast<int *>(m + P::M_SLOT)[32 * i + lane] = s[i];
                        const uint32_t live = __ballot_sync(0xFFFFFFFFu, s[i] >= 0);
                        const uint32_t d = __float_as_uint(fabsf(dv[i]));
                        if (d < 0x7F800000u) {
                            mx = max(mx, d);
                            if (d) mn = min(mn, d);
                        }
                        if (lane == 0) reinterpret_cast<uint32_t *>(m + P::M_LIVE)[i] = live;
                    }
                    mx = __reduce_max_sync(0xFFFFFFFFu, mx);
                    mn = __reduce_min_sync(0xFFFFFFFFu, mn);
                    if (lane == 0) *reinterpret_cast<uint2 *>(m + P::M_MAX) = make_uint2(mx, mn);
                    arrive_release(mfull(kc));
                }
            }
        }
        __syncwarp();
    } else if (wg == 3) {
        // ------------------------------------------- K and V converter ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        constexpr int CH = DH / 16, RPI = 32 / CH, ITS = KT / (4 * RPI);   // 16-code chunks of a row; rows per load
        const int tid = threadIdx.x - 384, c = lane % CH, r0 = (tid >> 5) * RPI + lane / CH;
        const int swap = (c >> 2) & 1;        // half the chunks are stored high half first: no bank conflicts
        uint32_t kc = 0;
        int ex = kNoScale;                    // exponent of the largest V scale of the run so far
        uint32_t least = 0xFFFFFFFFu;         // and the smallest of them
        bool wide = false;                    // from the first tile on that has them too far apart: V is the codes
        constexpr int VC = FMT == FP8_E4M3 ? P::VC_E4M3 : P::VC_E5M2;
        constexpr int SPREAD = FMT == FP8_E4M3 ? P::SPREAD_E4M3 : P::SPREAD_E5M2;
        auto meta = [&](uint32_t k) -> uint32_t { return sb + P::OFF_M + (k % P::META) * P::M_BYTES; };
        // waits for the slots of the k-th tile; the exponent its V is held against
        auto look_up = [&](uint32_t k, bool fresh) {
            wait_for(mfull(k), (k / P::META) & 1u, abort_flag, kErrProducer);
            const uint32_t mx = ld_shared_u32(meta(k) + P::M_MAX);
            if (fresh) {
                ex = kNoScale;
                least = 0xFFFFFFFFu;
                wide = false;
            }
            if (mx) ex = max(ex, max((int)(mx >> 23) - 127, -120));
            least = min(least, ld_shared_u32(meta(k) + P::M_MIN));
            wide |= (int)(least >> 23) - 127 < ex - SPREAD || ex > 125;   // 2^(VC - ex) is a float for -120 .. 125
            if (tid == 0) st_shared_u32(meta(k) + P::M_EXP, (uint32_t)(wide ? kWide : ex > kNoScale ? ex - VC : ex));
        };
        auto put = [&](uint32_t base, int row, const uint32_t (&x)[8]) {
            const uint32_t at_row = base + (c >> 2) * (KT * 128) + row * 128, ch = (c & 3) * 2;
            st_shared16(at_row + (((ch + swap) ^ (row & 7)) << 4), x[0], x[1], x[2], x[3]);
            st_shared16(at_row + (((ch + 1 - swap) ^ (row & 7)) << 4), x[4], x[5], x[6], x[7]);
        };
        // K and V by the same code (K times 1): it is half as long, and four roles share an instruction cache
        for (; run.live(); run.next()) {
            for (int k = 0; k < run.len; ++k, ++kc) {
                look_up(kc, k == 0);
                const float fp = wide ? 1.0f : ex > kNoScale ? pow2i(VC - ex) : 0.0f;
                const uint32_t dv = meta(kc) + P::M_DV + 4 * r0;
                uint32_t all = 0xFFFFFFFFu;
#pragma unroll
                for (int e = 0; e < KT / 32; ++e) all &= ld_shared_u32(meta(kc) + P::M_LIVE + 4 * e);
                // what is taken out of V here is what the results add again: tiles that some rows do not see, whether or
                // not pages are missing
                const bool dead = all != 0xFFFFFFFFu, part = !tile_full<KT>(pv, run.u, tile_pos<KT>(run.u, run.tile + k));
#pragma unroll 1
                for (uint32_t i = 2 * kc; i < 2 * kc + 2; ++i) {
                    const bool is_v = i & 1;
                    wait_for(rfull(i), phase(i), abort_flag, kErrProducer);
                    const uint32_t src = sb + P::OFF_RAW + i % RING * P::RAW + r0 * DH + 16 * c;
                    const uint32_t dst = sb + P::OFF_KV + i % RING * P::KVB;
                    wait_for(fempty(i), phase(i) ^ 1u, abort_flag, kErrProducer);
#pragma unroll 1
                    for (int e0 = 0; e0 < ITS; e0 += 4) {         // four rows' loads before their conversion
                        uint4 q[4];
                        float f[4] = {1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 w = ld_shared_f4(src + (e0 + e) * 4 * RPI * DH);
                            q[e] = make_uint4(__float_as_uint(swap ? w.z : w.x), __float_as_uint(swap ? w.w : w.y),
                                              __float_as_uint(swap ? w.x : w.z), __float_as_uint(swap ? w.y : w.w));
                        }
                        if (is_v) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[e] = __uint_as_float(ld_shared_u32(dv + (e0 + e) * 16 * RPI)) * fp;
                            if (dead || part) {
                                // slots that are no live position are zeros, and what only some rows see must be finite
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int r = (e0 + e) * 4 * RPI + r0;
                                    const bool live =
                                        (ld_shared_u32(meta(kc) + P::M_LIVE + 4 * (r >> 5)) >> (r & 31)) & 1u;
                                    if (!live) q[e] = make_uint4(0, 0, 0, 0);
                                    if (!part) continue;
                                    const uint32_t nf = nonfinite4<FMT>(q[e].x) | nonfinite4<FMT>(q[e].y) |
                                                        nonfinite4<FMT>(q[e].z) | nonfinite4<FMT>(q[e].w);
                                    if (nf || !(fabsf(f[e]) < INFINITY)) {
                                        s_poison = 1u;
                                        auto clean = [](uint32_t x) { return x & ~((nonfinite4<FMT>(x) >> 7) * 0xFFu); };
                                        q[e] = make_uint4(clean(q[e].x), clean(q[e].y), clean(q[e].z), clean(q[e].w));
                                        if (!(fabsf(f[e]) < INFINITY)) f[e] = 0.0f;
                                    }
                                }
                            }
                            if (wide) f[0] = f[1] = f[2] = f[3] = 1.0f;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[8];
                            to_f16x4<FMT>(q[e].x, x[0], x[1]);
                            to_f16x4<FMT>(q[e].y, x[2], x[3]);
                            to_f16x4<FMT>(q[e].z, x[4], x[5]);
                            to_f16x4<FMT>(q[e].w, x[6], x[7]);
                            const uint32_t f2 = pack_f16x2(f[e], f[e]);
#pragma unroll
                            for (int y = 0; y < 8; ++y) x[y] = mul_f16x2(x[y], f2);
                            put(dst, (e0 + e) * 4 * RPI + r0, x);
                        }
                    }
                    arrive_release(rempty(i));
                    fence_async();
                    arrive_release(ffull(i));
                }
            }
        }
    } else if (wg - 1 < MT) {
        // --------------------------------------------- softmax, results ---
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        const int mi = wg - 1, row = threadIdx.x - 128 * wg;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + mi * P::S_COL, to = tmem + lane_base + P::O_COL + mi * DH;
        auto wg_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(2 + mi) : "memory"); };
        auto wg_any = [&](bool x) {           // a barrier too
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(2 + mi), "r"((uint32_t)x) : "memory");
            return r != 0;
        };
        // S times f(column), first x, then y; rare, so eight columns of code
        auto scale_s = [&](auto f) {
#pragma unroll 1
            for (int c = 0; c < KT; c += 8) {
                uint32_t x[8];
                tmem_ld8_async(ts + c, x);
                tmem_ld_wait(x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 by = f(c + i);
                    x[i] = __float_as_uint(__uint_as_float(x[i]) * by.x * by.y);
                }
                tmem_st4(ts + c, x[0], x[1], x[2], x[3]);
                tmem_st4(ts + c + 4, x[4], x[5], x[6], x[7]);
            }
            tmem_st_wait();
        };
        uint32_t kc = 0, sc = 0;              // tiles of the CTA; S tiles of this row tile
        // the rows of this row tile in the run; Q as fp16
        int p = -1, wb = 0, qs = 0;           // qs: exponent of the row's Q less the tile's, where the warp's are `apart`
        bool apart = false;
        int64_t orow = 0;
        bool valid = false;
        float qf = 0.0f;
        auto mine = [&] { return mi == 0 || run.u.rho1 - run.u.rho0 > 128; };
        auto find = [&] {                     // on to a run of this row tile
            while (run.live() && !mine()) {
                kc += run.len;
                run.next();
            }
        };
        auto load_q = [&] {
            const Unit &u = run.u;
            const int rho = u.rho0 + mi * 128 + row, tok = (int)a.gdiv.div((uint32_t)rho), g = rho - tok * a.G;
            valid = rho < u.rho1;
            p = valid ? u.n - u.count + tok : -1;
            wb = p >= 0 ? pv.window_begin(p) : 0;
            orow = (u.t0 + tok) * (int64_t)pv.H * a.G + (int64_t)run.h * a.G + g;
            // A warp copies its 32 rows as they are, whole rows at a time; then each thread scales its own row in place,
            // in short loops, since code that runs once per unit comes from far away.  One power of two for the tile's
            // 128 rows: an element loses something only below 2^-31 of the tile's largest, so a row 2^-15 of it keeps
            // all down to 2^-16 of its own largest, and what it loses below stays under 2^-24 of that.  Rows further
            // apart than 2^15 get a power of two each, which S is then multiplied back by.
            constexpr int QC = DH / 8, QR = 32 / QC, QN = 32 / QR;    // 16-byte chunks of a row; rows per copy; copies
            const int qc = lane % QC, r0 = (warp & 3) * 32 + lane / QC;
            auto at_row = [&](int i) -> uint32_t {
                const int r = r0 + i * QR;
                return sb + mi * P::QB + (qc >> 3) * (128 * 128) + r * 128 + (((qc & 7) ^ (r & 7)) << 4);
            };
            const __nv_bfloat16 *qp = a.q + u.t0 * a.ld_q + (int64_t)run.h * a.G * pv.Dh + 8 * qc;
#pragma unroll 2
            for (int i = 0; i < QN; ++i) {
                const int rh = u.rho0 + mi * 128 + r0 + i * QR;
                const bool there = rh < u.rho1 && 8 * qc < pv.Dh;
                const int tk = (int)a.gdiv.div((uint32_t)rh), gg = rh - tk * a.G;
                const __nv_bfloat16 *src = there ? qp + tk * a.ld_q + gg * pv.Dh : a.q;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at_row(i)), "l"(src),
                             "r"(there ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            auto own = [&](int i) -> uint32_t { return sb + mi * P::QB + (i >> 3) * (128 * 128) + row * 128 + (((i & 7) ^ (row & 7)) << 4); };
            auto ld = [&](int i) -> uint4 {
                const float4 w = ld_shared_f4(own(i));
                return make_uint4(__float_as_uint(w.x), __float_as_uint(w.y), __float_as_uint(w.z), __float_as_uint(w.w));
            };
            uint32_t mx = 0;
#pragma unroll 4
            for (int i = 0; i < QC; ++i) mx = amax_fast8(mx, ld(i));
            mx = amax_fast_final(mx);
            if (mx == 0xFFFFFFFFu) {          // a NaN or infinity: the finite elements' maximum
                mx = 0;
                uint32_t bad = 0;
#pragma unroll 1
                for (int i = 0; i < QC; ++i) mx = amax_exact8(mx, ld(i), bad);
            }
            const uint32_t er = max(mx >> 7, 14u);               // exponent + 127; a row of zeros takes any
            const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, er), lo = __reduce_min_sync(0xFFFFFFFFu, mx ? er : 255u);
            if (lane == 0) s_q[mi][warp & 3] = make_uint2(hi, lo);
            wg_sync();
            const uint2 e0 = s_q[mi][0], e1 = s_q[mi][1], e2 = s_q[mi][2], e3 = s_q[mi][3];
            const int top = (int)max(max(e0.x, e1.x), max(e2.x, e3.x)), least = (int)min(min(e0.y, e1.y), min(e2.y, e3.y));
            apart = least < top - 15;
            qs = apart && mx ? (int)er - top : 0;
            const int e = top - 127;
            const float up = a.scale < 0.0f ? -pow2i(14 - e - qs) : pow2i(14 - e - qs);   // the sign of the scale goes to Q
            qf = pow2i(e) * 0x1p-14f;
#pragma unroll 2
            for (int i = 0; i < QC; ++i) {
                const uint4 v = ld(i);
                st_shared16(own(i), pack_f16x2(bf_lo(v.x) * up, bf_hi(v.x) * up),
                            pack_f16x2(bf_lo(v.y) * up, bf_hi(v.y) * up), pack_f16x2(bf_lo(v.z) * up, bf_hi(v.z) * up),
                            pack_f16x2(bf_lo(v.w) * up, bf_hi(v.w) * up));
            }
            fence_async();
            arrive_release(qfull(mi));
        };
        find();
        if (run.live()) load_q();
        while (run.live()) {
            const Unit u = run.u;
            const int tile = run.tile, len = run.len;
            float mr = kNoMax, l = 0.0f;
            int eo = kNoScale;                // O is in units of 2^eo
            for (int k = 0; k < len; ++k, ++kc, ++sc) {
                const uint32_t m = sb + P::OFF_M + (kc % P::META) * P::M_BYTES;
                uint32_t fk = smem_u32(s_factor[mi][kc & 1]);
                const int j0 = tile_pos<KT>(u, tile + k);
                // The columns' factors, before S is ready where their look-up can be waited for: from the second
                // tile of a run on, when the one before it in the ring is known to be past (a parity only tells a
                // phase from its neighbours); S of the first tile is behind its look-up.
                if (k == 0) wait_for(sfull(mi), sc & 1u, abort_flag, kErrEpilogue);
                else wait_for(mfull(kc), (kc / P::META) & 1u, abort_flag, kErrEpilogue);
                const float fcol = row < KT ? __uint_as_float(ld_shared_u32(m + P::M_DK + 4 * row)) * qf : 1.0f;
                // a factor that is no positive number is dealt with column by column below
                const bool odd = !(fcol > 0.0f && fcol < INFINITY);
                if (row < KT) reinterpret_cast<float *>(s_factor[mi][kc & 1])[row] = odd ? 1.0f : fcol;
                uint32_t all = 0xFFFFFFFFu;
#pragma unroll
                for (int i = 0; i < KT / 32; ++i) all &= ld_shared_u32(m + P::M_LIVE + 4 * i);
                const bool odd_column =
                    wg_any(odd && ((ld_shared_u32(m + P::M_LIVE + 4 * ((row % KT) >> 5)) >> (row & 31)) & 1u));
                const bool masked = odd_column || all != 0xFFFFFFFFu || !tile_full<KT>(pv, u, j0);
                if (k > 0) wait_for(sfull(mi), sc & 1u, abort_flag, kErrEpilogue);
                tc_fence_after();
                if (!__any_sync(0xFFFFFFFFu, valid)) {       // P is whatever S holds: it only reaches O's rows of no one
                    arrive_release(pfull(mi));
                    continue;
                }
                // The first tile's maximum sets the reference before any weight is taken.  Later tiles take their
                // weights against the reference they find, and their sum tells afterwards whether one may have passed
                // 2^15: P waits in registers (S's columns become P's), and such a tile is done again.
                uint32_t pk[KT / 2];
                float dm = 0.0f, sum = 0.0f;  // the old reference less the new one
                bool again = k == 0, bad = again, hide = masked;
                if (odd_column || apart) {
                    // S by the rows' own powers of two, in two steps (2^qs may be less than a float), and by the
                    // columns' odd factors
                    const float q0 = pow2i(qs >> 1), q1 = pow2i(qs - (qs >> 1));
                    scale_s([&](int c) {
                        const float o = __uint_as_float(ld_shared_u32(m + P::M_DK + 4 * c)) * qf;
                        return o > 0.0f && o < INFINITY ? make_float2(q0, q1) : make_float2(q0 * q1, o);
                    });
                }
                while (true) {
                    const bool raise = __any_sync(0xFFFFFFFFu, bad);
                    if (hide || raise) {
                        // The maximum; and into S, -inf for what the row does not see, so that the sweep needs no mask.
                        float top = -INFINITY;
#pragma unroll 1
                        for (int i = 0; i < KT / 32; ++i) {
                            const int c0 = j0 + 32 * i;
                            const uint32_t see = below(p + 1 - c0) & (~below(wb - c0) | below(pv.sinks - c0)) &
                                                 ld_shared_u32(m + P::M_LIVE + 4 * i);
                            uint32_t x[32];
                            tmem_ld32_async(ts + 32 * i, x);
                            tmem_ld_wait(x);
                            if (hide) {
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    if (!((see >> c) & 1u)) x[c] = 0xFF800000u;   // -inf
                                tmem_st16(ts + 32 * i, x);
                                tmem_st16(ts + 32 * i + 16, x + 16);
                            }
                            if (!raise) continue;
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 f = ld_shared_f4(fk + 128 * i + 4 * c);
                                top = fmaxf(top, fmaxf(__uint_as_float(x[c]) * f.x, __uint_as_float(x[c + 1]) * f.y));
                                top = fmaxf(top, fmaxf(__uint_as_float(x[c + 2]) * f.z, __uint_as_float(x[c + 3]) * f.w));
                            }
                        }
                        if (hide) tmem_st_wait();
                        if (bad && top > kNoMax) {
                            dm = mr - (top - kBelow);
                            mr = top - kBelow;
                        }
                        if (__any_sync(0xFFFFFFFFu, raise && top > kNoMax && fabsf(top) >= 0x1p24f)) {
                            // The sweep subtracts the reference from the exact product, which can lie above the
                            // rounded one by 2^-24 of it.  Where that counts, the rounded products go into S.
                            scale_s([&](int c) { return make_float2(__uint_as_float(ld_shared_u32(fk + 4 * c)), 1.0f); });
                            fk = smem_u32(s_ones);
                        }
                        again |= raise;
                        hide = false;
                    }
                    const uint64_t mr2 = pack_ff(-mr, -mr);
                    uint64_t acc[2] = {0ull, 0ull};
                    uint32_t xa[16], xb[16];
                    float ya[16], yb[16];
                    tmem_ld16_async(ts, xa);
#pragma unroll
                    for (int i = 0; i <= KT / 16; ++i) {
                        auto &x = i & 1 ? xb : xa;
                        auto &nx = i & 1 ? xa : xb;
                        auto &y = i & 1 ? yb : ya;
                        auto &py = i & 1 ? ya : yb;
                        if (i < KT / 16) {
                            tmem_ld_wait(x);
                            if (i + 1 < KT / 16) tmem_ld16_async(ts + 16 * (i + 1), nx);
                        }
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            if (i < KT / 16) {
                                const float4 f = ld_shared_f4(fk + 64 * i + 4 * c);
                                unpack_f32x2(fma_f32x2(pack_f32x2(x[c], x[c + 1]), pack_ff(f.x, f.y), mr2), y[c], y[c + 1]);
                                unpack_f32x2(fma_f32x2(pack_f32x2(x[c + 2], x[c + 3]), pack_ff(f.z, f.w), mr2), y[c + 2], y[c + 3]);
#pragma unroll
                                for (int e = c; e < c + 4; ++e) y[e] = exp2_fast(y[e]);
                            }
                            if (i > 0) {
                                acc[0] = add_f32x2(acc[0], pack_ff(py[c], py[c + 1]));
                                acc[1] = add_f32x2(acc[1], pack_ff(py[c + 2], py[c + 3]));
                                pk[(16 * (i - 1) + c) / 2] = pack_f16x2(py[c], py[c + 1]);
                                pk[(16 * (i - 1) + c) / 2 + 1] = pack_f16x2(py[c + 2], py[c + 3]);
                            }
                        }
                    }
                    float s0, s1;
                    unpack_f32x2(add_f32x2(acc[0], acc[1]), s0, s1);
                    sum = s0 + s1;
                    bad = !(sum < kMaxSum);
                    if (again || !__any_sync(0xFFFFFFFFu, bad)) break;   // a second NaN or infinity is the result
                }
                // ---- O against the new reference and exponent; P over S's columns
                const int unit = (int)ld_shared_u32(m + P::M_EXP);
                auto rescale = [&](float al) {
                    wait_for(pvdone(mi), (sc - 1) & 1u, abort_flag, kErrEpilogue);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DH; c += 16) {
                        uint32_t o[16];
                        tmem_ld16_async(to + c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                        tmem_st16(to + c, o);
                    }
                };
                if (unit != kWide) {
                    if (__any_sync(0xFFFFFFFFu, dm != 0.0f || unit != eo)) {
                        l *= exp2_fast(dm);
                        if (k > 0) rescale(exp2_fast(dm + (float)(eo - unit)));
                        eo = unit;
                    }
                    l += sum;
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i) tmem_st16(ts + 16 * i, pk + 16 * i);
                } else {
                    // V's scales are far apart: they multiply the weights, and every row brings its products to
                    // [2^13, 2^14) by a power of two of its own, so that a scale which it does not see, or hardly
                    // weighs, costs it nothing.  Twice over the columns, eight at a time: the largest product (times
                    // 2^-16, which keeps it finite), then P.
                    const bool full = tile_full<KT>(pv, u, j0);      // otherwise scales that are none come with the result
                    float top = 0.0f, g = 0.0f;
#pragma unroll 1
                    for (int c0 = 0; c0 < 2 * KT; c0 += 8) {
                        const int cc = c0 & (KT - 1);
                        uint32_t x[8];
                        float y[8];
                        tmem_ld8_async(ts + cc, x);
                        tmem_ld_wait(x);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            float d = __uint_as_float(ld_shared_u32(m + P::M_DV + 4 * (cc + c))) * 0x1p-16f;
                            if (!full && !(fabsf(d) < INFINITY)) d = 0.0f;
                            y[c] = exp2_fast(fmaf(__uint_as_float(x[c]), __uint_as_float(ld_shared_u32(fk + 4 * (cc + c))), -mr)) * d;
                        }
                        if (c0 < KT) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(y[c]) < INFINITY ? fabsf(y[c]) : 0.0f);
                            if (cc < KT - 8) continue;
                            // what O holds has shrunk by 2^dm; whole steps, within one of that however often it does
                            int eo_new = eo - (int)fminf(floorf(mr) - floorf(mr + dm), 2000.0f);
                            if (top > 0.0f) eo_new = max(eo_new, max((int)(__float_as_uint(top) >> 23) - 127, -113) + 3);
                            const float al = exp2_fast(dm + (float)(eo - eo_new));
                            if (k > 0 && __any_sync(0xFFFFFFFFu, al != 1.0f)) rescale(al);
                            l = l * exp2_fast(dm) + sum;
                            eo = eo_new;
                            g = eo >= -110 ? pow2i(16 - eo) : 0.0f;
                        } else {                      // P's columns lie behind those still to be read
                            tmem_st4(ts + cc / 2, pack_f16x2(y[0] * g, y[1] * g), pack_f16x2(y[2] * g, y[3] * g),
                                     pack_f16x2(y[4] * g, y[5] * g), pack_f16x2(y[6] * g, y[7] * g));
                        }
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                arrive_release(pfull(mi));
            }
            // ---- the next run's Q, so that its S is under way during this run's result
            const bool whole = run.whole(), valid_was = valid;
            const int p_was = p, wb_was = wb, h_was = run.h, seq = run.who.x;
            const int64_t orow_was = orow;
            if (tile == 0 && !whole && threadIdx.x == 128)
                a.split[blockIdx.x] = make_int4(run.bi, run.h, run.last_cta(), 0);
            run.next();
            find();
            if (run.live()) load_q();
            // ---- this run's result
            wait_for(pvdone(mi), (sc - 1) & 1u, abort_flag, kErrEpilogue);
            tc_fence_after();
            // 2^eo in two steps: it may be more than a float, and a weighted mean less
            const int e0 = max(eo >> 1, -126), e1 = max(eo - (eo >> 1), -126);
            const float r = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            float by = r * pow2i(e0) * pow2i(e1);
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (tile == 0 ? 1 : 0)) * ((int64_t)ROWS * (DH + 2));
            if (*reinterpret_cast<volatile uint32_t *>(&s_poison) != 0u) {
                // values that were taken out of V, all infinite or NaN: back into the rows that see them
#pragma unroll 1
                for (int c = 0; c < DH; c += 8) {
                    uint32_t o[8];
                    tmem_ld8_async(to + c, o);
                    tmem_ld_wait(o);
                    if (by == 0.0f)
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
#pragma unroll 1
                    for (int k = 0; k < len; ++k) {
                        const int j0 = tile_pos<KT>(u, tile + k);
                        if (c >= pv.Dh || tile_full<KT>(pv, u, j0)) continue;
#pragma unroll 1
                        for (int j = j0; j < j0 + KT; ++j) {
                            if (j > p_was || !(j >= wb_was || j < pv.sinks)) continue;
                            const int s = pv.slot(seq, j);
                            if (s < 0) continue;
                            const float d = pv.vs[(int64_t)s * pv.H + h_was];
                            const uint8_t *codes = pv.vc + (uint64_t)(uint32_t)s * (uint64_t)(pv.H * pv.Dh) + h_was * pv.Dh + c;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float w = fp8x2_to_float2<FMT>((uint16_t)codes[i]).x * d;
                                if (!(fabsf(w) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + w);
                            }
                        }
                    }
                    __syncwarp();
                    tmem_st4(to + c, o[0], o[1], o[2], o[3]);
                    tmem_st4(to + c + 4, o[4], o[5], o[6], o[7]);
                }
                tmem_st_wait();
                if (by == 0.0f) by = 1.0f;        // nothing finite is left; an infinity stays one
            }
#pragma unroll 1
            for (int c = 0; c < DH; c += 32) {
                uint32_t o[32];
                tmem_ld32_async(to + c, o);
                tmem_ld_wait(o);
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * by;
                if (!valid_was || c >= pv.Dh) continue;
                if (whole) {
                    __nv_bfloat16 *op = a.out + orow_was * pv.Dh + c;
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (c + i < pv.Dh) {
                            uint4 w;
                            w.x = pack_bf16x2(v[i], v[i + 1]);
                            w.y = pack_bf16x2(v[i + 2], v[i + 3]);
                            w.z = pack_bf16x2(v[i + 4], v[i + 5]);
                            w.w = pack_bf16x2(v[i + 6], v[i + 7]);
                            *reinterpret_cast<uint4 *>(op + i) = w;
                        }
                } else {
                    float *pp = part + (int64_t)(mi * 128 + row) * DH + c;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4 *>(pp + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            tc_fence_before();
            if (valid_was) {
                if (whole) {
                    if (a.lse) a.lse[orow_was] = l == 0.0f ? -INFINITY : (mr + log2f(l)) * kLn2;
                } else {
                    *reinterpret_cast<float2 *>(part + (int64_t)ROWS * DH + 2 * (mi * 128 + row)) = make_float2(mr, l);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// Joins the parts of the units that more than one CTA worked on: a warp per
// row, a lane per DH / 32 elements, the CTAs in order.
template <int DH>
__global__ void __launch_bounds__(256)
k_prefill_join(const PagedView pv, const PrefillArgs a) {
    using P = Pre<DH>;
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int first = blockIdx.x;             // the CTA that began the unit, with the second of its parts
    const int4 sp = a.split[first];
    if (sp.x < 0) return;
    const int2 who = a.block[sp.x];
    const int h = sp.y, last = sp.z;
    const Unit u = unit_of<P::ROWS, P::KT>(pv, a, who.x, who.y);
    const int64_t stride = (int64_t)P::ROWS * (DH + 2);
    for (int row = blockIdx.y * 8 + warp; row < u.rho1 - u.rho0; row += gridDim.y * 8) {
        const int rho = u.rho0 + row, tok = rho / a.G, g = rho - tok * a.G;
        const int64_t orow = (u.t0 + tok) * (int64_t)pv.H * a.G + (int64_t)h * a.G + g;
        float mx = kNoMax, sum = 0.0f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int c = first; c <= last; ++c) {
            const float *p = a.part + (2 * (int64_t)c + (c == first ? 1 : 0)) * stride;
            const float2 v = *reinterpret_cast<const float2 *>(p + (int64_t)P::ROWS * DH + 2 * row);
            const float nm = fmaxf(mx, v.x), al = exp2_fast(mx - nm), be = exp2_fast(v.x - nm);
            mx = nm;
            sum = fmaf(sum, al, v.y * be);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = fmaf(acc[e], al, p[(int64_t)row * DH + lane * E + e] * be);
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane * E + e < pv.Dh)
                a.out[orow * pv.Dh + lane * E + e] = __float2bfloat16(sum == 0.0f ? 0.0f : acc[e] / sum);
        if (lane == 0 && a.lse) a.lse[orow] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
}

}  // namespace

using namespace fp8q_host;

namespace {

struct PrefillPlan {
    int DH, ctas;
    int64_t blocks;           // row blocks, at most
    size_t part, split, hdr, first, block, start, total;
};

PrefillPlan prefill_plan(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t Dh, int sms) {
    PrefillPlan p;
    const int64_t G = Hq / H;
    p.DH = Dh <= 64 ? 64 : Dh <= 128 ? 128 : 256;
    p.ctas = sms;
    const int64_t rows = p.DH <= 128 ? 256 : 128, blocks = T * G / rows + std::min(B, T);
    p.blocks = blocks;
    size_t at = 0;
    auto take = [&at](size_t n) {
        const size_t was = at;
        at += (n + 255) & ~(size_t)255;
        return was;
    };
    p.part = take((size_t)p.ctas * 2 * rows * (p.DH + 2) * 4);
    p.split = take((size_t)p.ctas * 16);
    p.hdr = take(16);
    p.first = take((size_t)B * 8);
    p.block = take((size_t)blocks * 8);
    p.start = take((size_t)p.ctas * 16);
    p.total = at;
    return p;
}

// 3-D map over codes [slots, H, Dh]: boxes of `rows` slots of one head, DH bytes
// wide (a smaller head reads zeros behind its end).
bool make_map_tiles(CUtensorMap *map, const void *codes, const PagedView &pv, int DH, int rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)pv.Dh, (cuuint64_t)pv.H, (cuuint64_t)pv.bs.d * (cuuint64_t)pv.num_blocks};
    cuuint64_t strides[2] = {(cuuint64_t)pv.Dh, (cuuint64_t)pv.Dh * (cuuint64_t)pv.H};
    cuuint32_t box[3] = {(cuuint32_t)DH, 1, (cuuint32_t)rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(codes), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int DH, bool TMA>
cudaError_t launch_main(const PagedView &pv, const PrefillArgs &a, const PrefillPlan &p, cudaStream_t s) {
    using P = Pre<DH>;
    // shared memory and the register split are checked once per device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, k_prefill<FMT, DH, TMA>);
        if (e != cudaSuccess) return e;
        // the split adds up to what these give a block: with fewer, a warpgroup's share would be waited for for good
        if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(k_prefill<FMT, DH, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    CUtensorMap tk = {}, tv = {};
    if (TMA && (!make_map_tiles(&tk, pv.kc, pv, DH, a.box) || !make_map_tiles(&tv, pv.vc, pv, DH, a.box)))
        return cudaErrorInvalidValue;
    return pdl_launch(k_prefill<FMT, DH, TMA>, dim3(p.ctas), dim3(kThreads), P::SMEM, s, tk, tv, pv, a);
}

template <int FMT, int DH>
cudaError_t launch_prefill(const PagedView &pv, const PrefillArgs &a, const PrefillPlan &p, cudaStream_t s) {
    using P = Pre<DH>;
    cudaError_t e;
    e = pdl_launch(k_prefill_plan<P::ROWS, P::KT>, dim3(1), dim3(kPlanThreads), 0, s, pv, a);
    if (e != cudaSuccess) return e;
    // pages that 8 rows do not divide, and a pool without pages, have no boxes
    e = pv.bs.d % 8 == 0 && pv.num_blocks > 0 ? launch_main<FMT, DH, true>(pv, a, p, s)
                                              : launch_main<FMT, DH, false>(pv, a, p, s);
    if (e != cudaSuccess) return e;
    return pdl_launch(k_prefill_join<DH>, dim3(p.ctas, 8), dim3(256), 0, s, pv, a);
}

}  // namespace

fp8_status fp8q_host::prefill_workspace(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t Dh, size_t *bytes) {
    int sms;
    const fp8_status st = check_device(&sms);
    if (st != FP8_OK) return st;
    *bytes = prefill_plan(T, B, Hq, H, Dh, sms).total;
    return FP8_OK;
}

extern "C" fp8_status fp8_paged_attention_prefill(
    const void *q_bf16, int64_t ld_q, int64_t T, const int64_t *q_offsets, int64_t B, int64_t Hq,
    const uint8_t *k_cache, const float *k_scale, const uint8_t *v_cache, const float *v_scale, int64_t H, int64_t Dh,
    int64_t block_size, int64_t num_blocks, fp8_format fmt, const int32_t *block_table, const int32_t *seq_lens,
    int64_t max_blocks, int64_t window, int64_t sinks, float softmax_scale, void *out_bf16, float *lse,
    void *workspace, size_t workspace_bytes, void *stream) {
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return FP8_ERR_INVALID_ARG;
    fp8_status st = attn_shape(ld_q, T, B, Hq, H, Dh, block_size, num_blocks, max_blocks, window, sinks);
    if (st != FP8_OK) return st;
    if (!std::isfinite(softmax_scale)) return FP8_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return FP8_OK;
    if (!q_offsets) return FP8_ERR_INVALID_ARG;
    st = attn_pointers(q_bf16, ld_q, k_cache, k_scale, v_cache, v_scale, num_blocks, block_table, seq_lens, max_blocks,
                       out_bf16, workspace);
    if (st != FP8_OK) return st;
    int sms;
    st = check_device(&sms);
    if (st != FP8_OK) return st;
    const PrefillPlan p = prefill_plan(T, B, Hq, H, Dh, sms);
    if (!workspace || workspace_bytes < p.total) return FP8_ERR_INVALID_ARG;
    const PagedView pv = make_paged_view(k_cache, k_scale, v_cache, v_scale, H, Dh, block_size, num_blocks,
                                         block_table, seq_lens, max_blocks, window, sinks);
    uint8_t *ws = (uint8_t *)workspace;
    PrefillArgs a = {};
    a.q = (const __nv_bfloat16 *)q_bf16;
    a.ld_q = ld_q;
    a.q_off = q_offsets;
    a.T = T;
    a.B = (int)B;
    a.G = (int)(Hq / H);
    a.gdiv = make_fastdiv((uint32_t)a.G);
    a.ctas = p.ctas;
    a.max_blocks = p.blocks;
    a.box = block_size % 32 == 0 ? 32 : block_size % 16 == 0 ? 16 : 8;
    a.scale = softmax_scale;
    a.out = (__nv_bfloat16 *)out_bf16;
    a.lse = lse;
    a.part = (float *)(ws + p.part);
    a.split = (int4 *)(ws + p.split);
    a.hdr = (int64_t *)(ws + p.hdr);
    a.first_block = (int64_t *)(ws + p.first);
    a.block = (int2 *)(ws + p.block);
    a.start = (longlong2 *)(ws + p.start);
    cudaStream_t s = as_stream(stream);
    cudaError_t e;
    if (p.DH == 64) e = fmt == FP8_E4M3 ? launch_prefill<FP8_E4M3, 64>(pv, a, p, s) : launch_prefill<FP8_E5M2, 64>(pv, a, p, s);
    else if (p.DH == 128) e = fmt == FP8_E4M3 ? launch_prefill<FP8_E4M3, 128>(pv, a, p, s) : launch_prefill<FP8_E5M2, 128>(pv, a, p, s);
    else e = fmt == FP8_E4M3 ? launch_prefill<FP8_E4M3, 256>(pv, a, p, s) : launch_prefill<FP8_E5M2, 256>(pv, a, p, s);
    return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

// This file's device error word (fp8_device_error reads it with the others').
fp8_status fp8q_prefill_device_error(uint32_t *out, int clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof(v)) != cudaSuccess) return FP8_ERR_CUDA;
    *out = v;
    if (clear) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_gemm_error, &z, sizeof(z)) != cudaSuccess) return FP8_ERR_CUDA;
    }
    return FP8_OK;
}
