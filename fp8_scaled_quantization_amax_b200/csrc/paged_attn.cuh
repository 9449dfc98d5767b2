// paged_attn.cuh -- what the two attention calls over the paged FP8 KV cache
// share (paged_decode.cu, paged_prefill.cu): small device functions and
// host-side checks.
#pragma once

#include "paged.cuh"
#include "tc.cuh"

namespace {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// Four codes -> two fp16 pairs (exact).
template <int FMT>
__device__ __forceinline__ void to_f16x4(uint32_t c, uint32_t &lo, uint32_t &hi) {
    if (FMT == FP8_E4M3)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(c));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e5m2x2 %0, l;\n\tcvt.rn.f16x2.e5m2x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(c));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp; 0 at -inf and below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 2^e for -126 <= e <= 127; infinity at 128
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace

namespace fp8q_host {

constexpr int kAttnMaxDh = 256;
// rows of q times query heads: row numbers, and the ends of the row blocks that hold them, stay below 2^31
constexpr int64_t kAttnMaxRows = 0x7FFF0000ll;

inline fp8_status attn_shape(int64_t ld_q, int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t Dh,
                             int64_t block_size, int64_t num_blocks, int64_t max_blocks, int64_t window,
                             int64_t sinks) {
    const fp8_status st = paged_cache_shape(H, Dh, block_size, num_blocks);
    if (st != FP8_OK) return st;
    if (Dh % 16 || Dh > kAttnMaxDh || Hq < 1 || Hq > 0x7FFFFFFFll || Hq % H) return FP8_ERR_SHAPE;
    if (B < 0 || B > 65535 || T < 0 || T > 0x7FFFFFFFll || T * Hq > kAttnMaxRows || max_blocks < 0 || window < 0 ||
        sinks < 0)
        return FP8_ERR_SHAPE;
    if (max_blocks > kPagedMaxContext / block_size || ld_q < Hq * Dh) return FP8_ERR_SHAPE;
    return FP8_OK;
}

inline fp8_status attn_pointers(const void *q, int64_t ld_q, const uint8_t *kc, const float *ks, const uint8_t *vc,
                                const float *vs, int64_t num_blocks, const int32_t *table, const int32_t *lens,
                                int64_t max_blocks, const void *out, const void *ws) {
    if (!lens || !q || !out || (max_blocks > 0 && !table)) return FP8_ERR_INVALID_ARG;
    if (num_blocks > 0 && (!kc || !ks || !vc || !vs)) return FP8_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || ld_q % 8 || !aligned16(kc) || !aligned16(vc) || !aligned16(ws))
        return FP8_ERR_ALIGNMENT;
    return FP8_OK;
}

// Workspace of the prefill call (paged_prefill.cu), current device.
fp8_status prefill_workspace(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t Dh, size_t *bytes);

}  // namespace fp8q_host
