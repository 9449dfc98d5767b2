// paged_attn.cuh -- host-side checks shared by the two attention calls over
// the paged FP8 KV cache (paged_decode.cu, paged_prefill.cu).
#pragma once

#include "paged.cuh"

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
