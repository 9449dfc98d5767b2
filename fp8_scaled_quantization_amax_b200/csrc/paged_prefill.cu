// paged_prefill.cu -- causal attention of several new tokens per sequence over
// the paged FP8 KV cache, read in place.
#include "paged_attn.cuh"

using namespace fp8q;

namespace {

constexpr int kT = 128;       // threads = positions per tile
constexpr int kMaxDh = 256;

template <int FMT>
__device__ __forceinline__ float fp8_to_float(uint8_t c) { return fp8x2_to_float2<FMT>((uint16_t)c).x; }

__device__ __forceinline__ float block_reduce(float v, bool is_max, float *buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = is_max ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = buf[0];
    for (int i = 1; i < kT / 32; ++i) r = is_max ? fmaxf(r, buf[i]) : r + buf[i];
    return r;
}

// One CTA per (token, query head): 128 positions at a time, a thread's
// position each for the logits, a thread's two head elements each for P V.
template <int FMT>
__global__ void __launch_bounds__(kT)
k_paged_attn_rows(PagedView pv, const __nv_bfloat16 *__restrict__ q, int64_t ld_q, const int64_t *__restrict__ q_off,
                  int64_t B, int64_t T, int Hq, float scale, __nv_bfloat16 *__restrict__ out,
                  float *__restrict__ lse) {
    __shared__ float qs[kMaxDh], ps[kT], buf[kT / 32];
    __shared__ int ss[kT];
    const int64_t t = blockIdx.x / Hq;
    const int hq = (int)(blockIdx.x % Hq), h = hq / (Hq / pv.H), Dh = pv.Dh, tid = threadIdx.x;
    int64_t b = t;
    int p;
    if (q_off) {
        int64_t lo = 0, hi = B - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (q_off[mid] <= t) lo = mid; else hi = mid - 1;
        }
        b = lo;
        const int64_t o0 = max((int64_t)0, min(T, q_off[b])), o1 = max((int64_t)0, min(T, q_off[b + 1]));
        if (t < o0 || t >= o1) return;
        p = (int)max((int64_t)-1, pv.length(b) - (o1 - o0) + (t - o0));
    } else {
        p = pv.length(b) - 1;
    }
    for (int d = tid; d < Dh; d += kT) qs[d] = __bfloat162float(q[t * ld_q + (int64_t)hq * Dh + d]);
    const int w0 = pv.window_begin(p), sinks = min(pv.sinks, w0);
    const int vis = p + 1 - w0 + sinks;   // the sinks, then the window
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    bool any = false;
    for (int i0 = 0; i0 < vis; i0 += kT) {
        const int i = i0 + tid, j = i < sinks ? i : w0 + i - sinks;
        const int s = i < vis ? pv.slot(b, j) : -1;
        __syncthreads();
        float z = -INFINITY;
        if (s >= 0) {
            const uint8_t *k = pv.kc + ((int64_t)s * pv.H + h) * Dh;
            float a = 0.f;
            for (int d = 0; d < Dh; ++d) a = fmaf(qs[d], fp8_to_float<FMT>(k[d]), a);
            z = a * (pv.ks[(int64_t)s * pv.H + h] * scale);
        }
        any |= __syncthreads_or(s >= 0) != 0;
        const float mn = fmaxf(m, block_reduce(z, true, buf));
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float w = s >= 0 ? expf(z - ref) : 0.f;
        const float alpha = m == -INFINITY ? 0.f : expf(m - ref);
        l = l * alpha + block_reduce(w, false, buf);
        m = mn;
        ss[tid] = s;
        ps[tid] = s >= 0 ? w * pv.vs[(int64_t)s * pv.H + h] : 0.f;
        __syncthreads();
        acc[0] *= alpha;
        acc[1] *= alpha;
        for (int i1 = 0; i1 < kT; ++i1) {
            const int si = ss[i1];
            if (si < 0) continue;
            const uint8_t *v = pv.vc + ((int64_t)si * pv.H + h) * Dh;
            for (int e = 0; e < 2; ++e)
                if (tid + e * kT < Dh) acc[e] = fmaf(ps[i1], fp8_to_float<FMT>(v[tid + e * kT]), acc[e]);
        }
    }
    const int64_t row = t * Hq + hq;
    for (int e = 0; e < 2; ++e)
        if (tid + e * kT < Dh) out[row * Dh + tid + e * kT] = __float2bfloat16(any ? acc[e] / l : 0.f);
    if (lse && tid == 0) lse[row] = any ? m + logf(l) : -INFINITY;
}

}  // namespace

using namespace fp8q_host;

fp8_status fp8q_host::prefill_workspace(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t Dh, size_t *bytes) {
    *bytes = 0;
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
    const PagedView pv = make_paged_view(k_cache, k_scale, v_cache, v_scale, H, Dh, block_size, num_blocks,
                                         block_table, seq_lens, max_blocks, window, sinks);
    cudaStream_t s = as_stream(stream);
    auto run = [&](auto rows) {
        rows<<<dim3((unsigned)(T * Hq)), kT, 0, s>>>(pv, (const __nv_bfloat16 *)q_bf16, ld_q, q_offsets, B, T,
                                                     (int)Hq, softmax_scale, (__nv_bfloat16 *)out_bf16, lse);
    };
    if (fmt == FP8_E4M3) run(k_paged_attn_rows<FP8_E4M3>);
    else run(k_paged_attn_rows<FP8_E5M2>);
    return cudaPeekAtLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}
