// kvsel_prompt_attention: causal attention over packed prompts with grouped heads.
//
// Sequence s holds tokens [cu[s], cu[s+1]); row i of it sees its rows 0..i:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale log2e (q_i . k_j - max)),
//   lse = ln sum_j e^(scale q_i . k_j).
// One block per (token, query head): a thread takes one key's dot product of a chunk
// of 128, then one dim of the weighted sum, with the softmax's running maximum and
// sum kept across chunks in fp32.
#include <cuda_bf16.h>
#include <limits.h>

#include "kvsel_internal.h"

namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct PromptArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t* cu;
    int S, T, Hq, Hkv, D;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
};

__global__ void __launch_bounds__(kThreads) prompt_attention_kernel(const PromptArgs a) {
    __shared__ float qs[128], ps[kThreads], red[4];
    const int tid = threadIdx.x, h = blockIdx.y, i = blockIdx.x;
    const int g = h / (a.Hq / a.Hkv);
    // the last sequence that starts at or before token i
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= i) lo = mid; else hi = mid;
    }
    const int first = __ldg(a.cu + lo);
    if (i < first || i >= __ldg(a.cu + lo + 1)) return;
    if (first < 0) {
        if (tid == 0) atomicOr(a.err, (unsigned)KVSEL_DEV_BAD_LENGTH);
        return;
    }
    if (tid < a.D) qs[tid] = __bfloat162float(a.q[i * a.q_stride + (int64_t)h * a.D + tid]);
    float m = -INFINITY, l = 0.f, o = 0.f;
    const float c = a.scale * kLog2e;
    __syncthreads();
    for (int j0 = first; j0 <= i; j0 += kThreads) {
        const int j = j0 + tid;
        float x = -INFINITY;
        if (j <= i) {
            x = 0.f;
            const uint4* kr = reinterpret_cast<const uint4*>(a.k + j * a.k_stride + (int64_t)g * a.D);
            for (int d = 0; d < a.D / 8; ++d) {
                const uint4 w = __ldg(kr + d);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    x = fmaf(__uint_as_float(u[b] << 16), qs[d * 8 + 2 * b], x);
                    x = fmaf(__uint_as_float(u[b] & 0xFFFF0000u), qs[d * 8 + 2 * b + 1], x);
                }
            }
            x *= c;
        }
        float mx = x;
#pragma unroll
        for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float base = mn == -INFINITY ? 0.f : mn, corr = exp2f(m - base);
        m = mn;
        ps[tid] = j <= i ? exp2f(x - base) : 0.f;
        l *= corr, o *= corr;
        __syncthreads();
        const int cnt = min(kThreads, i + 1 - j0);
        for (int b = 0; b < cnt; ++b) {
            const float p = ps[b];
            l += p;
            if (tid < a.D) o = fmaf(p, __bfloat162float(a.v[(j0 + b) * a.v_stride + (int64_t)g * a.D + tid]), o);
        }
        __syncthreads();
    }
    if (tid < a.D) a.out[((int64_t)i * a.Hq + h) * a.D + tid] = __float2bfloat16_rn(o / l);
    if (a.lse && tid == 0) a.lse[(int64_t)i * a.Hq + h] = (m + log2f(l)) * kLn2;
}

}  // namespace

extern "C" int kvsel_prompt_attention(kvsel_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens, int S, int T, int Hq,
                                      int Hkv, int D, float scale, void* out, float* lse, void* stream) {
    const kvsel_trace trace_("kvsel_prompt_attention");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (S < 0 || T < 0 || Hq <= 0 || Hkv <= 0) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "prompt_attention: bad sizes");
    if (Hq % Hkv) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "prompt_attention: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
    if (D != 64 && D != 128) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "prompt_attention: D=%d unsupported", D);
    if (S > 65535 || Hq > 65535 || T > (1 << 24))
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "prompt_attention: S, T or Hq too large");
    if (!(scale > 0.f) || scale > 1e30f)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "prompt_attention: scale must be positive and finite");
    if (S == 0 || T == 0) return KVSEL_OK;
    if (!q || !k || !v || !cu_seqlens || !out) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "prompt_attention: null pointer");
    if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "prompt_attention: token stride smaller than a token's heads");
    auto off16 = [](const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15u) || (stride * 2) % 16; };
    if (off16(q, q_stride) || off16(k, k_stride) || off16(v, v_stride) || off16(out, 0))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "prompt_attention: q, k, v, out and the strides must be 16-byte aligned");
    const PromptArgs a{(const __nv_bfloat16*)q, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, q_stride, k_stride,
                       v_stride, cu_seqlens, S, T, Hq, Hkv, D, scale, (__nv_bfloat16*)out, lse, ctx->dev_err};
    prompt_attention_kernel<<<dim3(T, Hq), kThreads, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "prompt_attention launch");
}
