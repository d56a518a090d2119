// kvsel_pool_attention: attention of packed new tokens over the bf16 page pools.
//
// Token i of a session sits at position pos = len - count + i and sees the live tokens j <= pos:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = e^(scale q . k_j - max),  lse = ln sum_j e^(scale q . k_j).
//
// A warp per (token, head), its lanes on the dims; one pass over the keys with the running maximum and sum.
#include <cuda_bf16.h>

#include "pool_tokens.cuh"

namespace {

struct PoolArgs {
    const __nv_bfloat16* q;
    int64_t q_stride;
    const int32_t *cu, *lens;
    int S, T, Hq, Hkv;
    const __nv_bfloat16 *k, *v;
    int64_t k_stride, v_stride;
    TokenMap map;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
};

template <int D>
__global__ void __launch_bounds__(256) pool_attention_kernel(const PoolArgs a) {
    const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kPer = D / 32;
    unsigned err = blockIdx.x == 0 ? session_errors(a.cu, a.lens, a.T, a.map.reach, s) : 0u;
    const Session x = session_at(a.cu, a.lens, a.T, a.map.reach, s);
    const int32_t* const row = a.map.map + (int64_t)s * a.map.ld;
    for (int64_t w = (int64_t)blockIdx.x * 8 + warp; w < (int64_t)x.count * a.Hq; w += (int64_t)gridDim.x * 8) {
        const int i = (int)(w / a.Hq), h = (int)(w % a.Hq), g = h / (a.Hq / a.Hkv), pos = x.len - x.count + i;
        float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
        for (int e = 0; e < kPer; ++e) {
            q[e] = __bfloat162float(a.q[(int64_t)(x.first + i) * a.q_stride + (int64_t)h * D + lane + 32 * e]);
            o[e] = 0.f;
        }
        for (int j = 0; j <= pos; ++j) {
            const int slot = live_slot(a.map, row, j, err);
            if (slot < 0) continue;
            float dot = 0.f;
            for (int e = 0; e < kPer; ++e)
                dot += q[e] * __bfloat162float(a.k[(int64_t)slot * a.k_stride + (int64_t)g * D + lane + 32 * e]);
            for (int k = 16; k; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
            dot *= a.scale;
            const float top = !(dot <= m) ? dot : m, f = m == top ? 1.f : expf(m - top), p = dot == -INFINITY ? 0.f : expf(dot - top);
            m = top;
            l = l * f + p;
            for (int e = 0; e < kPer; ++e)
                o[e] = o[e] * f + p * __bfloat162float(a.v[(int64_t)slot * a.v_stride + (int64_t)g * D + lane + 32 * e]);
        }
        const int64_t at = (int64_t)(x.first + i) * a.Hq + h;
        for (int e = 0; e < kPer; ++e) a.out[at * D + lane + 32 * e] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] / l);
        if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : m + logf(l);
    }
    if (err) atomicOr(a.err, err);
}

}  // namespace

extern "C" int kvsel_pool_attention(kvsel_ctx* ctx, const void* q, int64_t q_stride, const int32_t* cu_new, int S, int T,
                                    int Hq, int Hkv, int D, const void* k_pool, const void* v_pool, int64_t k_stride,
                                    int64_t v_stride, int P, int page, const int32_t* seq_lens, const int32_t* slot_map,
                                    const int32_t* block_table, int ld, int dead_slot, float scale, void* out, float* lse,
                                    void* stream) {
    const kvsel_trace trace_("kvsel_pool_attention");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    const void* pools[2] = {k_pool, v_pool};
    const int64_t strides[2] = {k_stride, v_stride};
    TokenMap map;
    rc = check_pool_call(ctx, "pool_attention", S, T, Hq, Hkv, D, q_stride, pools, strides, 2, P, page, slot_map, block_table,
                         ld, dead_slot, scale, &map);
    if (rc) return rc;
    if (S == 0 || T == 0) return KVSEL_OK;
    if (!q || !cu_new || !seq_lens || !out) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "pool_attention: null pointer");
    if ((reinterpret_cast<uintptr_t>(q) & 15u) || (reinterpret_cast<uintptr_t>(out) & 15u))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "pool_attention: q and out must be 16-byte aligned");
    const PoolArgs a{(const __nv_bfloat16*)q, q_stride, cu_new, seq_lens, S, T, Hq, Hkv, (const __nv_bfloat16*)k_pool,
                     (const __nv_bfloat16*)v_pool, k_stride, v_stride, map, scale, (__nv_bfloat16*)out, lse, ctx->dev_err};
    const dim3 grid((unsigned)min((int64_t)T * Hq / 8 + 1, (int64_t)8 * ctx->num_sms), S);
    if (D == 64)
        pool_attention_kernel<64><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    else
        pool_attention_kernel<128><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "pool_attention launch");
}
