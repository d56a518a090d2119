// kvsel_attention_mass: the softmax weight that the new tokens give to each token of their session.
//
//   score_out[s,j] = score_in[s,j] + sum_{i,h} e^(scale q_ih . k_j - lse_ih)   over the rows whose token i sees j.
//
// A thread per token j, its key row in registers; one kv head after the other.
#include <cuda_bf16.h>

#include "pool_tokens.cuh"

namespace {

struct MassArgs {
    const __nv_bfloat16* q;
    int64_t q_stride;
    const float* lse;
    const int32_t *cu, *lens;
    int S, T, Hq, Hkv;
    const __nv_bfloat16* k;
    int64_t k_stride;
    TokenMap map;
    float scale;
    const float* before;
    float* score;
    int64_t score_ld;
    unsigned* err;
};

template <int D>
__global__ void __launch_bounds__(128) attention_mass_kernel(const MassArgs a) {
    const int s = blockIdx.y;
    unsigned err = blockIdx.x == 0 ? session_errors(a.cu, a.lens, a.T, a.map.reach, s) : 0u;
    const Session x = session_at(a.cu, a.lens, a.T, a.map.reach, s);
    const int32_t* const row = a.map.map + (int64_t)s * a.map.ld;
    const int G = a.Hq / a.Hkv;
    for (int64_t j = (int64_t)blockIdx.x * 128 + threadIdx.x; j < a.map.reach; j += (int64_t)gridDim.x * 128) {
        float sum = a.before ? a.before[s * a.score_ld + j] : 0.f;
        const int slot = j < x.len && x.count > 0 ? live_slot(a.map, raw_entry(a.map, row, (int)j), (int)j, err) : -1;
        if (slot >= 0) {
            const int i0 = max(0, (int)j - (x.len - x.count));
            float mass = 0.f;
            for (int g = 0; g < a.Hkv; ++g) {
                float k[D];
                for (int e = 0; e < D; ++e) k[e] = __bfloat162float(a.k[(int64_t)slot * a.k_stride + (int64_t)g * D + e]);
                for (int i = i0; i < x.count; ++i)
                    for (int h = g * G; h < (g + 1) * G; ++h) {
                        const float lse = a.lse[(int64_t)(x.first + i) * a.Hq + h];
                        const __nv_bfloat16* const q = a.q + (int64_t)(x.first + i) * a.q_stride + (int64_t)h * D;
                        float dot = 0.f;
#pragma unroll
                        for (int e = 0; e < D; ++e) dot += k[e] * __bfloat162float(q[e]);
                        if (lse != -INFINITY) mass += expf(dot * a.scale - lse);
                    }
            }
            sum += mass;
        }
        a.score[s * a.score_ld + j] = sum;
    }
    if (err) atomicOr(a.err, err);
}

}  // namespace

extern "C" int kvsel_attention_mass(kvsel_ctx* ctx, const void* q, int64_t q_stride, const float* lse, const int32_t* cu_new,
                                    int S, int T, int Hq, int Hkv, int D, const void* k_pool, int64_t k_stride, int P, int page,
                                    const int32_t* seq_lens, const int32_t* slot_map, const int32_t* block_table, int ld,
                                    int dead_slot, float scale, const float* score_in, float* score_out, int64_t score_ld,
                                    void* stream) {
    const kvsel_trace trace_("kvsel_attention_mass");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    const void* pools[1] = {k_pool};
    TokenMap map;
    rc = check_pool_call(ctx, "attention_mass", S, T, Hq, Hkv, D, q_stride, pools, &k_stride, 1, P, page, slot_map, block_table,
                         ld, dead_slot, scale, &map);
    if (rc) return rc;
    if (score_ld < map.reach) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "attention_mass: score rows shorter than the map's reach");
    if (S == 0 || map.reach == 0) return KVSEL_OK;
    if (!cu_new || !seq_lens || !score_out || (T > 0 && (!q || !lse)))
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "attention_mass: null pointer");
    if (reinterpret_cast<uintptr_t>(q) & 15u) return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "attention_mass: q must be 16-byte aligned");
    const MassArgs a{(const __nv_bfloat16*)q, q_stride, lse, cu_new, seq_lens, S, T, Hq, Hkv, (const __nv_bfloat16*)k_pool,
                     k_stride, map, scale, score_in, score_out, score_ld, ctx->dev_err};
    const dim3 grid((unsigned)min(map.reach / 128 + 1, 8 * ctx->num_sms), S);
    if (D == 64)
        attention_mass_kernel<64><<<grid, 128, 0, (cudaStream_t)stream>>>(a);
    else
        attention_mass_kernel<128><<<grid, 128, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "attention_mass launch");
}
