// kvsel_kv4_attention: attention of a few query rows per session over the 4-bit
// paged cache.
//
// Row (s, t, h) sits at position pos = len_s - Tq + t of session s and sees the
// tokens j <= pos whose slot is live:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale log2e (q . k_j - max)),
//   lse = ln sum_j e^(scale q . k_j).
// One block per row; a chunk of 128 tokens at a time: a thread takes one token's
// dot product, then one or two dims of the weighted sum, with the running maximum
// and sum of the softmax kept across chunks in fp32.
#include <cuda_bf16.h>
#include <limits.h>

#include "kv4_format.cuh"
#include "kvsel_internal.h"

namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnArgs {
    const __nv_bfloat16* q;
    int64_t q_stride;
    int Tq, Hq, Hkv, D;
    const uint8_t *kc, *ks, *vc, *vs;
    int P, page;
    const int32_t* lens;
    const int32_t* slot_map;
    const int32_t* table;
    int ld;             // of slot_map or table
    int max_len;        // tokens that the map or table reaches
    int dead;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    unsigned* err;
};

// Slot of token j, -1 where it is not live; bad slots set err.
__device__ __forceinline__ int slot_of(const AttnArgs& a, int s, int j, unsigned& err) {
    int slot;
    if (a.slot_map) {
        slot = __ldg(a.slot_map + (int64_t)s * a.ld + j);
    } else {
        const int b = j / a.page, pg = __ldg(a.table + (int64_t)s * a.ld + b);
        if (pg < 0) return -1;
        if (pg >= a.P) {
            err |= KVSEL_DEV_BAD_PAGE;
            return -1;
        }
        slot = pg * a.page + (j - b * a.page);
    }
    if (slot < 0 || slot == a.dead) return -1;
    if ((int64_t)slot >= (int64_t)a.P * a.page) {
        err |= KVSEL_DEV_BAD_SLOT;
        return -1;
    }
    return slot;
}

__global__ void __launch_bounds__(kThreads) kv4_attention_kernel(const AttnArgs a) {
    __shared__ float qs[256], ps[kThreads], red[4];
    __shared__ int slots[kThreads];
    const int tid = threadIdx.x, h = blockIdx.x, t = blockIdx.y, s = blockIdx.z;
    const int g = h / (a.Hq / a.Hkv), per = a.D / kKv4Group;
    const int64_t row = (int64_t)s * a.Tq + t;
    for (int d = tid; d < a.D; d += kThreads) qs[d] = __bfloat162float(a.q[row * a.q_stride + (int64_t)h * a.D + d]);
    const int len = __ldg(a.lens + s);
    unsigned err = 0;
    if (len < 0 || len > a.max_len) err |= KVSEL_DEV_BAD_LENGTH;
    const int n = min(max(len, 0), a.max_len) - a.Tq + t + 1;  // tokens the row may see
    float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
    const float c = a.scale * kLog2e;
    __syncthreads();
    for (int j0 = 0; j0 < n; j0 += kThreads) {
        const int j = j0 + tid;
        const int slot = j < n ? slot_of(a, s, j, err) : -1;
        float x = -INFINITY;
        if (slot >= 0) {
            const int pg = slot / a.page;
            const int64_t r = ((int64_t)pg * a.Hkv + g) * a.page + (slot - pg * a.page);
            x = 0.f;
            for (int i = 0; i < per; ++i) {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.kc + (r * per + i) * 8));
                const float sc = kv4_scale(__ldg(a.ks + r * per + i));
                float dot = 0.f;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint32_t h2 = kv4_pair(((b < 4 ? w.x : w.y) >> (8 * (b & 3))) & 0xFFu);
                    dot = fmaf(__half2float(__ushort_as_half((uint16_t)h2)), qs[i * 16 + 2 * b], dot);
                    dot = fmaf(__half2float(__ushort_as_half((uint16_t)(h2 >> 16))), qs[i * 16 + 2 * b + 1], dot);
                }
                x = fmaf(dot, sc, x);
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
        ps[tid] = x == -INFINITY ? 0.f : exp2f(x - base);
        slots[tid] = slot;
        l *= corr, o[0] *= corr, o[1] *= corr;
        __syncthreads();
        for (int i = 0; i < min(kThreads, n - j0); ++i) {
            const int sl = slots[i];
            if (sl < 0) continue;
            const float p = ps[i];
            l += p;
            const int pg = sl / a.page;
            const int64_t r = ((int64_t)pg * a.Hkv + g) * a.page + (sl - pg * a.page);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = tid + k * kThreads;
                if (d >= a.D) break;
                const uint32_t h2 = kv4_pair(__ldg(a.vc + r * per * 8 + d / 2));
                const float v = __half2float(__ushort_as_half((uint16_t)(d & 1 ? h2 >> 16 : h2))) *
                                kv4_scale(__ldg(a.vs + r * per + d / kKv4Group));
                o[k] = fmaf(p, v, o[k]);
            }
        }
        __syncthreads();
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int k = 0; k < 2; ++k) {
        const int d = tid + k * kThreads;
        if (d < a.D) a.out[(row * a.Hq + h) * a.D + d] = __float2bfloat16_rn(o[k] * inv);
    }
    if (a.lse && tid == 0) a.lse[row * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    if (err) atomicOr(a.err, err);
}

}  // namespace

extern "C" int kvsel_kv4_attention(kvsel_ctx* ctx, const void* q, int64_t q_stride, int S, int Tq, int Hq, int Hkv, int D,
                                   const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                                   const uint8_t* v_scales, int P, int page, const int32_t* seq_lens,
                                   const int32_t* slot_map, const int32_t* block_table, int ld, int dead_slot,
                                   float scale, void* out, float* lse, void* stream) {
    const kvsel_trace trace_("kvsel_kv4_attention");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (S < 0 || Tq < 0 || Hq <= 0 || Hkv <= 0 || P < 0 || page <= 0 || ld < 0)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "kv4_attention: bad sizes");
    if (Hq % Hkv) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "kv4_attention: Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
    if (D != 64 && D != 128 && D != 256)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: D=%d unsupported", D);
    if (!slot_map == !block_table)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_attention: one of slot_map and block_table is needed");
    const int64_t reach = slot_map ? ld : (int64_t)ld * page;
    if ((int64_t)P * page > INT_MAX || reach > INT_MAX - 4096)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: slots and positions must fit 31 bits");
    if (S > 65535 || Tq > 1024 || Hq > 65535)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "kv4_attention: S, Tq or Hq too large");
    if (!(scale > 0.f) || scale > 1e30f)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_attention: scale must be positive and finite");
    if (S == 0 || Tq == 0) return KVSEL_OK;
    if (!q || !seq_lens || !out || (P > 0 && (!k_codes || !k_scales || !v_codes || !v_scales)))
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_attention: null pointer");
    if (q_stride < (int64_t)Hq * D) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "kv4_attention: token stride < Hq*D");
    auto off16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; };
    if (off16(q) || (q_stride * 2) % 16 || off16(out) || off16(k_codes) || off16(k_scales) || off16(v_codes) ||
        off16(v_scales))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "kv4_attention: q, its stride, out and the caches must be 16-byte aligned");
    const AttnArgs a{(const __nv_bfloat16*)q, q_stride, Tq, Hq, Hkv, D, k_codes, k_scales, v_codes, v_scales, P, page,
                     seq_lens, slot_map, block_table, ld, (int)reach, dead_slot, scale, (__nv_bfloat16*)out, lse,
                     ctx->dev_err};
    kv4_attention_kernel<<<dim3(Hq, Tq, S), kThreads, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_attention launch");
}
