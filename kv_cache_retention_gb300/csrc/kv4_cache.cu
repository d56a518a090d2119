// kvsel_kv4_store and kvsel_kv4_load: rows of K and V written to the 4-bit paged
// cache and read back from it.
//
// A group of 16 values x becomes one scale s, the smallest of the format with
// max|x| <= 6 s, and 16 codes, the nearest E2M1 magnitudes to |x| / s with ties to
// the even code.  The codes are found by comparing |x| with the borders between
// magnitudes times s: those products are exact in fp32 (3 bits times 4), so the
// rounding is exact for fp32 rows too, where a quotient could land on a tie that the
// values are not on.
#include <cuda_bf16.h>
#include <limits.h>

#include "kv4_format.cuh"
#include "kvsel_internal.h"

namespace {

constexpr int kThreads = 256;

struct CacheArgs {
    const void* src[2];       // K, V rows (store)
    void* dst[2];             // K, V rows (load)
    int64_t stride[2];        // elements between tokens of the rows
    uint8_t* codes[2];
    uint8_t* scales[2];
    const int32_t* slots;
    int64_t n;                // groups of one of K, V: T * Hkv * D / 16
    int64_t n_slots;
    int Hkv, D, page;
    unsigned* err;
};

// Group g of the rows: its token, and where it lies in a row and in the cache.
struct Place {
    int64_t token, row, cache;  // row: element of the token's row; cache: group index
    bool real;
};
__device__ __forceinline__ Place place_of(const CacheArgs& a, int64_t g) {
    const int per = a.D / kKv4Group;
    const int64_t th = g / per;
    const int i = (int)(g - th * per);
    Place p;
    p.token = th / a.Hkv;
    const int h = (int)(th - p.token * a.Hkv);
    p.row = (int64_t)h * a.D + i * kKv4Group;
    const int slot = __ldg(a.slots + p.token);
    p.real = slot >= 0 && slot < a.n_slots;
    if (slot >= 0 && !p.real) atomicOr(a.err, (unsigned)KVSEL_DEV_BAD_SLOT);
    const int pg = slot / a.page;
    p.cache = (((int64_t)pg * a.Hkv + h) * a.page + (slot - pg * a.page)) * per + i;
    return p;
}

__device__ __forceinline__ void load16(const __nv_bfloat16* src, float (&x)[16]) {
    const uint4 w[2] = {__ldg(reinterpret_cast<const uint4*>(src)), __ldg(reinterpret_cast<const uint4*>(src) + 1)};
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load16(const float* src, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(src) + i);
        x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const CacheArgs a) {
    const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (g >= a.n) return;
    const Place p = place_of(a, g);
    if (!p.real) return;
    const int kv = blockIdx.y;
    float x[16];
    load16(static_cast<const T*>(a.src[kv]) + p.token * a.stride[kv] + p.row, x);
    float top = 0.f;
    bool broken = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        top = fmaxf(top, fabsf(x[i]));
        broken |= !(fabsf(x[i]) <= kKv4Max);  // NaN too
    }
    uint32_t byte = kKv4NanByte, w[2] = {0, 0};
    if (!broken) {
        byte = kv4_scale_byte(top);
        const float s = kv4_scale(byte);
        const float b0 = 0.25f * s, b1 = 0.75f * s, b2 = 1.25f * s, b3 = 1.75f * s, b4 = 2.5f * s, b5 = 3.5f * s,
                    b6 = 5.f * s;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float m = fabsf(x[i]);
            uint32_t c = (m > b0) + (m > b2) + (m > b4) + (m > b6);
            if (byte) c += (m >= b1) + (m >= b3) + (m >= b5);  // ties to the even code above
            c |= (__float_as_uint(x[i]) >> 28) & 8u;
            w[i >> 3] |= c << (4 * (i & 7));
        }
    }
    *reinterpret_cast<uint2*>(a.codes[kv] + p.cache * 8) = make_uint2(w[0], w[1]);
    a.scales[kv][p.cache] = (uint8_t)byte;
}

__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const CacheArgs a) {
    const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (g >= a.n) return;
    const Place p = place_of(a, g);
    const int kv = blockIdx.y;
    uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.real) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(a.codes[kv] + p.cache * 8));
        const float s = kv4_scale(__ldg(a.scales[kv] + p.cache));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h2 = kv4_pair(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu);
            const float lo = __half2float(__ushort_as_half((uint16_t)(h2 & 0xFFFFu))) * s;
            const float hi = __half2float(__ushort_as_half((uint16_t)(h2 >> 16))) * s;
            const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);  // exact
            o[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dst[kv]) + p.token * a.stride[kv] + p.row);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

bool misaligned(const void* p, int64_t stride_bytes) { return (reinterpret_cast<uintptr_t>(p) & 15u) || stride_bytes % 16; }

// The rules of kvsel_kv4_store and kvsel_kv4_load that they share.
int check(kvsel_ctx* ctx, const char* who, const void* k, const void* v, int64_t k_stride, int64_t v_stride, int esize,
          int T, int Hkv, int D, const int32_t* slots, const void* kc, const void* ks, const void* vc, const void* vs,
          int P, int page) {
    if (T < 0 || Hkv <= 0 || page <= 0 || P < 0) return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "%s: bad sizes", who);
    if (D != 64 && D != 128 && D != 256) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: D=%d unsupported", who, D);
    if ((int64_t)P * page > INT_MAX)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: P*page does not fit 31 bits", who);
    if (Hkv > 65535) return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: Hkv=%d unsupported", who, Hkv);
    if (T == 0) return KVSEL_OK;
    if (!k || !v || !slots) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "%s: null pointer", who);
    if (P > 0 && (!kc || !ks || !vc || !vs)) return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "%s: null cache", who);
    if (k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
        return kvsel_fail(ctx, KVSEL_ERR_SHAPE, "%s: token stride < Hkv*D", who);
    if (misaligned(k, k_stride * esize) || misaligned(v, v_stride * esize) || misaligned(kc, 0) || misaligned(ks, 0) ||
        misaligned(vc, 0) || misaligned(vs, 0))
        return kvsel_fail(ctx, KVSEL_ERR_ALIGN, "%s: rows, strides and caches must be 16-byte aligned", who);
    const int64_t groups = (int64_t)T * Hkv * (D / kKv4Group);
    if ((groups + kThreads - 1) / kThreads > INT_MAX)
        return kvsel_fail(ctx, KVSEL_ERR_UNSUPPORTED, "%s: too many rows", who);
    return KVSEL_OK;
}

}  // namespace

extern "C" int kvsel_kv4_store(kvsel_ctx* ctx, const void* k, const void* v, int src_dtype, int64_t k_stride,
                               int64_t v_stride, int T, int Hkv, int D, const int32_t* slots, uint8_t* k_codes,
                               uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, int P, int page, void* stream) {
    const kvsel_trace trace_("kvsel_kv4_store");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    if (src_dtype != KVSEL_F32 && src_dtype != KVSEL_BF16)
        return kvsel_fail(ctx, KVSEL_ERR_INVALID_ARG, "kv4_store: bad dtype");
    rc = check(ctx, "kv4_store", k, v, k_stride, v_stride, src_dtype == KVSEL_BF16 ? 2 : 4, T, Hkv, D, slots, k_codes,
               k_scales, v_codes, v_scales, P, page);
    if (rc || T == 0) return rc;
    const int64_t n = (int64_t)T * Hkv * (D / kKv4Group);
    const CacheArgs a{{k, v}, {nullptr, nullptr}, {k_stride, v_stride}, {k_codes, v_codes}, {k_scales, v_scales}, slots,
                      n, (int64_t)P * page, Hkv, D, page, ctx->dev_err};
    const dim3 grid((unsigned)((n + kThreads - 1) / kThreads), 2);
    if (src_dtype == KVSEL_BF16)
        kv4_store_kernel<__nv_bfloat16><<<grid, kThreads, 0, (cudaStream_t)stream>>>(a);
    else
        kv4_store_kernel<float><<<grid, kThreads, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_store launch");
}

extern "C" int kvsel_kv4_load(kvsel_ctx* ctx, const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                              const uint8_t* v_scales, int P, int page, const int32_t* slots, int T, int Hkv, int D,
                              void* k, void* v, int64_t k_stride, int64_t v_stride, void* stream) {
    const kvsel_trace trace_("kvsel_kv4_load");
    const kvsel_device_scope scope_;
    int rc = kvsel_enter(ctx);
    if (rc) return rc;
    rc = check(ctx, "kv4_load", k, v, k_stride, v_stride, 2, T, Hkv, D, slots, k_codes, k_scales, v_codes, v_scales, P,
               page);
    if (rc || T == 0) return rc;
    const int64_t n = (int64_t)T * Hkv * (D / kKv4Group);
    const CacheArgs a{{nullptr, nullptr}, {k, v}, {k_stride, v_stride},
                      {const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes)},
                      {const_cast<uint8_t*>(k_scales), const_cast<uint8_t*>(v_scales)}, slots,
                      n, (int64_t)P * page, Hkv, D, page, ctx->dev_err};
    const dim3 grid((unsigned)((n + kThreads - 1) / kThreads), 2);
    kv4_load_kernel<<<grid, kThreads, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_load launch");
}
