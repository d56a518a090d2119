// kvsel_kv4_store and kvsel_kv4_load: rows of K and V written to the 4-bit paged
// cache and read back from it.
//
// A group of 16 values x becomes one scale s, the smallest of the format with
// max|x| <= 6 s, and 16 codes, the nearest E2M1 magnitudes to |x| / s with ties to
// the even code.  The hardware conversion rounds the quotient so; what has to be
// exact is on which side of a border between two magnitudes the quotient lies:
//   q = x (1/s) and one correction by its remainder is the quotient rounded to
//   nearest, so a quotient that is a border is met exactly.  A bf16 quotient that is
//   none is at least 2^-9 of it away.
//   An fp32 quotient can round to a border that it is not: where q has a border's bit
//   pattern and the remainder x - q s, exact in one fma, is not zero, q is moved by
//   one unit to its side.
// Borders have 3 significant bits and scales 4, so border * s is a bf16 value too.
//
// Both kernels are bound by memory.  A thread takes one group at a time: its 32 or 64
// bytes of a row (in accesses of 32 where they lie on 32: with 16, which touch every
// sector twice, 38 us instead of 34 below), 8 bytes of codes, and one scale byte, of which
// four neighbours' are joined to one store.  A block takes whole tokens, so places come
// from 32-bit divisions of small numbers.  32768 tokens of 8 heads, D 128, bf16, are 172 MB
// a call, which takes 34 us: 5.1 TB/s, 75% of the rate of a plain copy.  Two groups' loads on
// their way together in each thread took 36 us, and quotients by division with codes found
// by seven comparisons a value 86 us.
#include <cuda_bf16.h>
#include <limits.h>

#include "kv4_format.cuh"
#include "kvsel_internal.h"

namespace {

constexpr int kThreads = 128;

struct CacheArgs {
    const void* src[2];       // K, V rows (store)
    void* dst[2];             // K, V rows (load)
    int64_t stride[2];        // elements between tokens of the rows
    uint8_t* codes[2];
    uint8_t* scales[2];
    const int32_t* slots;
    int T, Hkv, page, page_shift;  // page_shift: log2(page), or -1
    int n_slots;
    int per, per_shift;       // groups of a row: D / 16 = 1 << per_shift
    int groups;               // of a token: Hkv * per
    int tokens;               // of a block
    unsigned* err;
    bool wide[2];             // K, V rows lie on 32 bytes
};

// Group `local` of the block's tokens: its token, and where it lies in a row and in the cache.
struct Place {
    int token, row;           // row: element of the token's row
    int64_t cache;            // group of the cache
    bool in, real;            // a token of the call; with a slot of the cache
};
__device__ __forceinline__ Place place_of(const CacheArgs& a, unsigned local) {
    Place p;
    const unsigned t = local / (unsigned)a.groups, g = local - t * a.groups;
    const int64_t token = (int64_t)blockIdx.x * a.tokens + t;
    p.in = t < (unsigned)a.tokens && token < a.T;
    p.token = (int)token;
    const unsigned h = g >> a.per_shift, i = g & (a.per - 1);
    p.row = (int)g * kKv4Group;
    const int slot = p.in ? __ldg(a.slots + p.token) : -1;
    p.real = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots) atomicOr(a.err, (unsigned)KVSEL_DEV_BAD_SLOT);
    const int pg = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page;
    p.cache = ((((int64_t)pg * a.Hkv + h) * a.page + (slot - pg * a.page)) << a.per_shift) + i;
    return p;
}

// 32 bytes.  wide: they lie on 32, and one access takes them.
__device__ __forceinline__ void load32(const void* src, uint32_t (&u)[8], bool wide) {
    if (wide) {
        asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
            : "l"(src));
    } else {
        const uint4 a = __ldg(static_cast<const uint4*>(src)), b = __ldg(static_cast<const uint4*>(src) + 1);
        u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
    }
}
__device__ __forceinline__ void store32(void* dst, const uint32_t (&u)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]),
                     "r"(u[5]), "r"(u[6]), "r"(u[7]), "l"(dst)
                     : "memory");
    } else {
        static_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        static_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

// 16 values, and the largest magnitude (a NaN if there is one).
__device__ __forceinline__ float load16(const __nv_bfloat16* src, float (&x)[16], bool wide) {
    uint32_t u[8], top = 0;
    load32(src, u, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(u[i] & 0x7FFF7FFFu));
    }
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(__uint_as_float(top << 16)), "f"(__uint_as_float(top & 0xFFFF0000u)));
    return m;
}
__device__ __forceinline__ float load16(const float* src, float (&x)[16], bool wide) {
    float m = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t u[8];
        load32(src + 8 * h, u, wide);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[8 * h + i] = __uint_as_float(u[i]);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[8 * h + i])));
        }
    }
    return m;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const CacheArgs a) {
    const int kv = blockIdx.y;
    const unsigned total = (unsigned)a.tokens * a.groups;
    for (unsigned base = 0; base < total; base += kThreads) {
        const Place p = place_of(a, base + threadIdx.x);
        if (!__any_sync(0xffffffffu, p.real)) continue;
        float x[16], top = 0.f;
        uint32_t byte = kKv4NanByte, w[2] = {0, 0};
        if (p.real) top = load16(static_cast<const T*>(a.src[kv]) + (int64_t)p.token * a.stride[kv] + p.row, x, a.wide[kv]);
        if (p.real && top <= kKv4Max) {
            byte = kv4_scale_byte(top);
            const float s = kv4_scale(byte), r = byte ? 1.f / s : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float q = x[i] * r;
                q = fmaf(-fmaf(q, s, -x[i]), r, q);  // the signs as they are: a negative zero stays one
                if constexpr (sizeof(T) == 4) {
                    const float rest = fmaf(-q, s, x[i]);
                    const uint32_t b = __float_as_uint(q);
                    if (rest != 0.f && (b & 0xFFFFFu) == 0 && (b << 1))  // a border's pattern
                        q = __uint_as_float(b + (((int32_t)(__float_as_uint(rest) ^ b) >> 31) | 1));
                }
                x[i] = q;
            }
            w[0] = kv4_codes(x);
            w[1] = kv4_codes(x + 8);
        }
        // a row's groups are neighbours, a multiple of four: one store for four scale bytes
        uint32_t four = byte | __shfl_xor_sync(0xffffffffu, byte, 1) << 8;
        four |= __shfl_xor_sync(0xffffffffu, four, 2) << 16;
        if (p.real) {
            *reinterpret_cast<uint2*>(a.codes[kv] + p.cache * 8) = make_uint2(w[0], w[1]);
            if ((threadIdx.x & 3) == 0) *reinterpret_cast<uint32_t*>(a.scales[kv] + p.cache) = four;
        }
    }
}

__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const CacheArgs a) {
    const int kv = blockIdx.y;
    const unsigned total = (unsigned)a.tokens * a.groups;
    for (unsigned base = 0; base < total; base += kThreads) {
        const Place p = place_of(a, base + threadIdx.x);
        if (!p.in) continue;
        uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (p.real) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(a.codes[kv] + p.cache * 8));
            const uint32_t s = __ldg(a.scales[kv] + p.cache);
            const __half2 s2 = __half2half2(__ushort_as_half((uint16_t)(s << 7)));
            uint32_t h[8];
            kv4_pairs(c.x, *reinterpret_cast<uint32_t(*)[4]>(h));
            kv4_pairs(c.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // exact products, exact in bf16
                const float2 v = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(h + i), s2));
                const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
                o[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        store32(static_cast<__nv_bfloat16*>(a.dst[kv]) + (int64_t)p.token * a.stride[kv] + p.row, o, a.wide[kv]);
    }
}

// Fills in the sizes.  A block takes whole tokens, about four groups per thread; one where few blocks would be left (36
// tokens of 8 heads: 2.0 us a call with one, 2.6 with two; 32768 tokens: 40 us with one, 34 with four, 35 with eight).
CacheArgs sized(CacheArgs a, const kvsel_ctx* ctx, int esize, int T, int Hkv, int D, int P, int page) {
    a.T = T, a.Hkv = Hkv, a.page = page, a.n_slots = P * page, a.err = ctx->dev_err;
    a.page_shift = -1;
    if ((page & (page - 1)) == 0)
        for (a.page_shift = 0; (1 << a.page_shift) < page;) ++a.page_shift;
    a.per = D / kKv4Group;
    a.per_shift = D == 64 ? 2 : D == 128 ? 3 : 4;
    a.groups = Hkv * a.per;
    for (int i = 0; i < 2; ++i)
        a.wide[i] = ((reinterpret_cast<uintptr_t>(a.src[i] ? a.src[i] : a.dst[i]) | (uintptr_t)(a.stride[i] * esize)) & 31u) == 0;
    a.tokens = ((int64_t)T * a.groups > (int64_t)ctx->num_sms * 16 * kThreads ? 4 : 1) * kThreads / a.groups;
    if (a.tokens < 1) a.tokens = 1;
    return a;
}
dim3 grid_of(const CacheArgs& a) { return dim3((unsigned)(((int64_t)a.T + a.tokens - 1) / a.tokens), 2); }

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
    const CacheArgs a = sized({{k, v}, {nullptr, nullptr}, {k_stride, v_stride}, {k_codes, v_codes}, {k_scales, v_scales}, slots},
                              ctx, src_dtype == KVSEL_BF16 ? 2 : 4, T, Hkv, D, P, page);
    if (src_dtype == KVSEL_BF16)
        kv4_store_kernel<__nv_bfloat16><<<grid_of(a), kThreads, 0, (cudaStream_t)stream>>>(a);
    else
        kv4_store_kernel<float><<<grid_of(a), kThreads, 0, (cudaStream_t)stream>>>(a);
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
    const CacheArgs a = sized({{nullptr, nullptr}, {k, v}, {k_stride, v_stride},
                               {const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes)},
                               {const_cast<uint8_t*>(k_scales), const_cast<uint8_t*>(v_scales)}, slots},
                              ctx, 2, T, Hkv, D, P, page);
    kv4_load_kernel<<<grid_of(a), kThreads, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KVSEL_OK : kvsel_cuda_fail(ctx, e, "kv4_load launch");
}
