// tg_cache.cuh -- what the 8-bit cache's kernels share: the block scales, the
// conversions between codes and numbers, and the host's check of a cache.
#pragma once

#include <cuda_fp16.h>

#include "tg_host.cuh"

namespace tg {
namespace q8 {

constexpr int kBlock = TG_CACHE_BLOCK;

// A cache as the kernels see it (checked on the host).
struct Cache {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int32_t* lengths;
    float *s, *w;
    int64_t capacity, ld_token, ld_seq;
    int Hkv, batch;
    __device__ __forceinline__ int64_t blocks() const { return capacity / kBlock; }
};

// The length of sequence b within [0, capacity]; one outside is flagged.
__device__ __forceinline__ int length_of(const Cache& c, int b, unsigned int* status) {
    const int n = __ldg(c.lengths + b);
    if (n >= 0 && n <= c.capacity) return n;
    atomicOr(status, TG_STATUS_CACHE_LENGTH);
    return n < 0 ? 0 : static_cast<int>(c.capacity);
}

// The least 2^e, e >= -126, with amax <= qmax * 2^e, from the fp32 bits of amax
// = m 2^x: qmax = 448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6, so e is x - 8 or x - 6, one
// more where m exceeds qmax's own.  Whole arithmetic: no rounding, no tie.
template <int FMT>
__device__ __forceinline__ float scale_for(float amax) {
    const int bits = __float_as_int(amax);
    const int x = (bits >> 23) - 127, frac = bits & 0x7fffff;
    const int e = FMT == TG_CACHE_E4M3 ? x - 8 + (frac > 0x600000) : x - 6 + (frac > 0x7e0000);
    return __int_as_float((max(e, -126) + 127) << 23);
}

// Four numbers (already divided by the scale) to four codes, nearest even; e4m3
// saturates infinities and keeps NaN.  int8 takes finite values within 127.5 only.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (FMT == TG_CACHE_E4M3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    } else {
        // x + 1.5 * 2^23 holds round-half-even(x) in its low bits
        constexpr float kMagic = 12582912.0f;
        const uint32_t ab = __byte_perm(__float_as_uint(__fadd_rn(a, kMagic)), __float_as_uint(__fadd_rn(b, kMagic)),
                                        0x0040);
        const uint32_t cd = __byte_perm(__float_as_uint(__fadd_rn(c, kMagic)), __float_as_uint(__fadd_rn(d, kMagic)),
                                        0x0040);
        return __byte_perm(ab, cd, 0x5410);
    }
}

// Two codes (the low 16 bits of w, or the high ones) as two fp16 numbers, exactly: an
// e4m3 number has 4 significant bits and an exponent within fp16's; an int8 code c
// stands as 1024 + (c + 128) in fp16's last bits, less 1152.
template <int FMT, bool HIGH>
__device__ __forceinline__ uint32_t decode2(uint32_t w) {
    uint32_t r;
    if constexpr (FMT == TG_CACHE_E4M3) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(HIGH ? w >> 16 : w & 0xffffu)));
    } else {
        const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, HIGH ? 0x4342 : 0x4140);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
    }
    return r;
}

template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
    const uint32_t lo = decode2<FMT, false>(w), hi = decode2<FMT, true>(w);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

// Host: the cache's shape, pointers and strides.
inline tg_status check_cache(const tg_cache_q8* c, Cache* out) {
    if (!c) return TG_ERR_INVALID_ARG;
    if (c->format != TG_CACHE_E4M3 && c->format != TG_CACHE_INT8) return TG_ERR_INVALID_ARG;
    if (c->batch < 0 || c->capacity < 0 || c->Hkv <= 0) return TG_ERR_INVALID_ARG;
    if (c->d_h != 64 && c->d_h != 128) return TG_ERR_UNSUPPORTED;
    if (c->Hkv > 64 || c->batch > 65535 || c->capacity >= 0x7fff0000LL) return TG_ERR_UNSUPPORTED;
    if (c->capacity % kBlock) return TG_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(c->Hkv) * c->d_h;
    if (c->ld_token < row || (c->ld_token % 16) || (c->ld_seq % 16)) return TG_ERR_INVALID_ARG;
    // sequences may not overlap: the next one starts behind the last token's row
    if (c->batch > 1 && c->capacity > 0 && c->ld_seq < (c->capacity - 1) * c->ld_token + row) return TG_ERR_INVALID_ARG;
    if (c->batch > 0 && !c->lengths) return TG_ERR_INVALID_ARG;
    if (c->batch > 0 && c->capacity > 0 &&
        (!c->k || !c->v || !c->k_scale || !c->v_scale || !aligned16(c->k) || !aligned16(c->v)))
        return TG_ERR_INVALID_ARG;
    out->k = static_cast<uint8_t*>(c->k);
    out->v = static_cast<uint8_t*>(c->v);
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->lengths = c->lengths;
    out->s = c->s;
    out->w = c->w;
    out->capacity = c->capacity;
    out->ld_token = c->ld_token;
    out->ld_seq = c->ld_seq;
    out->Hkv = c->Hkv;
    out->batch = c->batch;
    return TG_OK;
}

// Whether [p, p + bytes) and [q, q + more) share memory.
inline bool overlap(const void* p, size_t bytes, const void* q, size_t more) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return p && q && x < y + more && y < x + bytes;
}

// Launch with programmatic dependent launch (every kernel calls pdl_wait() first).
template <typename... P, typename... A>
inline tg_status launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1] = {pdl_attr()};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? launch_status() : TG_ERR_CUDA;
}

}  // namespace q8
}  // namespace tg
