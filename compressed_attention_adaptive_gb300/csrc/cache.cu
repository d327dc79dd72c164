// Writing rows into the 4-bit paged cache and reading them back (the format
// and the layout of a group are in cache.cuh).
//
// Both directions move 2 elem d + 2 (d/2 + d/16) bytes per token and head and
// do a handful of operations per element, so both are bound by HBM. A thread
// owns one block of 16 channels: its maximum, its scale and its codes need
// nothing from another thread.
#include <limits.h>

#include "cache.cuh"

namespace mita {

// The 16 elements of a block as fp32.
__device__ __forceinline__ void load16(const float* p, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void store16(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// y (16 values, already times 2^-e) -> 16 codes and the scale byte.
//
// s = RN_e4m3(amax / 6) and code = RN_e2m1(y / s), as if the quotients were
// exact: a correctly rounded fp32 quotient equals a midpoint of the target
// grid only if the exact one does. (A midpoint M has at most 5 significant
// bits and the divisor at most 4, so M times the divisor is a float; the next
// float is at least 2^-23 / f away relative to it, f in [1, 2) its
// significand, which is more than half a step of the quotient, 2^-24 / h, h in
// [1, 2) that of M. Below a power of two the float spacing halves, and so does
// the quotient's if M is one too; the divisors' significands leave no other
// case.)
__device__ __forceinline__ void quantise16(const float* y, uint32_t* codes, uint32_t* scale) {
    uint32_t amax = 0;  // as bits: NaN > infinity > every number
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(y[i]) & 0x7fffffffu);
    codes[0] = codes[1] = 0;
    if (amax > 0x7f800000u) {  // a NaN stays visible: the whole block reads as NaN
        *scale = 0x7f;
        return;
    }
    const float raw = __fdiv_rn(__uint_as_float(amax), 6.0f);
    uint16_t sb;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(raw));
    *scale = sb & 0xff;
    if ((sb & 0xff) == 0) return;
    const float s = half2_to_float2(e4m3x2_to_half2(sb)).x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t b;
        asm("{.reg .b8 t; .reg .b16 u; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; mov.b16 u, {t, 0}; cvt.u32.u16 %0, u;}"
            : "=r"(b)
            : "f"(__fdiv_rn(y[2 * i + 1], s)), "f"(__fdiv_rn(y[2 * i], s)));
        codes[i >> 2] |= b << (8 * (i & 3));
    }
}

// Place of a block: which group, and which bytes of it. Returns false for
// padding rows and for places outside the sequence or the pool.
struct BlockAt {
    int which, b, h, t, blk;
    long long row;  // of [B, Hkv, T]
};

template <int D>
__device__ __forceinline__ bool place(const CacheArgs& a, const BlockAt& x, long long* group, int* tok) {
    const int n = cache_len(a, x.b), c = cache_count(a, x.b);
    const int pos = n - c + x.t;
    if (x.t >= c || pos < 0) return false;
    const int g = cache_group(a, x.b, x.h, pos / kGroup);
    *group = g;
    *tok = pos % kGroup;
    return g >= 0;
}

// Thread i: block i % (d/16) of row i / (d/16); blockIdx.y: keys or values.
template <int D>
__device__ __forceinline__ bool block_at(const CacheArgs& a, BlockAt* x) {
    constexpr int NB = Grp<D>::kBlocks;
    const long long i = (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
    x->which = blockIdx.y;
    x->blk = (int)(i % NB);
    x->row = i / NB;
    if (x->row >= (long long)a.B * a.Hkv * a.T) return false;
    x->t = (int)(x->row % a.T);
    const int bh = (int)(x->row / a.T);
    x->b = bh / a.Hkv;
    x->h = bh - x->b * a.Hkv;
    return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(256) k_cache_write(CacheArgs a, const T* __restrict__ K, const T* __restrict__ V,
                                                     uint8_t* __restrict__ cache) {
    using L = Grp<D>;
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0) cache_check_call(a, true);
        return;
    }
    BlockAt x;
    long long group;
    int tok;
    if (!block_at<D>(a, &x) || !place<D>(a, x, &group, &tok)) return;
    float y[16];
    load16((x.which ? V : K) + x.row * D + x.blk * 16, y);
    const float up = pow2(-cache_exp(a, x.which, x.h));
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] *= up;
    uint32_t codes[2], scale;
    quantise16(y, codes, &scale);
    uint8_t* g = cache + group * L::kBytes;
    if (x.which == 0) {
        *reinterpret_cast<uint2*>(g + L::k_code(tok, x.blk)) = make_uint2(codes[0], codes[1]);
        g[L::k_scale(tok, x.blk)] = (uint8_t)scale;
    } else {
        // a block is one chunk for d = 128, two for d = 64
        const int row = L::v_row(tok);
        if (D == 128) {
            *reinterpret_cast<uint2*>(g + L::v_chunk(row, x.blk)) = make_uint2(codes[0], codes[1]);
        } else {
            *reinterpret_cast<uint32_t*>(g + L::v_chunk(row, 2 * x.blk)) = codes[0];
            *reinterpret_cast<uint32_t*>(g + L::v_chunk(row, 2 * x.blk + 1)) = codes[1];
        }
        g[L::v_scale(tok, x.blk)] = (uint8_t)scale;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) k_cache_read(CacheArgs a, const uint8_t* __restrict__ cache, T* __restrict__ K,
                                                    T* __restrict__ V) {
    using L = Grp<D>;
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0) cache_check_call(a, true);
        return;
    }
    BlockAt x;
    long long group;
    int tok;
    if (!block_at<D>(a, &x) || !place<D>(a, x, &group, &tok)) return;
    const uint8_t* g = cache + group * L::kBytes;
    uint32_t codes[2];
    uint32_t scale;
    if (x.which == 0) {
        const uint2 w = *reinterpret_cast<const uint2*>(g + L::k_code(tok, x.blk));
        codes[0] = w.x; codes[1] = w.y;
        scale = g[L::k_scale(tok, x.blk)];
    } else {
        const int row = L::v_row(tok);
        if (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2*>(g + L::v_chunk(row, x.blk));
            codes[0] = w.x; codes[1] = w.y;
        } else {
            codes[0] = *reinterpret_cast<const uint32_t*>(g + L::v_chunk(row, 2 * x.blk));
            codes[1] = *reinterpret_cast<const uint32_t*>(g + L::v_chunk(row, 2 * x.blk + 1));
        }
        scale = g[L::v_scale(tok, x.blk)];
    }
    const uint32_t s2 = e4m3x2_to_half2(scale | scale << 8);
    const float down = pow2(cache_exp(a, x.which, x.h));
    float y[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t r[4];
        e2m1x8_to_half2(codes[i], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = half2_to_float2(hmul2(r[j], s2));
            y[8 * i + 2 * j] = v.x * down;
            y[8 * i + 2 * j + 1] = v.y * down;
        }
    }
    store16((x.which ? V : K) + x.row * D + x.blk * 16, y);
}

template <typename T, int D>
static cudaError_t rows_t(const CacheArgs& a, bool write, void* K, void* V, uint8_t* cache, cudaStream_t st) {
    const long long blocks = (long long)a.B * a.Hkv * a.T * (D / 16);
    const dim3 grid((unsigned)((blocks + 255) / 256) + 1, 2);
    if (write)
        k_cache_write<T, D><<<grid, 256, 0, st>>>(a, (const T*)K, (const T*)V, cache);
    else
        k_cache_read<T, D><<<grid, 256, 0, st>>>(a, cache, (T*)K, (T*)V);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_cache_rows(const CacheArgs& a, int d, int dtype, bool write, void* K, void* V, void* cache,
                              cudaStream_t st) {
    prof_mark(st, write ? "cache_write" : "cache_read");
    uint8_t* c = (uint8_t*)cache;
    if (dtype == 0) return d == 64 ? rows_t<float, 64>(a, write, K, V, c, st) : rows_t<float, 128>(a, write, K, V, c, st);
    return d == 64 ? rows_t<__nv_bfloat16, 64>(a, write, K, V, c, st)
                   : rows_t<__nv_bfloat16, 128>(a, write, K, V, c, st);
}

}  // namespace mita
