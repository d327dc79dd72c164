// Writing rows into the 4-bit paged cache and reading them back (the format
// and the layout of a group are in cache.cuh).
//
// Both directions move 2 elem d + 2 (d/2 + d/16) bytes per token and head and
// do a handful of operations per element, so both are bound by HBM. A thread
// owns one block of 16 channels of a row's keys and values: its maximum, its scale
// and its codes need nothing from another thread.
//
// Measured, calls back to back, two prompts of 32768, 16 heads, d = 128: bf16 (688 MB)
// written in 109 us (6.3 TB/s, 0.94 of the copy rate; issue slots 83 %) and read back in 106
// (0.97), float32 (1225 MB) in 199 (0.92) and 183 (1.00). One new
// token of 48 sequences: 3.2 us each, the latency of a length, a table entry and
// a row one after the other.
//   - A true division per element made writing 228 us (issue-bound), three operations instead of it
//     136, packed maxima and packing four code pairs at a time 108 (bf16; float32 divides).
//   - 32-byte accesses, and keys and values in one thread, took reading from 140 us to 106.
#include "cache.cuh"

namespace mita {

// 32 bytes at a time where the caller's tensor allows it (`wide`: 32-byte
// aligned), else 16.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t* r) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
        }
    }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t* r) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                     "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "l"(p)
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    }
}

// A block's 16 elements: as they are in memory, and as fp32.
template <typename T> struct Raw {
    static constexpr int kWords = 4 * sizeof(T);
    uint32_t r[kWords];
    __device__ __forceinline__ void load(const T* p, bool wide) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8) load32(reinterpret_cast<const uint32_t*>(p) + i, wide, r + i);
    }
    __device__ __forceinline__ void store(T* p, bool wide) const {
#pragma unroll
        for (int i = 0; i < kWords; i += 8) store32(reinterpret_cast<uint32_t*>(p) + i, wide, r + i);
    }
    __device__ __forceinline__ float get(int i) const {
        if (sizeof(T) == 4) return __uint_as_float(r[i % kWords]);
        return __uint_as_float(i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
    }
    __device__ __forceinline__ void set2(int i, float x, float y) {  // elements i (even) and i + 1
        if (sizeof(T) == 4) {
            r[i] = __float_as_uint(x);
            r[(i + 1) % kWords] = __float_as_uint(y);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            r[i >> 1] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};

// Largest magnitude of a block, NaN if it has one.
__device__ __forceinline__ float block_amax(const Raw<float>& x) {
    uint32_t m = 0;  // as bits: NaN > infinity > every number
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, x.r[i] & 0x7fffffffu);
    return __uint_as_float(m);
}
__device__ __forceinline__ float block_amax(const Raw<__nv_bfloat16>& x) {
    uint32_t m = x.r[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.r[i] & 0x7fff7fffu));
    uint16_t lo = (uint16_t)m, hi = (uint16_t)(m >> 16);
    asm("max.NaN.bf16 %0, %0, %1;" : "+h"(lo) : "h"(hi));
    return __uint_as_float((uint32_t)lo << 16);
}

// x * up / s for the code grid: up a power of two, s an e4m3 number, rs = up / s
// rounded. The rounding must not move a quotient onto or off a midpoint M of the
// grid {1/4, 3/4, 5/4, 7/4, 5/2, 7/2, 5}.
//   float32: the correctly rounded quotient. It equals M only if y = x up is M s: M s is a
//   float (3 and 4 significant bits), the next float is 2^-23 / f away relative to it, f in
//   [1, 2) its significand, and half a step of the quotient is 2^-24 / h, h in [1, 2) that
//   of M. (Below a power of two the spacing of floats halves; M s is one only where M is
//   one too, and then half a step of the quotient halves as well.)
//   bf16: y has 8 significant bits and M s has 7, so y is M s or at least 2^-8 of it
//   away. x rs is within 2^-24 of the quotient, relative: adding and subtracting
//   48 rounds it to a multiple of 2^-18, which is M itself in the first case and
//   on the quotient's side of M in the second. Two operations per element instead
//   of a division.
template <typename T> __device__ __forceinline__ float code_quotient(float x, float up, float s, float rs) {
    if (sizeof(T) == 4) return __fdiv_rn(x * up, s);
    return __fadd_rn(__fmaf_rn(x, rs, 48.0f), -48.0f);
}

// A block (times up = 2^-e) -> 16 codes and the scale byte, s = RN_e4m3(amax / 6),
// code = RN_e2m1(y / s). For s too the fp32 quotient is a midpoint of the grid
// (5 significant bits, the divisor 2) only if the exact one is.
template <typename T>
__device__ __forceinline__ void quantise16(const Raw<T>& x, float up, uint32_t* codes, uint32_t* scale) {
    const float amax = block_amax(x);
    codes[0] = codes[1] = 0;
    *scale = 0x7f;
    if (amax != amax) return;  // a NaN stays visible: the whole block reads as NaN
    const float raw = __fdiv_rn(amax * up, 6.0f);
    uint16_t sb;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(raw));
    *scale = sb & 0xff;
    if ((sb & 0xff) == 0) return;
    const float s = half2_to_float2(e4m3x2_to_half2(sb)).x, rs = __frcp_rn(s) * up;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = code_quotient<T>(x.get(8 * w + i), up, s, rs);
        asm("{.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};}"
            : "=r"(codes[w])
            : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    }
}

// Block blk of row `row` of [B, Hkv, T]: the thread has it for keys and values,
// which share the sequence's place. found() loads the lengths, group() the
// table, so that the rows can be loaded in between.
template <int D> struct BlockAt {
    int b, h, pos, blk;
    uint32_t row;

    // false: past the last row, padding, or before the sequence's first token
    __device__ __forceinline__ bool found(const CacheArgs& a) {
        constexpr int NB = Grp<D>::kBlocks;
        const long long i = (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
        blk = (int)(i % NB);
        const long long r = i / NB;
        if (r >= (long long)a.B * a.Hkv * a.T) return false;
        row = (uint32_t)r;  // B * H * T <= 2^30
        const uint32_t bh = row / (uint32_t)a.T;
        const int t = (int)(row - bh * a.T);
        b = (int)(bh / (uint32_t)a.Hkv);
        h = (int)(bh - (uint32_t)b * a.Hkv);
        const int n = cache_len(a, b), c = cache_count(a, b);
        pos = n - c + t;
        return t < c && pos >= 0;
    }
    __device__ __forceinline__ int group(const CacheArgs& a) const { return cache_group(a, b, h, pos / kGroup); }
    __device__ __forceinline__ int tok() const { return pos % kGroup; }
    __device__ __forceinline__ long long element() const { return (long long)row * D + blk * 16; }
};

// Run by one whole block of a call: checks every index that the call uses and stores the
// call's status word; the other blocks only leave out what is out of range.
__device__ __forceinline__ void check_call(const CacheArgs& a) {
    const bool bad = __syncthreads_or(bad_call<false>(a));
    if (threadIdx.x == 0) *a.status = bad ? kStBounds : kStOk;
}

template <typename T, int D>
__global__ void __launch_bounds__(256) k_cache_write(CacheArgs a, const T* __restrict__ K, const T* __restrict__ V,
                                                     uint8_t* __restrict__ cache, bool wide) {
    using L = Grp<D>;
    if (blockIdx.x == 0) {
        check_call(a);
        return;
    }
    BlockAt<D> x;
    if (!x.found(a)) return;
    Raw<T> k, v;
    k.load(K + x.element(), wide);
    v.load(V + x.element(), wide);
    const int group = x.group(a), ke = cache_exp(a, 0, x.h), ve = cache_exp(a, 1, x.h), tok = x.tok();
    if (group < 0) return;
    uint8_t* g = cache + (long long)group * L::kBytes;
    uint32_t codes[2], scale;
    quantise16(k, pow2(-ke), codes, &scale);
    *reinterpret_cast<uint2*>(g + L::k_code(tok, x.blk)) = make_uint2(codes[0], codes[1]);
    g[L::k_scale(tok, x.blk)] = (uint8_t)scale;
    quantise16(v, pow2(-ve), codes, &scale);
    const int row = L::v_row(tok);
    if (D == 128) {  // a block is one chunk
        *reinterpret_cast<uint2*>(g + L::v_chunk(row, x.blk)) = make_uint2(codes[0], codes[1]);
    } else {  // or two
        *reinterpret_cast<uint32_t*>(g + L::v_chunk(row, 2 * x.blk)) = codes[0];
        *reinterpret_cast<uint32_t*>(g + L::v_chunk(row, 2 * x.blk + 1)) = codes[1];
    }
    g[L::v_scale(tok, x.blk)] = (uint8_t)scale;
}

// 16 codes and their scale byte -> the block.
template <typename T>
__device__ __forceinline__ void widen16(const uint32_t* codes, uint32_t scale, float down, Raw<T>* x) {
    const uint32_t s2 = e4m3x2_to_half2(scale | scale << 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t r[4];
        e2m1x8_to_half2(codes[i], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 y = half2_to_float2(hmul2(r[j], s2));
            x->set2(8 * i + 2 * j, y.x * down, y.y * down);
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) k_cache_read(CacheArgs a, const uint8_t* __restrict__ cache, T* __restrict__ K,
                                                    T* __restrict__ V, bool wide) {
    using L = Grp<D>;
    if (blockIdx.x == 0) {
        check_call(a);
        return;
    }
    BlockAt<D> x;
    if (!x.found(a)) return;
    const int group = x.group(a), ke = cache_exp(a, 0, x.h), ve = cache_exp(a, 1, x.h), tok = x.tok();
    if (group < 0) return;
    const uint8_t* g = cache + (long long)group * L::kBytes;
    const int row = L::v_row(tok);
    const uint2 kc = *reinterpret_cast<const uint2*>(g + L::k_code(tok, x.blk));
    const uint32_t ks = g[L::k_scale(tok, x.blk)], vs = g[L::v_scale(tok, x.blk)];
    uint32_t codes[2];
    if (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(g + L::v_chunk(row, x.blk));
        codes[0] = w.x; codes[1] = w.y;
    } else {
        codes[0] = *reinterpret_cast<const uint32_t*>(g + L::v_chunk(row, 2 * x.blk));
        codes[1] = *reinterpret_cast<const uint32_t*>(g + L::v_chunk(row, 2 * x.blk + 1));
    }
    Raw<T> y;
    widen16(codes, vs, pow2(ve), &y);
    y.store(V + x.element(), wide);
    codes[0] = kc.x; codes[1] = kc.y;
    widen16(codes, ks, pow2(ke), &y);
    y.store(K + x.element(), wide);
}

template <typename T, int D>
static cudaError_t rows_t(const CacheArgs& a, bool write, void* K, void* V, uint8_t* cache, cudaStream_t st) {
    const long long blocks = (long long)a.B * a.Hkv * a.T * (D / 16);
    const unsigned grid = (unsigned)((blocks + 255) / 256) + 1;
    const bool wide = (((uintptr_t)K | (uintptr_t)V) & 31) == 0;
    if (write)
        k_cache_write<T, D><<<grid, 256, 0, st>>>(a, (const T*)K, (const T*)V, cache, wide);
    else
        k_cache_read<T, D><<<grid, 256, 0, st>>>(a, cache, (T*)K, (T*)V, wide);
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
