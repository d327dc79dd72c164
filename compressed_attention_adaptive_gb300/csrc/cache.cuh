// The 4-bit paged key/value cache: sizes, the layout of a group of 16 tokens
// and the conversions between numbers and codes (cache.cu, cache_attn.cu).
//
// A cache is n_pages pages, each [Hkv][page / 16] groups of 16 tokens, so that
// a (page, head) is one run of bytes and a group is the unit that copies and
// tensor-core steps work in. A group of d channels takes 18 d bytes:
//
//   K codes   8 d   16 rows of d / 2 bytes, natural order
//   K scales    d   one byte per (token, block of 16 channels)
//   V codes   8 d   16 rows of d / 2 bytes, rows and chunks permuted
//   V scales    d
//
// The order inside a group is the order in which the lanes of a warp feed
// m16n8k16 tensor-core steps (cache_attn.cu). With g = lane / 4, t = lane % 4:
//   - lane (g, t) multiplies token 8 a + g (a = 0, 1) in channels
//     [t d/4, (t + 1) d/4), the same channels of Q being in the same lanes;
//     its scales for both a are adjacent;
//   - lane (g, t) weighs the values of tokens 8 a + 2 t + c (a, c = 0, 1), the
//     columns of its scores, in channels [g d/8, (g + 1) d/8). Row
//     t + 4 (2 a + c) holds token 8 a + 2 t + c, so that the four t read
//     neighbouring rows, and for d = 128 the upper two rows of each four have
//     their halves exchanged: without that two rows fall on the same shared
//     memory banks. A lane's four scales are one 32-bit word.
#pragma once

#include <cuda_fp16.h>
#include <limits.h>

#include "internal.h"

namespace mita {

constexpr int kGroup = 16;  // tokens per group, and channels per scale

template <int D> struct Grp {
    static constexpr int kRow = D / 2;            // bytes of one token's codes
    static constexpr int kBlocks = D / 16;        // scales per token
    static constexpr int kKs = 8 * D, kVc = 9 * D, kVs = 17 * D, kBytes = 18 * D;

    __host__ __device__ static constexpr int k_code(int tok, int blk) { return tok * kRow + blk * 8; }
    // lane (g, t) finds [a][block of its own] from g * kBlocks * 2 + t * kBlocks / 2
    __host__ __device__ static constexpr int k_scale(int tok, int blk) {
        constexpr int own = kBlocks / 4;  // blocks per lane
        return kKs + (tok & 7) * (2 * kBlocks) + (blk / own) * (2 * own) + (tok >> 3) * own + blk % own;
    }
    // row of a token: t + 4 (2 a + c)
    __host__ __device__ static constexpr int v_row(int tok) { return ((tok >> 1) & 3) + 4 * (2 * (tok >> 3) + (tok & 1)); }
    // byte of chunk g (d / 8 channels) of a row
    __host__ __device__ static constexpr int v_chunk(int row, int g) {
        return kVc + row * kRow + (D == 128 ? (g ^ ((row & 2) << 1)) : g) * (D / 16);
    }
    __host__ __device__ static constexpr int v_scale(int tok, int blk) {
        return kVs + blk * 16 + ((tok >> 1) & 3) * 4 + 2 * (tok >> 3) + (tok & 1);
    }
};

// A call's parameters and index arrays, passed to every kernel by value.
struct CacheArgs {
    int B, H, Hkv, T, G;
    int page, pgroups;      // tokens and groups per page
    int n_pages, cols;      // pages in the pool, columns of the page table
    int causal;
    int stall;       // fault test: a signal is left out
    float scale;
    const int *table, *len, *count, *exps;
    int* status;
    long long spin;  // cycles that a wait takes at most
};

constexpr int kMaxExp = 60;

// How the attention splits one call: rows of a tile, pieces of the line of
// chunks, and the rows of partial results that the workspace holds.
struct CachePlan {
    bool tensor;  // tensor cores, else CUDA cores
    bool tile;    // tcgen05 tiles (cache_tile.cu)
    bool fits;    // the attention's units of work can be counted in 32 bits
    int rows, pieces;
    size_t parts;
};

// Partial results of the attention, in the workspace.
struct CacheParts {
    float* part;  // [parts][d]
    float2* ml;   // [parts]
    int* found;   // [pieces]
};

// cache.cu
cudaError_t launch_cache_rows(const CacheArgs& a, int d, int dtype, bool write, void* K, void* V, void* cache,
                              cudaStream_t st);
// cache_weigh.cu
cudaError_t launch_cache_weigh(const CacheArgs& a, int d, int dtype, unsigned flags, const void* Q, const void* cache,
                               const float* lse, float decay, const float* acc, float* acc_out, cudaStream_t st);
// cache_evict.cu
struct EvictArgs {
    const int* keep;
    int first, recent;
    const float* acc;
    float* acc_out;  // may be acc
    int *src, *len_out;
    int* age;       // or null: recent tokens are the last places
    int* moves;     // [B * Hkv][2 half]: places that are freed, then places that move there
    long long cap;  // places of a sequence
};
cudaError_t launch_cache_evict(const CacheArgs& a, const EvictArgs& e, int d, void* cache, cudaStream_t st);
// cache_attn.cu
CachePlan cache_attn_plan(const CacheArgs& a, int d, int dtype, unsigned flags);
long long cache_spin(bool stall);
cudaError_t launch_cache_attn(const CacheArgs& a, const CachePlan& p, int d, int dtype, const void* Q,
                              const void* cache, void* O, float* lse, const CacheParts& parts, cudaStream_t st);

__host__ __device__ __forceinline__ int cache_len(const CacheArgs& a, int b) {
    return min(max(a.len[b], 0), a.cols * a.page);
}
__host__ __device__ __forceinline__ int cache_count(const CacheArgs& a, int b) {
    return a.count ? min(max(a.count[b], 0), a.T) : a.T;
}
__device__ __forceinline__ int cache_exp(const CacheArgs& a, int which, int h) {
    return a.exps ? min(max(a.exps[which * a.Hkv + h], -kMaxExp), kMaxExp) : 0;
}
// 2^e for |e| <= 126
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }

// Group number of sequence b's 16 tokens from 16 * gi on in head h, or -1 when
// the table names no page of the pool (the kernels record it).
__host__ __device__ __forceinline__ int cache_group(const CacheArgs& a, int b, int h, int gi) {
    const int col = gi / a.pgroups;
    const int pg = a.table[(long long)b * a.cols + col];
    if ((unsigned)pg >= (unsigned)a.n_pages) return -1;
    return (pg * a.Hkv + h) * a.pgroups + (gi - col * a.pgroups);
}

__device__ __forceinline__ bool bad_len(const CacheArgs& a, int b) {
    return a.len[b] != cache_len(a, b) || (a.count && a.count[b] != cache_count(a, b));
}
// Run by the threads of one block.
__device__ __forceinline__ bool bad_exps(const CacheArgs& a) {
    bool bad = false;
    if (a.exps)
        for (int i = threadIdx.x; i < 2 * a.Hkv; i += blockDim.x)
            bad |= (unsigned)a.exps[i] + kMaxExp > 2u * kMaxExp;
    return bad;
}

// Whether an index that a call uses is out of range, as far as the calling thread has looked;
// run by one whole block of at most 256 threads. One block can do it for all: a page's entry is 4 bytes, its
// rows at least 1152 bytes for each head. A thread takes a sequence, with its pages if they are
// few; the block takes the others' pages together. WHOLE: the call uses all places of a sequence, else its
// own rows, which then have to be among them.
template <bool WHOLE> __device__ __forceinline__ bool bad_call(const CacheArgs& a) {
    constexpr int kFewPages = 4;
    bool bad = bad_exps(a);
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        int first = 0, last = 0;
        if (b < a.B) {
            const int n = cache_len(a, b), c = WHOLE ? n : cache_count(a, b);
            bad |= bad_len(a, b) || c > n;
            if (c > 0) {
                first = max(n - c, 0) / a.page;
                last = (n + a.page - 1) / a.page;
            }
        }
        const bool few = last - first <= kFewPages;
        if (few)
            for (int i = first; i < last; ++i)
                bad |= (unsigned)a.table[(long long)b * a.cols + i] >= (unsigned)a.n_pages;
        if (!__syncthreads_or(!few)) continue;
        __shared__ int2 range[256];
        range[threadIdx.x] = few ? make_int2(0, 0) : make_int2(first, last);
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int s = threadIdx.x >> 5; s < blockDim.x && b0 + s < a.B; s += blockDim.x >> 5) {  // a warp a sequence
            const int* tb = a.table + (long long)(b0 + s) * a.cols;
#pragma unroll 8
            for (int i = range[s].x + lane; i < range[s].y; i += 32) bad |= (unsigned)tb[i] >= (unsigned)a.n_pages;
        }
        __syncthreads();
    }
    return bad;
}

// ------------------------------------------------------------- conversions

// Two scale bytes -> two halves (the lower byte first). Exact: e4m3's
// subnormals are normal halves.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    uint32_t r;
    asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(two));
    return r;
}

// Eight 4-bit codes -> four pairs of halves, pair i from byte i, the lower
// nibble first. Exact.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t* r) {
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// Product of a pair of codes and a pair of scales. Exact in halves: 2
// significant bits times 4, between 2^-10 and 2688.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace mita
