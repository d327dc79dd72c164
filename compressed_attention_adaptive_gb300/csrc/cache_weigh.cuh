// What the kernels that weigh cached tokens share (cache_weigh.cu, cache_weigh_tile.cu): the arguments, a
// worker's way along the tokens of all sequences, and a score's weight.
#pragma once

#include "cache_walk.cuh"

namespace mita {

struct WeighArgs {
    const float* lse;
    const float* acc;
    float* acc_out;
    float decay;
    long long cap;  // places of a sequence
};

// n / d; as 32-bit numbers where n is one.
__device__ __forceinline__ unsigned long long divide(unsigned long long n, unsigned d) {
    return n >> 32 ? n / d : (unsigned)n / d;
}

// Where a worker (a warp, or a block) is on the line of steps of TOK tokens. begin() is called by the whole
// block, of THREADS.
template <int THREADS> struct LineStart {
    unsigned long long before[THREADS], warps[THREADS / 32];
};
template <int TOK, int THREADS> struct Place {
    int b, h, at, steps, n, count;  // sequence, cache head, step of it; the sequence's
    long long left;                 // steps of the worker's part from here on

    __device__ __forceinline__ void enter(const CacheArgs& a, int seq) {
        b = seq;
        n = cache_len(a, b);
        count = cache_count(a, b);
        steps = (n + TOK - 1) / TOK;
    }
    // Steps of the sequences from `first` on, `per` of them.
    __device__ __forceinline__ static unsigned long long share(const CacheArgs& a, int first, int per) {
        unsigned long long sum = 0;
#pragma unroll 4
        for (int i = 0; i < per; ++i)
            if (first + i < a.B) sum += (unsigned long long)((cache_len(a, first + i) + TOK - 1) / TOK) * a.Hkv;
        return sum;
    }
    // The part of worker `me` of `all`. A thread sums up its share of the sequences: of a block's, or (WARPS), when they are
    // few, of each warp's for itself, without barriers (a call for one sequence of 1000 tokens takes 5.0 us with them, 4.7
    // without; the tiles' registers spill over the second way, and 55 us become 58).
    template <bool WARPS> __device__ __forceinline__ void begin(const CacheArgs& a, LineStart<THREADS>& s, long long me, long long all) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const bool few = WARPS && a.B <= 128;
        const int per = few ? (a.B + 31) / 32 : (a.B + THREADS - 1) / THREADS;
        const unsigned long long mine = share(a, (few ? lane : threadIdx.x) * per, per);
        unsigned long long x = mine, total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (few) {
            total = __shfl_sync(0xffffffffu, x, 31);
        } else {
            if (lane == 31) s.warps[warp] = x;
            __syncthreads();
            unsigned long long base = 0;
            total = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w == warp) base = total;
                total += s.warps[w];
            }
            s.before[threadIdx.x] = base + x - mine;
            __syncthreads();
        }
        const unsigned long long q = divide(total, (unsigned)all), r = total - q * all;
        const unsigned long long w0 = me * q + min((unsigned long long)me, r);
        left = (long long)(q + ((unsigned long long)me < r));
        b = a.B;
        if (left == 0) return;
        int slices = 0;  // threads whose share begins at or before w0
        unsigned long long off;
        if (few) {
            slices = __popc(__ballot_sync(0xffffffffu, x - mine <= w0));
            off = w0 - __shfl_sync(0xffffffffu, x - mine, slices - 1);
        } else {
#pragma unroll
            for (int i = 0; i < THREADS; i += 32) slices += __popc(__ballot_sync(0xffffffffu, s.before[i + lane] <= w0));
            off = w0 - s.before[slices - 1];
        }
        // (shares of threads without sequences begin at the total, which is above w0; a sequence without
        // tokens shares its beginning with the next)
        bool found = false;
        for (int seq = (slices - 1) * per; seq < a.B && !found; ++seq) {
            enter(a, seq);
            const unsigned long long units = (unsigned long long)steps * a.Hkv;
            found = off < units;
            if (!found) off -= units;
        }
        if (!found) {  // lengths that changed under the call
            left = 0;
            return;
        }
        h = (int)divide(off, (unsigned)steps);
        at = (int)(off - (unsigned long long)h * steps);
    }
    // Behind `done` steps of the same head.
    __device__ __forceinline__ bool next(const CacheArgs& a, int done) {
        left -= done;
        at += done;
        if (left <= 0) return false;
        if (at < steps) return true;
        at = 0;
        if (++h < a.Hkv) return true;
        h = 0;
        for (int seq = b + 1; seq < a.B; ++seq) {
            enter(a, seq);
            if (steps) return true;
        }
        return false;
    }
};

// exp(z - lse), at most 1, for a score z = dot f: one rounding of the difference, so that the weights that
// matter, whose scores are near lse, keep their bits. (Scores of 2^28 and more are further from
// a rounded lse than exponents reach; a sum that became infinite would stay so.) NaN stays NaN.
__device__ __forceinline__ float weight(float dot, float f, float lse) {
    float t = fmaf(dot, f, -lse);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(0.0f));
    return tc::ex2(t * kLog2e);
}

// Two at a time (the packed forms take one issue slot).
__device__ __forceinline__ uint64_t pack2(float2 x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(x)), "l"(pack2(y)));
    return unpack2(r);
}
__device__ __forceinline__ float2 weight2(float2 dot, float2 f, float2 minus_lse) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(dot)), "l"(pack2(f)), "l"(pack2(minus_lse)));
    float2 t = unpack2(r);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(t.x) : "f"(0.0f));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(t.y) : "f"(0.0f));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(t)), "l"(pack2(make_float2(kLog2e, kLog2e))));
    t = unpack2(r);
    return make_float2(tc::ex2(t.x), tc::ex2(t.y));
}

template <int N> __device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

// cache_weigh_tile.cu
cudaError_t launch_cache_weigh_tile(const CacheArgs& a, const WeighArgs& w, int d, int dtype, const void* Q,
                                    const uint8_t* cache, cudaStream_t st);

}  // namespace mita
