// The attention weight that each cached token gets from a call's rows (format and layout of
// the cache: cache.cuh):
//
//   acc'_j = decay acc_j + sum over rows r that see j of exp(scale q_r.k_j - lse_r)
//
// With the rows' log sums given there is no maximum to find and no sum over tokens: a token's sum needs
// its own key alone, so tokens can be cut anywhere and nothing is joined. It reads
// d/2 + d/16 + 4 bytes per token and cache head, writes 4, and does 2 d flops and an exponential
// per row.
//
// Work split. The groups of 16 tokens of all (sequence, cache head) form one line, cut into equal
// parts, one per warp; warps share nothing but the search for their place. A token's sum is
// added in an order of its own, whatever the cut, so the same call gives the same bits.
#include <algorithm>

#include "cache.cuh"
#include "tc.cuh"

namespace mita {

namespace {

constexpr int kThreads = 128;  // of a block
constexpr float kLog2e = 1.4426950408889634f;

struct WeighArgs {
    const float* lse;
    const float* acc;
    float* acc_out;
    float decay;
    long long cap;  // places of a sequence
};

// Where a warp is on the line. begin() is called by the whole block.
struct LineStart {
    unsigned long long before[kThreads], warps[kThreads / 32];
};
struct Place {
    int b, h, g, groups, n, count;  // sequence, cache head, group of it; the sequence's
    long long left;                 // groups of the warp's part from here on

    __device__ __forceinline__ void enter(const CacheArgs& a, int seq) {
        b = seq;
        n = cache_len(a, b);
        count = cache_count(a, b);
        groups = (n + kGroup - 1) / kGroup;
    }
    // The part of warp `me` of `all`. A thread sums up its share of the sequences.
    __device__ __forceinline__ void begin(const CacheArgs& a, LineStart& s, long long me, long long all) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int per = (a.B + kThreads - 1) / kThreads;
        unsigned long long mine = 0;
#pragma unroll 4
        for (int i = 0; i < per; ++i) {
            const int q = threadIdx.x * per + i;
            if (q < a.B) mine += (unsigned long long)((cache_len(a, q) + kGroup - 1) / kGroup) * a.Hkv;
        }
        unsigned long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s.warps[warp] = x;
        __syncthreads();
        unsigned long long total = 0, base = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp) base = total;
            total += s.warps[w];
        }
        s.before[threadIdx.x] = base + x - mine;
        __syncthreads();
        const unsigned long long q = total / all, r = total - q * all;
        const unsigned long long w0 = me * q + min((unsigned long long)me, r);
        left = (long long)(q + ((unsigned long long)me < r));
        b = a.B;
        if (left == 0) return;
        int slices = 0;  // threads whose share begins at or before w0
#pragma unroll
        for (int i = 0; i < kThreads; i += 32) slices += __popc(__ballot_sync(0xffffffffu, s.before[i + lane] <= w0));
        unsigned long long at = w0 - s.before[slices - 1];
        // (shares of threads without sequences begin at the total, which is above w0; a sequence without
        // tokens shares its beginning with the next)
        bool found = false;
        for (int seq = (slices - 1) * per; seq < a.B && !found; ++seq) {
            enter(a, seq);
            const unsigned long long units = (unsigned long long)groups * a.Hkv;
            found = at < units;
            if (!found) at -= units;
        }
        if (!found) {  // lengths that changed under the call
            left = 0;
            return;
        }
        h = (int)(at / groups);
        g = (int)(at - (unsigned long long)h * groups);
    }
    // Behind `step` groups of the same head.
    __device__ __forceinline__ bool next(const CacheArgs& a, int step) {
        left -= step;
        g += step;
        if (left <= 0) return false;
        if (g < groups) return true;
        g = 0;
        if (++h < a.Hkv) return true;
        h = 0;
        for (int seq = b + 1; seq < a.B; ++seq) {
            enter(a, seq);
            if (groups) return true;
        }
        return false;
    }
};

__device__ __forceinline__ int rows_of(const CacheArgs& a, int count) { return count * a.G; }
// Row r of a sequence: token r / G of the call, query head h G + r % G.
__device__ __forceinline__ long long row_offset(const CacheArgs& a, int b, int h, int r, int* t) {
    *t = r / a.G;
    return ((long long)(b * a.H + h * a.G + (r - *t * a.G)) * a.T + *t);
}
// Keys that token t of the call sees.
__device__ __forceinline__ int row_limit(const CacheArgs& a, int n, int count, int t) {
    return a.causal ? max(n - (count - 1 - t), 0) : n;
}
// exp(z - lse), at most 1, for a score z = dot f: one rounding of the difference, so that the weights that
// matter, whose scores are near lse, keep their bits. (Scores of 2^28 and more are further from
// a rounded lse than exponents reach; a sum that became infinite would stay so.) NaN stays NaN.
__device__ __forceinline__ float weight(float dot, float f, float lse) {
    float t = fmaf(dot, f, -lse);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(0.0f));
    return tc::ex2(t * kLog2e);
}

}  // namespace

// ------------------------------------------------------------ CUDA cores

// fp32 throughout: eight lanes share a token, each with the d/8 channels of two blocks' halves or of one
// block, and a warp takes four tokens at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_cache_weigh_simt(CacheArgs a, WeighArgs w, const T* __restrict__ Q, const uint8_t* __restrict__ cache) {
    using L = Grp<D>;
    constexpr int E = D / 8;  // channels of a lane
    __shared__ LineStart start;
    const int lane = threadIdx.x & 31, sub = lane >> 3, ch = lane & 7, blk = D == 128 ? ch : ch >> 1;
    Place at;
    at.begin(a, start, (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), (long long)gridDim.x * (kThreads / 32));
    if (at.left == 0) return;
    do {
        const int group = cache_group(a, at.b, at.h, at.g);
        if (group < 0) continue;
        const uint8_t* gr = cache + (long long)group * L::kBytes;
        const float f = a.scale * pow2(cache_exp(a, 0, at.h));
        float k[4][E], sum[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int tok = 4 * u + sub;
            sum[u] = 0.0f;
            const uint32_t sb = gr[L::k_scale(tok, blk)], s2 = e4m3x2_to_half2(sb | sb << 8);
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                uint32_t r[4];
                e2m1x8_to_half2(reinterpret_cast<const uint32_t*>(gr + tok * L::kRow)[ch * (E / 8) + i], r);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = half2_to_float2(hmul2(r[j], s2));
                    k[u][8 * i + 2 * j] = x.x;
                    k[u][8 * i + 2 * j + 1] = x.y;
                }
            }
        }
        const int rows = rows_of(a, at.count);
        for (int r = 0; r < rows; ++r) {
            int t;
            const long long row = row_offset(a, at.b, at.h, r, &t);
            const int lim = row_limit(a, at.n, at.count, t);
            if (lim <= at.g * kGroup) continue;
            float q[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = to_f(Q[row * D + ch * E + i]);
                q[i] = isfinite(x) ? x : __int_as_float(0x7fc00000);  // the row becomes NaN, as its softmax is
            }
            const float lse = w.lse[row];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) z = fmaf(q[i], k[u][i], z);
#pragma unroll
                for (int x = 4; x; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
                if (at.g * kGroup + 4 * u + sub < lim) sum[u] += weight(z, f, lse);
            }
        }
        const long long base = ((long long)at.b * a.Hkv + at.h) * w.cap;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = at.g * kGroup + 4 * u + sub;
            if (ch || j >= at.n) continue;
            if (w.decay != 0.0f && j < at.n - at.count) sum[u] = fmaf(w.decay, w.acc[base + j], sum[u]);
            w.acc_out[base + j] = sum[u];
        }
    } while (at.next(a, 1));
}

// Block behind the others' work: the call's status word.
__global__ void __launch_bounds__(256) k_cache_weigh_check(CacheArgs a) {
    const bool bad = __syncthreads_or(bad_call<true>(a));
    if (threadIdx.x == 0) *a.status = bad ? kStBounds : kStOk;
}

// ------------------------------------------------------------------ launch

template <typename T, int D>
static cudaError_t weigh_t(const CacheArgs& a, const WeighArgs& w, const void* Q, const uint8_t* cache, cudaStream_t st) {
    const long long groups = (long long)a.B * a.Hkv * ((w.cap + kGroup - 1) / kGroup);
    const int blocks = (int)std::min<long long>((groups + kThreads / 32 - 1) / (kThreads / 32), 8LL * num_sms());
    k_cache_weigh_simt<T, D><<<blocks, kThreads, 0, st>>>(a, w, (const T*)Q, cache);
    k_cache_weigh_check<<<1, 256, 0, st>>>(a);
    count_launch(2);
    return cudaGetLastError();
}

cudaError_t launch_cache_weigh(const CacheArgs& a, int d, int dtype, unsigned flags, const void* Q, const void* cache,
                               const float* lse, float decay, const float* acc, float* acc_out, cudaStream_t st) {
    const WeighArgs w{lse, acc, acc_out, decay, (long long)a.cols * a.page};
    const uint8_t* c = (const uint8_t*)cache;
    prof_mark(st, "cache_weights");
    if (dtype == 0) return d == 64 ? weigh_t<float, 64>(a, w, Q, c, st) : weigh_t<float, 128>(a, w, Q, c, st);
    return d == 64 ? weigh_t<__nv_bfloat16, 64>(a, w, Q, c, st) : weigh_t<__nv_bfloat16, 128>(a, w, Q, c, st);
}

}  // namespace mita
