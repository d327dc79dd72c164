// Eviction from the 4-bit cache by the weight that tokens got (format and layout: cache.cuh).
//
// Each (sequence, cache head) that has more than keep tokens keeps its first, its last
// and, of the others, the K with the largest sums. The K-th largest is found by radix: counts of the
// sums' leading digits, then of the next digit among those that share the leading ones, and so on
// through 32 bits (sums as ordered integers); what is equal to the K-th is
// told apart by place, in the same way. Kept rows behind the new length then go to the freed places before
// it, i-th to i-th: what is read is behind the new length and what is written before it, so rows
// move in any order and at once.
#include <algorithm>

#include "cache.cuh"

namespace mita {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kDigit = 11, kBins = 1 << kDigit;  // 32 bits in digits of 11, 11 and 10

// Larger sums have larger keys; NaN the largest.
__device__ __forceinline__ uint32_t sum_key(float x) { return x != x ? 0xffffffffu : order_key(x); }

// What a place is ranked by: its sum, then the lower place.
__device__ __forceinline__ unsigned long long rank_of(float x, int j) {
    return (unsigned long long)sum_key(x) << 32 | ~(uint32_t)j;
}

struct Select {
    int hist[kBins];
    int scan[kWarps + 1];
    int holes[kWarps], movers[kWarps];
    unsigned long long bound;
    int left, bin;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads) k_cache_evict(CacheArgs a, EvictArgs e, uint8_t* __restrict__ cache) {
    using L = Grp<D>;
    __shared__ Select s;
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x - b * a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = cache_len(a, b), keep = e.keep[b];
    if (a.len[b] != n || (long long)e.first + e.recent > keep) return;  // left as it is
    const long long row = (long long)blockIdx.x * e.cap;
    const float* acc = e.acc + row;
    if (n <= keep) {
        for (int j = threadIdx.x; j < n; j += kThreads) {
            if (e.acc_out != e.acc) e.acc_out[row + j] = acc[j];
            if (e.src) e.src[row + j] = j;
        }
        return;
    }
    // those between: places [m0, m1), of which K stay, the ones with a rank of at least `bound`
    const int m0 = e.first, m1 = n - e.recent, K = keep - e.first - e.recent;
    unsigned long long bound = 0;
    for (int left = K, bin = m1 - m0, shift = 64; K > 0 && left < bin && shift > 0;) {
        const int top = shift;  // bits known
        shift = shift == 42 || shift == 10 ? shift - 10 : shift - 11;
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
        __syncthreads();
        for (int j = m0 + threadIdx.x; j < m1; j += kThreads) {
            const unsigned long long r = rank_of(acc[j], j);
            if (top == 64 || r >> top == bound >> top) atomicAdd(&s.hist[(r >> shift) & ((1u << (top - shift)) - 1)], 1);
        }
        __syncthreads();
        // from the largest digit down, four a thread
        int c[4], sum = 0, total;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = s.hist[kBins - 1 - (4 * threadIdx.x + i)];
            sum += c[i];
        }
        int before = block_excl_scan(sum, s.scan, &total);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (before < left && left <= before + c[i]) {
                s.bound = bound | (unsigned long long)(kBins - 1 - (4 * threadIdx.x + i)) << shift;
                s.left = left - before;
                s.bin = c[i];
            }
            before += c[i];
        }
        __syncthreads();
        bound = s.bound;
        left = s.left;
        bin = s.bin;
        __syncthreads();
    }
    auto stays = [&](int j) { return j < m0 || j >= m1 || (K > 0 && rank_of(acc[j], j) >= bound); };

    // Freed places before `keep` and kept rows from there on, numbered in order: a warp takes a run of
    // places, counts, and writes them behind what the warps before it have.
    const int run = ((n + kWarps - 1) / kWarps + 31) & ~31, j0 = warp * run, j1 = min(n, j0 + run);
    const long long half = (e.cap + 1) / 2;
    int* holes = e.moves + 2 * half * blockIdx.x;
    int* movers = holes + half;
    int nh = 0, nm = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int ch = nh, cm = nm;  // (pass 1) those of the warps before
        for (int j = j0 + lane; j < j0 + run && j - lane < j1; j += 32) {
            const bool in = j < j1, stay = in && stays(j);
            const uint32_t hb = __ballot_sync(0xffffffffu, in && j < keep && !stay);
            const uint32_t mb = __ballot_sync(0xffffffffu, in && j >= keep && stay);
            if (pass) {
                const uint32_t below = (1u << lane) - 1;
                const int ih = ch + __popc(hb & below), im = cm + __popc(mb & below);
                if ((hb >> lane & 1) && ih < half) holes[ih] = j;
                if ((mb >> lane & 1) && im < half) movers[im] = j;
                if (stay && j < keep) {
                    if (e.acc_out != e.acc) e.acc_out[row + j] = acc[j];
                    if (e.src) e.src[row + j] = j;
                }
            }
            ch += __popc(hb);
            cm += __popc(mb);
        }
        if (pass) break;
        if (lane == 0) {
            s.holes[warp] = ch;
            s.movers[warp] = cm;
        }
        __syncthreads();
        nh = nm = 0;
        for (int w = 0; w < warp; ++w) {
            nh += s.holes[w];
            nm += s.movers[w];
        }
    }
    // (as many of the one as of the other, and at most half of the places each; sums that change
    // under the call leave the results undefined, but no list is left)
    int ah = 0, am = 0;
    for (int w = 0; w < kWarps; ++w) {
        ah += s.holes[w];
        am += s.movers[w];
    }
    const int moves = (int)min((long long)min(ah, am), half);
    __syncthreads();  // the lists, and acc read

    // A thread moves 16 channels of keys and values, as they are held.
    constexpr int NB = L::kBlocks;
    for (long long i = threadIdx.x; i < (long long)moves * NB; i += kThreads) {
        const int r = (int)(i / NB), blk = (int)(i - (long long)r * NB), to = holes[r], from = movers[r];
        if (blk == 0) {
            e.acc_out[row + to] = acc[from];
            if (e.src) e.src[row + to] = from;
        }
        const int gt = cache_group(a, b, h, to / kGroup), gf = cache_group(a, b, h, from / kGroup);
        if (gt < 0 || gf < 0) continue;
        uint8_t* dst = cache + (long long)gt * L::kBytes;
        const uint8_t* src = cache + (long long)gf * L::kBytes;
        const int tt = to % kGroup, tf = from % kGroup, vt = L::v_row(tt), vf = L::v_row(tf);
        *reinterpret_cast<uint2*>(dst + L::k_code(tt, blk)) = *reinterpret_cast<const uint2*>(src + L::k_code(tf, blk));
        dst[L::k_scale(tt, blk)] = src[L::k_scale(tf, blk)];
#pragma unroll
        for (int x = 0; x < (D == 128 ? 1 : 2); ++x) {  // a block is one chunk, or two
            if (D == 128)
                *reinterpret_cast<uint2*>(dst + L::v_chunk(vt, blk)) = *reinterpret_cast<const uint2*>(src + L::v_chunk(vf, blk));
            else
                *reinterpret_cast<uint32_t*>(dst + L::v_chunk(vt, 2 * blk + x)) =
                    *reinterpret_cast<const uint32_t*>(src + L::v_chunk(vf, 2 * blk + x));
        }
        dst[L::v_scale(tt, blk)] = src[L::v_scale(tf, blk)];
    }
}

// The new lengths, which no block of the call reads any more, and the call's status word.
__global__ void __launch_bounds__(256) k_cache_evict_end(CacheArgs a, EvictArgs e) {
    bool bad = bad_call<true>(a);
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int n = a.len[b], keep = e.keep[b];
        const bool out = (long long)e.first + e.recent > keep;
        bad |= out;
        e.len_out[b] = out || n != cache_len(a, b) ? n : min(n, keep);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = bad ? kStBounds : kStOk;
}

cudaError_t launch_cache_evict(const CacheArgs& a, const EvictArgs& e, int d, void* cache, cudaStream_t st) {
    prof_mark(st, "cache_evict");
    const unsigned grid = (unsigned)(a.B * a.Hkv);
    if (d == 64)
        k_cache_evict<64><<<grid, kThreads, 0, st>>>(a, e, (uint8_t*)cache);
    else
        k_cache_evict<128><<<grid, kThreads, 0, st>>>(a, e, (uint8_t*)cache);
    k_cache_evict_end<<<1, 256, 0, st>>>(a, e);
    count_launch(2);
    return cudaGetLastError();
}

}  // namespace mita
