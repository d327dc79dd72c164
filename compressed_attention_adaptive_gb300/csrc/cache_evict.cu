// Eviction from the 4-bit cache by the weight that tokens got (format and layout: cache.cuh).
//
// Each (sequence, cache head) that has more than keep tokens keeps its first, its last
// and, of the others, the K with the largest sums. The K-th largest is found by radix: counts of the
// sums' leading digits, then of the next digit among those that share the leading ones, and so on
// through 32 bits (sums as ordered integers); what is equal to the K-th is
// told apart by place, in the same way. Kept rows behind the new length then go to the freed places before
// it, i-th to i-th: what is read is behind the new length and what is written before it, so rows
// move in any order and at once.
//
// Work split. A row of sums is shared by a cluster of C blocks, each with its run of places: it holds their
// keys in shared memory (they are read from memory once, if they fit), counts digits there, and
// adds up the cluster's counts through distributed shared memory, one cluster barrier per
// digit. The same blocks then number the freed places and the rows that move, and move them.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "cache_walk.cuh"

namespace mita {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kDigit = 11, kBins = 1 << kDigit;  // 32 bits in digits of 11, 11 and 10
constexpr int kMaxKeys = 48 * 1024;              // keys that a block holds

// Larger sums have larger keys; NaN the largest.
__device__ __forceinline__ uint32_t sum_key(float x) { return x != x ? 0xffffffffu : order_key(x); }

struct Select {
    alignas(16) int hist[2][kBins];
    int scan[kWarps];
    int holes[kWarps], movers[kWarps];
    int all_holes, all_movers;  // of the block
    unsigned long long bound;
    int left, bin;
};

template <int C> __device__ __forceinline__ void cluster_sync() {
    if (C > 1)
        cg::this_cluster().sync();
    else
        __syncthreads();
}
template <int C, typename T> __device__ __forceinline__ const T* of_rank(const T* p, int rank) {
    if (C == 1) return p;
    return cg::this_cluster().map_shared_rank(const_cast<T*>(p), rank);
}

}  // namespace

template <int D, int C>
__global__ void __launch_bounds__(kThreads) k_cache_evict(CacheArgs a, EvictArgs e, uint8_t* __restrict__ cache, int room) {
    using L = Grp<D>;
    extern __shared__ __align__(16) uint32_t keys[];  // [room]
    __shared__ Select s;
    allow_next();
    const int rowi = blockIdx.x / C, rank = blockIdx.x - rowi * C;
    const int b = rowi / a.Hkv, h = rowi - b * a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = cache_len(a, b), keep = e.keep[b];
    if (a.len[b] != n || (long long)e.first + e.recent > keep) return;  // left as it is
    const long long row = (long long)rowi * e.cap;
    const float* acc = e.acc + row;
    // the block's places
    const int run = (int)(((long long)n + C - 1) / C + 3) & ~3, p0 = min(n, rank * run), p1 = min(n, p0 + run);
    if (n <= keep) {
        for (int j = p0 + threadIdx.x; j < p1; j += kThreads) {
            if (e.acc_out != e.acc) e.acc_out[row + j] = acc[j];
            if (e.src) e.src[row + j] = j;
        }
        return;
    }
    // those between: places [m0, m1), of which K stay, the ones with a rank of at least `bound`
    const int m0 = e.first, m1 = n - e.recent, K = keep - e.first - e.recent;
    const bool held = run <= room;
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[0][i] = 0;
    __syncthreads();
    auto first_digit = [&](int j, uint32_t key) {
        if (j >= m0 && j < m1) atomicAdd(&s.hist[0][key >> (32 - kDigit)], 1);
    };
    if (((uintptr_t)(acc + p0) & 15) == 0) {
        const int quads = (p1 - p0) / 4;
#pragma unroll 4
        for (int i = threadIdx.x; i < quads; i += kThreads) {
            const float4 v = reinterpret_cast<const float4*>(acc + p0)[i];
            const uint4 k = make_uint4(sum_key(v.x), sum_key(v.y), sum_key(v.z), sum_key(v.w));
            if (held) reinterpret_cast<uint4*>(keys)[i] = k;
            first_digit(p0 + 4 * i, k.x);
            first_digit(p0 + 4 * i + 1, k.y);
            first_digit(p0 + 4 * i + 2, k.z);
            first_digit(p0 + 4 * i + 3, k.w);
        }
        for (int j = p0 + 4 * quads + threadIdx.x; j < p1; j += kThreads) {
            const uint32_t k = sum_key(acc[j]);
            if (held) keys[j - p0] = k;
            first_digit(j, k);
        }
    } else {
#pragma unroll 8
        for (int j = p0 + threadIdx.x; j < p1; j += kThreads) {
            const uint32_t k = sum_key(acc[j]);
            if (held) keys[j - p0] = k;
            first_digit(j, k);
        }
    }
    // what a place is ranked by: its sum, then the lower place
    auto rank_of = [&](int j) {
        return (unsigned long long)(held ? keys[j - p0] : sum_key(acc[j])) << 32 | ~(uint32_t)j;
    };

    unsigned long long bound = 0;
    for (int left = K, bin = m1 - m0, shift = 64, at = 0; K > 0 && left < bin && shift > 0; at ^= 1) {
        const int top = shift;  // bits known
        shift = shift == 42 || shift == 10 ? shift - 10 : shift - 11;
        if (top < 64) {
            for (int j = max(p0, m0) + threadIdx.x; j < min(p1, m1); j += kThreads) {
                const unsigned long long r = rank_of(j);
                if (r >> top == bound >> top) atomicAdd(&s.hist[at][(r >> shift) & ((1u << (top - shift)) - 1)], 1);
            }
        }
        cluster_sync<C>();
        // the other counts are of the digit before, which the whole cluster has read
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[at ^ 1][i] = 0;
        // from the largest digit down, four a thread
        const int quad = kBins / 4 - 1 - threadIdx.x;
        int4 c = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const int4 x = reinterpret_cast<const int4*>(of_rank<C>(&s.hist[at][0], r))[quad];
            c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
        }
        const int four[4] = {c.w, c.z, c.y, c.x}, sum = c.x + c.y + c.z + c.w;
        int before = warp_scan(sum, lane);
        if (lane == 31) s.scan[warp] = before;
        before -= sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += s.scan[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (before < left && left <= before + four[i]) {
                s.bound = bound | (unsigned long long)(4 * quad + 3 - i) << shift;
                s.left = left - before;
                s.bin = four[i];
            }
            before += four[i];
        }
        __syncthreads();
        bound = s.bound;
        left = s.left;
        bin = s.bin;
    }
    if (held) __syncthreads();  // (K = 0: the keys)
    auto stays = [&](int j) { return j < m0 || j >= m1 || (K > 0 && rank_of(j) >= bound); };

    // Freed places before `keep` and kept rows from there on, numbered in order: a warp takes a run of
    // places, counts, and writes them behind what the warps and blocks before it have.
    const int wrun = ((p1 - p0 + kWarps - 1) / kWarps + 31) & ~31, j0 = p0 + warp * wrun;
    const long long half = (e.cap + 1) / 2;
    int* holes = e.moves + 2 * half * rowi;
    int* movers = holes + half;
    int nh = 0, nm = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int ch = nh, cm = nm;  // (pass 1) those before
        for (int i = 0; i < wrun && j0 + i < p1; i += 32) {
            const int j = j0 + i + lane;
            const bool in = j < p1, stay = in && stays(j);
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
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) {
                ch = nh;
                cm = nm;
            }
            nh += s.holes[w];
            nm += s.movers[w];
        }
        if (threadIdx.x == 0) {
            s.all_holes = nh;
            s.all_movers = nm;
        }
        nh = ch;
        nm = cm;
        cluster_sync<C>();
        for (int r = 0; r < rank; ++r) {
            nh += *of_rank<C>(&s.all_holes, r);
            nm += *of_rank<C>(&s.all_movers, r);
        }
    }
    // (as many of the one as of the other, and at most half of the places each; sums that change
    // under the call leave the results undefined, but no list is left)
    int ah = 0, am = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        ah += *of_rank<C>(&s.all_holes, r);
        am += *of_rank<C>(&s.all_movers, r);
    }
    const int moves = (int)min((long long)min(ah, am), half);
    cluster_sync<C>();  // the lists are there, acc has been read, and no block reads another's memory any more

    // A thread moves 16 channels of keys and values, as they are held, of two rows at a time.
    constexpr int NB = L::kBlocks, kAtOnce = 2, kStride = C * kThreads;
    const long long all = (long long)moves * NB;
    for (long long i0 = rank * kThreads + threadIdx.x; i0 < all; i0 += kAtOnce * kStride) {
        int to[kAtOnce], from[kAtOnce], gt[kAtOnce], gf[kAtOnce];
        uint2 k[kAtOnce], v[kAtOnce];
        uint8_t ks[kAtOnce], vs[kAtOnce];
        const int blk = (int)(i0 % NB);  // kStride is a multiple of NB
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const long long i = i0 + u * kStride;
            gt[u] = -1;
            if (i >= all) continue;
            to[u] = __ldcg(holes + i / NB);
            from[u] = __ldcg(movers + i / NB);
            gt[u] = cache_group(a, b, h, to[u] / kGroup);
            gf[u] = cache_group(a, b, h, from[u] / kGroup);
            if (blk == 0) {
                e.acc_out[row + to[u]] = acc[from[u]];
                if (e.src) e.src[row + to[u]] = from[u];
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (gt[u] < 0 || gf[u] < 0) {
                gt[u] = -1;
                continue;
            }
            const uint8_t* src = cache + (long long)gf[u] * L::kBytes;
            const int tok = from[u] % kGroup, vr = L::v_row(tok);
            k[u] = *reinterpret_cast<const uint2*>(src + L::k_code(tok, blk));
            ks[u] = src[L::k_scale(tok, blk)];
            if (D == 128) {  // a block is one chunk
                v[u] = *reinterpret_cast<const uint2*>(src + L::v_chunk(vr, blk));
            } else {  // or two
                v[u].x = *reinterpret_cast<const uint32_t*>(src + L::v_chunk(vr, 2 * blk));
                v[u].y = *reinterpret_cast<const uint32_t*>(src + L::v_chunk(vr, 2 * blk + 1));
            }
            vs[u] = src[L::v_scale(tok, blk)];
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (gt[u] < 0) continue;
            uint8_t* dst = cache + (long long)gt[u] * L::kBytes;
            const int tok = to[u] % kGroup, vr = L::v_row(tok);
            *reinterpret_cast<uint2*>(dst + L::k_code(tok, blk)) = k[u];
            dst[L::k_scale(tok, blk)] = ks[u];
            if (D == 128) {
                *reinterpret_cast<uint2*>(dst + L::v_chunk(vr, blk)) = v[u];
            } else {
                *reinterpret_cast<uint32_t*>(dst + L::v_chunk(vr, 2 * blk)) = v[u].x;
                *reinterpret_cast<uint32_t*>(dst + L::v_chunk(vr, 2 * blk + 1)) = v[u].y;
            }
            dst[L::v_scale(tok, blk)] = vs[u];
        }
    }
}

// The new lengths, which no block of the call reads any more, and the call's status word.
__global__ void __launch_bounds__(256) k_cache_evict_end(CacheArgs a, EvictArgs e) {
    bool bad = bad_call<true>(a);
    wait_previous();  // the others have read the lengths
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int n = a.len[b], keep = e.keep[b];
        const bool out = (long long)e.first + e.recent > keep;
        bad |= out;
        e.len_out[b] = out || n != cache_len(a, b) ? n : min(n, keep);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = bad ? kStBounds : kStOk;
}

template <int D, int C>
static cudaError_t evict_c(const CacheArgs& a, const EvictArgs& e, uint8_t* cache, cudaStream_t st) {
    const int room = (int)std::min<long long>(kMaxKeys, ((e.cap + C - 1) / C + 3) & ~3LL);
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = set_smem_once((const void*)k_cache_evict<D, C>, kMaxKeys * 4, &done);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(a.B * a.Hkv) * C);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = room * 4;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = C > 1;
    err = cudaLaunchKernelEx(&c, k_cache_evict<D, C>, a, e, cache, room);
    if (err != cudaSuccess) return err;
    count_launch();
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3(1);
    c.blockDim = dim3(256);
    c.dynamicSmemBytes = 0;
    c.numAttrs = 1;
    err = cudaLaunchKernelEx(&c, k_cache_evict_end, a, e);
    if (err == cudaSuccess) count_launch();
    return err;
}

template <int D> static cudaError_t evict_t(const CacheArgs& a, const EvictArgs& e, uint8_t* cache, cudaStream_t st) {
    // Blocks of a row: more while they have many places each and the GPU has room for them.
    const long long rows = (long long)a.B * a.Hkv;
    int c = 1;
    while (c < 8 && e.cap > 4096LL * c && rows * c < 4LL * num_sms()) c *= 2;
    return c == 1   ? evict_c<D, 1>(a, e, cache, st)
           : c == 2 ? evict_c<D, 2>(a, e, cache, st)
           : c == 4 ? evict_c<D, 4>(a, e, cache, st)
                    : evict_c<D, 8>(a, e, cache, st);
}

cudaError_t launch_cache_evict(const CacheArgs& a, const EvictArgs& e, int d, void* cache, cudaStream_t st) {
    prof_mark(st, "cache_evict");
    return d == 64 ? evict_t<64>(a, e, (uint8_t*)cache, st) : evict_t<128>(a, e, (uint8_t*)cache, st);
}

}  // namespace mita
