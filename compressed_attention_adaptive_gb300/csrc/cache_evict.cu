// Eviction from the 4-bit cache by the weight that tokens got (format and layout: cache.cuh).
//
// Each (sequence, cache head) that has more than keep tokens keeps its first, its last
// and, of the others, the K with the largest sums. The K-th largest is found by radix: counts of the
// sums' leading digits, then of the next digit among those that share the leading ones, and so on
// through 32 bits (sums as ordered integers); what is equal to the K-th is told apart by place, in the
// same way. Once few share the digits so far they are compared with each other. Kept rows behind the new
// length then go to the freed places before it, i-th to i-th: what is read is behind the new length and
// what is written before it, so rows move in any order and at once.
//
// Moves put places out of the order of age, so from a sequence's second eviction on its newest tokens are not its last places.
// AGED: age[j] is how much older the token at place j is than its place says (an unmoved token at place j - age[j]
// would be as old; negative: younger). The newest have the largest key of all, the rest is the same. A token
// that stays has come n - keep places nearer to the sequence's beginning; one that moves takes its place's age along; places from
// keep on hold 0 again, for the tokens that will be appended there.
//
// Work split. A row of sums is shared by a cluster of C blocks, each with its run of places: it holds their
// keys in shared memory (they are read from memory once, if they fit), counts digits there, and
// adds up the cluster's counts through distributed shared memory, one cluster barrier per
// digit. The same blocks then number the freed places and the rows that move, and move them.
//
// What it reads and writes is 4 bytes a sum, and a row that moves 2 x 288 bytes in sectors of 32 (144 held), which for long
// rows is a fifth of the time; what bounds it is the chain of steps. 32 rows of 32768, of a block's 40,000 to 42,500 clocks: loads
// and the first digit's counts 4500 to 5600; four cluster barriers, 1200 to 1800 each, the last up to 3600; the digit
// 1700; the last few gathered and compared 6700; what moves counted 2300 and listed 4500; rows that stay 1500; moves 10,000 to
// 12,000.
// Measured, in a graph: 128 rows of 2112 cut to 2048 11.0 us, 144 of 700 to 9001 cut to 1500 22.7, 32 of 32768 cut
// to 4096 25.1. A thread for each block of a row that moves, which looked its places up itself: 13.2, 26.4 and 31.0.
// With ages, 4 more bytes read and written a place, calls back to back on warm caches take 11.3, 23.0 and 26.8 us for these where
// calls without take 8.9, 19.9 and 22.0.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "cache_walk.cuh"

namespace mita {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kDigit = 11, kBins = 1 << kDigit;  // 32 bits in digits of 11, 11 and 10
constexpr int kCoarse = kBins / 32;              // runs of 32 counts
constexpr int kMaxKeys = 48 * 1024;              // keys that a block holds
constexpr int kList = 1024;                      // freed places and rows that move whose list is in shared memory
constexpr int kCompared = 256;                        // keys that are compared with each other
// The first digit is not the leading bits, which hold a sign and exponents that weights do not come near: 32 steps for each power of
// two from 2^-40 to 2^24, and one for all that is below or above. (If it is one of those, leading bits after all.)
constexpr int kFirstShift = 18, kFirstLow = (int)((0x80000000u | 87u << 23) >> kFirstShift);

__device__ __forceinline__ uint32_t first_digit(uint32_t key) {
    return (uint32_t)min(max((int)(key >> kFirstShift) - kFirstLow, 0), kBins - 1);
}

// Larger sums have larger keys; NaN the largest.
__device__ __forceinline__ uint32_t sum_key(float x) { return x != x ? 0xffffffffu : order_key(x); }
// AGED: the newest tokens' key, above all of these (order_key's largest number is infinity's, 0xff800000).
constexpr uint32_t kNewest = 0xffffffffu;
// Ages stop here: a token that far back is old for every window, which a sequence of 2^30 places is at most.
constexpr long long kMaxAge = 1 << 30;

struct Select {
    alignas(16) int hist[2][kBins];
    int coarse[2][kCoarse];
    int events[kWarps], all;  // freed places and rows that move: of a warp's run, of the block's
    int list[kList];
    unsigned long long few[kCompared], all_few[kCompared];  // ranks of the block's, and of all
    int found;
    unsigned long long bound;
    int digit, left, bin;
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

// Counts digits; equal ones in a row (sums of zero are often many) at once.
struct Counter {
    int* hist;
    uint32_t digit = 0;
    int n = 0;
    __device__ __forceinline__ explicit Counter(int* h) : hist(h) {}
    __device__ __forceinline__ void add(uint32_t d) {
        if (n && d != digit) {
            atomicAdd(hist + digit, n);
            n = 0;
        }
        digit = d;
        ++n;
    }
    __device__ __forceinline__ void end() {
        if (n) atomicAdd(hist + digit, n);
    }
};

// The lane, and what is before it, at which a running count over the warp's lanes reaches `left`.
__device__ __forceinline__ int reach(int count, int left, int lane, int* before) {
    const int incl = warp_scan(count, lane);
    const int at = __ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1;
    *before = __shfl_sync(0xffffffffu, incl - count, max(at, 0));
    return max(at, 0);
}

}  // namespace

template <int D, int C, bool AGED>
__global__ void __launch_bounds__(kThreads, 2) k_cache_evict(CacheArgs a, EvictArgs e, uint8_t* __restrict__ cache, int room) {
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
    const int m0 = e.first, m1 = AGED ? n : n - e.recent, K = keep - e.first - (AGED ? 0 : e.recent);
    int* age = AGED ? e.age + row : nullptr;
    // The key of place j, whose token's sum is x.
    auto key_of = [&](int j, float x, int a) {
        const uint32_t key = sum_key(x);
        return !AGED ? key : a <= j - (n - e.recent) ? kNewest : min(key, kNewest - 1);
    };
    // A token's age after the call, at place `to`.
    auto aged = [&](int to, int from, int a) {
        return (int)min(max((long long)to - from + a + (n - keep), -kMaxAge), kMaxAge);
    };
    const bool held = run <= room;
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[0][i] = 0;
    if (threadIdx.x == 0) s.found = 0;
    __syncthreads();
    const int places = p1 - p0;
    const bool wide = (((uintptr_t)(acc + p0) | (uintptr_t)(AGED ? age + p0 : nullptr)) & 15) == 0;
    // the keys of places p0 + x to p0 + x + 3 (x a multiple of four; 0 behind the block's places)
    auto load4 = [&](int x) {
        float4 v = make_float4(0, 0, 0, 0);
        int4 a = make_int4(0, 0, 0, 0);
        if (wide && x + 3 < places) {
            v = *reinterpret_cast<const float4*>(acc + p0 + x);
            if (AGED) a = *reinterpret_cast<const int4*>(age + p0 + x);
        } else {
            if (x < places) v.x = acc[p0 + x];
            if (x + 1 < places) v.y = acc[p0 + x + 1];
            if (x + 2 < places) v.z = acc[p0 + x + 2];
            if (x + 3 < places) v.w = acc[p0 + x + 3];
            if (AGED) {
                if (x < places) a.x = age[p0 + x];
                if (x + 1 < places) a.y = age[p0 + x + 1];
                if (x + 2 < places) a.z = age[p0 + x + 2];
                if (x + 3 < places) a.w = age[p0 + x + 3];
            }
        }
        const int j = p0 + x;
        return make_uint4(key_of(j, v.x, a.x), key_of(j + 1, v.y, a.y), key_of(j + 2, v.z, a.z), key_of(j + 3, v.w, a.w));
    };
    auto keys4 = [&](int x) { return held ? *reinterpret_cast<const uint4*>(keys + x) : load4(x); };
    {
        Counter count(s.hist[0]);
#pragma unroll 4
        for (int x = 4 * threadIdx.x; x < places; x += 4 * kThreads) {
            const uint4 k = load4(x);
            if (held) *reinterpret_cast<uint4*>(keys + x) = k;  // (room is a multiple of four)
            const uint32_t four[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p0 + x + i >= m0 && p0 + x + i < min(m1, p1)) count.add(first_digit(four[i]));
        }
        count.end();
    }
    // what a place is ranked by: its sum, then the lower place
    auto rank_of = [](int j, uint32_t key) { return (unsigned long long)key << 32 | ~(uint32_t)j; };

    unsigned long long bound = 0;
    int left = K, bin = m1 - m0, top = 64;  // of the `bin` places with the bits of bound from `top` on, `left` stay
    // Calls f(place, key) for those of the block's.
    auto sharing = [&](auto f) {
        const uint32_t high = (uint32_t)(bound >> 32), low = (uint32_t)bound;
        for (int x = 4 * threadIdx.x; x < places; x += 4 * kThreads) {
            const uint4 k = keys4(x);
            const uint32_t four[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = p0 + x + i;
                if (j < m0 || j >= min(m1, p1)) continue;
                const bool in = top > 32 ? top == 64 || (four[i] ^ high) >> (top - 32) == 0
                                         : four[i] == high && (top == 32 || (~(uint32_t)j ^ low) >> top == 0);
                if (in) f(j, four[i]);
            }
        }
    };
    bool first = true;
    for (int at = 0; K > 0 && left < bin && top > 0; at ^= 1) {
        if (bin <= kCompared) {
            sharing([&](int j, uint32_t key) {
                const int i = atomicAdd(&s.found, 1);
                if (i < kCompared) s.few[i] = rank_of(j, key);
            });
            cluster_sync<C>();
            int total = 0, from = 0, i = threadIdx.x;
            int of[C];
#pragma unroll
            for (int r = 0; r < C; ++r) of[r] = min(*of_rank<C>(&s.found, r), kCompared);
#pragma unroll
            for (int r = 0; r < C; ++r) {
                if (total <= (int)threadIdx.x) {
                    from = r;
                    i = (int)threadIdx.x - total;
                }
                total += of[r];
            }
            total = min(total, kCompared);
            if ((int)threadIdx.x < total) s.all_few[threadIdx.x] = of_rank<C>(&s.few[0], from)[i];
            __syncthreads();
            if ((int)threadIdx.x < total) {
                const unsigned long long mine = s.all_few[threadIdx.x];
                int above = 0;
#pragma unroll 4
                for (int i = 0; i < total; ++i) above += s.all_few[i] > mine;
                if (above == left - 1) s.bound = mine;
            }
            __syncthreads();
            bound = s.bound;
            break;
        }
        const int next = first ? 32 + kFirstShift : max(top - kDigit, top > 32 ? 32 : 0);
        if (!first) {
            Counter count(s.hist[at]);
            const uint32_t mask = (1u << (top - next)) - 1;
            sharing([&](int j, uint32_t key) { count.add((uint32_t)(rank_of(j, key) >> next) & mask); });
            count.end();
        }
        __syncthreads();
        {
            const int4 x = reinterpret_cast<const int4*>(s.hist[at])[threadIdx.x];
            int sum = x.x + x.y + x.z + x.w;
#pragma unroll
            for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if ((lane & 7) == 0) s.coarse[at][threadIdx.x >> 3] = sum;
        }
        cluster_sync<C>();
        // the other counts are of the digit before, which the whole cluster has read
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[at ^ 1][i] = 0;
        // One warp finds the digit, from the largest down: two runs of 32 a lane, then one run.
        if (warp == 0) {
            int hi = 0, lo = 0, before, then;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const int2 x = reinterpret_cast<const int2*>(of_rank<C>(&s.coarse[at][0], r))[kCoarse / 2 - 1 - lane];
                hi += x.y;
                lo += x.x;
            }
            int l = reach(hi + lo, left, lane, &before);
            const int top_run = __shfl_sync(0xffffffffu, hi, l);
            const bool lower = left > before + top_run;
            const int run32 = kCoarse - 1 - 2 * l - lower;
            if (lower) before += top_run;
            int fine = 0;
#pragma unroll
            for (int r = 0; r < C; ++r) fine += of_rank<C>(&s.hist[at][0], r)[32 * run32 + 31 - lane];
            l = reach(fine, left - before, lane, &then);
            fine = __shfl_sync(0xffffffffu, fine, l);
            if (lane == 0) {
                s.digit = 32 * run32 + 31 - l;
                s.left = left - before - then;
                s.bin = fine;
            }
        }
        __syncthreads();
        const int digit = s.digit;
        if (!first || (digit > 0 && digit < kBins - 1)) {
            bound |= (unsigned long long)(first ? digit + kFirstLow : digit) << next;
            left = s.left;
            bin = s.bin;
            top = next;
        }
        first = false;
    }
    if (held) __syncthreads();  // (K = 0: the keys)
    const uint32_t bound_key = (uint32_t)(bound >> 32), bound_at = ~(uint32_t)bound;  // the last place with that sum that stays
    auto stays = [&](int j, uint32_t key) {
        return j < m0 || j >= m1 || (K > 0 && (key > bound_key || (key == bound_key && (uint32_t)j <= bound_at)));
    };

    // Freed places before `keep` and kept rows from there on, numbered in order: there are as many of the one as of the
    // other, so the first half of a list of both has the places and the second the rows. A warp takes a run of
    // places, counts, and writes them behind what the warps and blocks before it have.
    const int wrun = ((places + kWarps - 1) / kWarps + 127) & ~127, x0 = warp * wrun, x1 = min(places, x0 + wrun);
    const long long half = (e.cap + 1) / 2;
    int* list = e.moves + 2 * half * rowi;  // (few moves of one block: in shared memory)
    int cap_list = (int)min(2 * half, (long long)INT_MAX);
    // Which of the four places from p0 + x + 4 lane on are such.
    auto events = [&](int x) {
        const int at = x + 4 * lane, j = p0 + at;
        uint32_t bits = 0;
        if (at < places) {
            const uint4 k = keys4(at);
            const uint32_t four[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (stays(j + i, four[i]) == (j + i >= keep) && j + i < p1) bits |= 1u << i;
        }
        return bits;
    };
    int mine = 0;
    for (int x = x0; x < x1; x += 128) mine += __popc(events(x));
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) s.events[warp] = mine;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s.events[w];
        all += s.events[w];
    }
    if (threadIdx.x == 0) s.all = all;
    if (C == 1 && all <= kList) {
        list = s.list;
        cap_list = kList;
    }
    cluster_sync<C>();
    all = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const int x = *of_rank<C>(&s.all, r);
        all += x;
        if (r < rank) before += x;
    }
    for (int x = x0; x < x1; x += 128) {
        const uint32_t bits = events(x), below = (1u << lane) - 1, count = __popc(bits);
        const uint32_t b0 = __ballot_sync(0xffffffffu, count & 1), b1 = __ballot_sync(0xffffffffu, count & 2),
                       b2 = __ballot_sync(0xffffffffu, count & 4);
        int at = before + __popc(b0 & below) + 2 * __popc(b1 & below) + 4 * __popc(b2 & below);
        before += __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (bits >> i & 1) {
                if (at < cap_list) list[at] = p0 + x + 4 * lane + i;
                ++at;
            }
    }
    // Rows that stay where they are, by the whole cluster: those places are its first blocks'. (AGED: each block its own
    // places, since ages change where they are and another block's keys may come from them.)
    if (AGED) {
        __syncthreads();  // the block has its list, and looks at no age again but at the thread's own places
        for (int x = 4 * threadIdx.x; x < places; x += 4 * kThreads) {
            const uint4 k = keys4(x);
            const uint32_t four[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = p0 + x + i;
                if (j >= p1) continue;
                const bool st = stays(j, four[i]);
                if (j >= keep) {
                    if (!st) age[j] = 0;
                } else if (st) {
                    if (e.acc_out != e.acc) e.acc_out[row + j] = acc[j];
                    if (e.src) e.src[row + j] = j;
                    age[j] = aged(j, j, age[j]);
                }
            }
        }
    } else if (e.src || e.acc_out != e.acc) {
#pragma unroll 4
        for (int j = rank * kThreads + threadIdx.x; j < keep; j += C * kThreads) {
            const float x = acc[j];
            if (!stays(j, sum_key(x))) continue;
            if (e.acc_out != e.acc) e.acc_out[row + j] = x;
            if (e.src) e.src[row + j] = j;
        }
    }
    // (sums that change under the call leave the results undefined, but no list is left)
    const int moves = min(all, cap_list) / 2;
    cluster_sync<C>();  // the lists are there, acc has been read, and no block reads another's memory any more

    // A warp takes up to 32 moves: a lane looks up one of them, then NB lanes share each, with 16 channels of
    // keys and values as they are held. Few moves are spread over all warps.
    constexpr int NB = L::kBlocks, kTeams = 32 / NB, kAtOnce = 4, kAll = C * kWarps;
    const int turns = max(1, (moves + 32 * kAll - 1) / (32 * kAll));
    const int per = ((moves + turns * kAll - 1) / (turns * kAll) + kTeams - 1) / kTeams * kTeams;  // of a warp's turn, at most 32
    const int blk = lane % NB, team = lane / NB;
    for (long long i1 = (long long)(rank * kWarps + warp) * per; i1 < moves; i1 += (long long)kAll * per) {
        int to = 0, from = 0, gt = -1, gf = -1;  // places, their groups (-1: nothing to move)
        if (lane < per && i1 + lane < moves) {
            to = list[i1 + lane];
            from = list[moves + i1 + lane];
            if ((unsigned)to < (unsigned)n && (unsigned)from < (unsigned)n) {  // (else sums changed under the call)
                gt = cache_group(a, b, h, to / kGroup);
                gf = cache_group(a, b, h, from / kGroup);
                e.acc_out[row + to] = acc[from];
                if (e.src) e.src[row + to] = from;
                if (AGED) {
                    age[to] = aged(to, from, age[from]);
                    age[from] = 0;
                }
            }
        }
        if (gt < 0 || gf < 0) gt = -1;
        for (int i0 = 0; i0 < per; i0 += kAtOnce * kTeams) {
            uint2 k[kAtOnce], v[kAtOnce];
            uint8_t ks[kAtOnce], vs[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int i = i0 + u * kTeams + team;  // (below 32; those from per on have no groups)
                const int at = __shfl_sync(0xffffffffu, from, i) % kGroup, group = __shfl_sync(0xffffffffu, gf, i);
                if (__shfl_sync(0xffffffffu, gt, i) < 0) continue;
                const uint8_t* src = cache + (long long)group * L::kBytes;
                const int vr = L::v_row(at);
                k[u] = *reinterpret_cast<const uint2*>(src + L::k_code(at, blk));
                ks[u] = src[L::k_scale(at, blk)];
                if (D == 128) {  // a block is one chunk
                    v[u] = *reinterpret_cast<const uint2*>(src + L::v_chunk(vr, blk));
                } else {  // or two
                    v[u].x = *reinterpret_cast<const uint32_t*>(src + L::v_chunk(vr, 2 * blk));
                    v[u].y = *reinterpret_cast<const uint32_t*>(src + L::v_chunk(vr, 2 * blk + 1));
                }
                vs[u] = src[L::v_scale(at, blk)];
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int i = i0 + u * kTeams + team;
                const int at = __shfl_sync(0xffffffffu, to, i) % kGroup, group = __shfl_sync(0xffffffffu, gt, i);
                if (group < 0) continue;
                uint8_t* dst = cache + (long long)group * L::kBytes;
                const int vr = L::v_row(at);
                *reinterpret_cast<uint2*>(dst + L::k_code(at, blk)) = k[u];
                dst[L::k_scale(at, blk)] = ks[u];
                if (D == 128) {
                    *reinterpret_cast<uint2*>(dst + L::v_chunk(vr, blk)) = v[u];
                } else {
                    *reinterpret_cast<uint32_t*>(dst + L::v_chunk(vr, 2 * blk)) = v[u].x;
                    *reinterpret_cast<uint32_t*>(dst + L::v_chunk(vr, 2 * blk + 1)) = v[u].y;
                }
                dst[L::v_scale(at, blk)] = vs[u];
            }
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

template <int D, int C, bool AGED>
static cudaError_t evict_c(const CacheArgs& a, const EvictArgs& e, uint8_t* cache, cudaStream_t st) {
    const int room = (int)std::min<long long>(kMaxKeys, ((e.cap + C - 1) / C + 3) & ~3LL);
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = set_smem_once((const void*)k_cache_evict<D, C, AGED>, kMaxKeys * 4, &done);
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
    err = cudaLaunchKernelEx(&c, k_cache_evict<D, C, AGED>, a, e, cache, room);
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

template <int D, bool AGED> static cudaError_t evict_t(const CacheArgs& a, const EvictArgs& e, uint8_t* cache, cudaStream_t st) {
    // Blocks of a row: more while they have many places each and two of them for each SM hold all
    // rows at once. (32 rows of 32768 places in 2, 4 and 8 blocks: 49, 30 and 26 us; 144 rows of up to 9001 in
    // 1, 2 and 4: 24.1, 24.3 and 31.) Lengths are on the device, so the blocks and their shared memory go by the table's
    // width: where it is far above the lengths that costs (128 rows of 2112 with room for 131,072 places 18.4 us instead of
    // 8.9, 144 of 700 to 9001 with room for 98,304 28.9 instead of 19.9).
    const long long rows = (long long)a.B * a.Hkv;
    int c = 1;
    while (c < 8 && e.cap > 4096LL * c && rows * c <= num_sms()) c *= 2;
    return c == 1   ? evict_c<D, 1, AGED>(a, e, cache, st)
           : c == 2 ? evict_c<D, 2, AGED>(a, e, cache, st)
           : c == 4 ? evict_c<D, 4, AGED>(a, e, cache, st)
                    : evict_c<D, 8, AGED>(a, e, cache, st);
}

cudaError_t launch_cache_evict(const CacheArgs& a, const EvictArgs& e, int d, void* cache, cudaStream_t st) {
    prof_mark(st, "cache_evict");
    uint8_t* c = (uint8_t*)cache;
    if (e.age) return d == 64 ? evict_t<64, true>(a, e, c, st) : evict_t<128, true>(a, e, c, st);
    return d == 64 ? evict_t<64, false>(a, e, c, st) : evict_t<128, false>(a, e, c, st);
}

}  // namespace mita
