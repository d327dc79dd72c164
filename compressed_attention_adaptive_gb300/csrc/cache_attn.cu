// Attention of a call's rows over everything a sequence has in the 4-bit paged
// cache (format and layout: cache.cuh).
//
// For a row q of query head h and the keys k_j, values v_j, j < m that it sees
// in the cache head of its group:
//
//   z_j = scale q.k_j,  M = max z_j,  p_j = exp(z_j - M),  l = sum p_j
//   o = sum p_j v_j / l,   lse = M + ln l
//
// in one pass over the cache with a running maximum and sum. It reads
// len 2 (d/2 + d/16) bytes per sequence and cache head and does 4 d flops per
// row and key, so with few rows per cache head it is bound by HBM: at the
// measured copy rate an SM has 6.3 clocks per token of 128 channels, 3.1 of 64.
//
// Measured (one row per cache head, d = 128, 32 heads, calls in a graph): 7.5 us for 1024
// tokens, 32 for 32,768 (4.7 TB/s), 102 for 131,072 (5.9), 195 for 262,144 (6.2); each further
// token costs 1.03 times what it does at the copy rate. The other 9 us are the same for
// every length: 2 to launch, 1.4 to find a block's place on the line, 1.5 until
// the first codes arrive, an SM's last blocks alone, 2 for the join. Calls launched one by
// one take about 3 us more (35 for 32,768 tokens).
//
// Work split. An item is one (sequence, tile of query rows, cache head); it is
// cut into chunks of 128 tokens. The chunks of all items form one line, and the
// line is cut into equal pieces, one per block: lengths that differ from
// sequence to sequence balance by themselves, and one long sequence spreads
// over the whole GPU. A block that has all of an item's chunks writes its rows;
// one that has a part writes the unnormalized sums, and k_cache_join adds the
// parts. Everything is derived from the lengths on the device, so a captured
// call follows them when it is replayed.
#include <algorithm>
#include <atomic>

#include "cache_walk.cuh"

namespace mita {

constexpr int kStep = 32;  // tokens of a warp's step (4 warps)
constexpr int kThreads = 128;

// ------------------------------------------------------ staging of groups

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The groups of a warp's steps in a segment: step i is the 32 tokens from
// (c0 + i) * 128 + 32 * warp on, two groups. Lane l holds the group number of
// group l & 1 of step l >> 1 in the current run of 16 steps; the next run's
// table entries are loaded a run ahead.
struct GroupRun {
    int cur, nxt;
    // -1: behind the segment or the last key that a row sees (n), or no page of the pool
    __device__ __forceinline__ static int load(const CacheArgs& a, const Segment& s, int n, int warp, int lane, int i0,
                                               int* found) {
        const int step = i0 + (lane >> 1);
        const int gi = ((s.c0 + step) * kChunk + warp * kStep) / kGroup + (lane & 1);
        if (s.c0 + step >= s.c1 || gi * kGroup >= n) return -1;
        const int g = cache_group(a, s.b, s.h, gi);
        if (g < 0) *found |= kFoundBounds;
        return g;
    }
    __device__ __forceinline__ void begin(const CacheArgs& a, const Segment& s, int n, int warp, int lane, int* found) {
        cur = load(a, s, n, warp, lane, 0, found);
        nxt = load(a, s, n, warp, lane, 16, found);
    }
    // group g of step i; called once per step, in order
    __device__ __forceinline__ int get(int i, int g) const { return __shfl_sync(0xffffffffu, cur, 2 * (i & 15) + g); }
    __device__ __forceinline__ void advance(const CacheArgs& a, const Segment& s, int n, int warp, int lane, int i,
                                            int* found) {
        if ((i & 15) == 15) {
            cur = nxt;
            nxt = load(a, s, n, warp, lane, i + 17, found);
        }
    }
};

// Copies step i's two groups into `dst` (bytes of a group without a page are
// filled with zeros) and commits the copies as one group of the thread.
template <int D>
__device__ __forceinline__ void stage_step(const uint8_t* cache, uint32_t dst, int g0, int g1, int lane) {
    constexpr int N = Grp<D>::kBytes / 16;
#pragma unroll
    for (int j = 0; j < (2 * N + 31) / 32; ++j) {
        const int k = lane + 32 * j;
        if (2 * N % 32 == 0 || k < 2 * N) {
            const int g = k < N ? g0 : g1;
            tc::cp_async16(dst + k * 16, cache + (long long)max(g, 0) * Grp<D>::kBytes + (k < N ? k : k - N) * 16, g >= 0);
        }
    }
    copy_commit();
}

// ------------------------------------------------------------ CUDA cores

constexpr int kSimtStages = 2;

template <int D, int R> constexpr int simt_smem() {
    constexpr int ring = 4 * kSimtStages * 2 * Grp<D>::kBytes, merge = 16 * R * (D + 2) * 4;
    return ring > merge ? ring : merge;
}

// fp32 throughout. Eight lanes share a token, each with the d/8 channels of its
// chunk: a warp takes four tokens at a time, and a lane keeps the sums of its
// own tokens and channels, so that only the scores cross lanes (three
// exchanges). The 16 sets of sums of a block are joined at a segment's end.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads)
k_cache_attn_simt(CacheArgs a, const T* __restrict__ Q, const uint8_t* __restrict__ cache, AttnOut out) {
    using L = Grp<D>;
    constexpr int E = D / 8;  // channels of a lane
    extern __shared__ __align__(128) uint8_t smem[];
    allow_next();
    int found = 0;
    const int piece = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> 3, ch = lane & 7;  // token of four, chunk
    __shared__ Walk<R> walk;
    __shared__ LineScan sums;
    if (!walk.begin(a, piece, out.pieces, sums)) {
        end_piece(a, out, piece, 0);
        return;
    }
    uint8_t* ring = smem + warp * (kSimtStages * 2 * L::kBytes);
    const uint32_t ring_addr = tc::smem_u32(ring);

    do {
        const Segment& s = walk.s();
        const int n = s.n, count = s.count, b = s.b;
        const float kscale = a.scale * kLog2e * pow2(cache_exp(a, 0, s.h)), vscale = pow2(cache_exp(a, 1, s.h));
        float q[R][E], o[R][E], m[R], l[R];
        int lim[R];
        int top = 0;  // keys that any row of the tile sees
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int t = 0;
            const long long at = row_offset(a, b, s.h, s.row0 + min(r, s.rows - 1), &t) * D + ch * E;
            lim[r] = r < s.rows ? row_limit(a, n, count, t) : 0;
            top = max(top, lim[r]);
            m[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = to_f(Q[at + i]);
                q[r][i] = isfinite(x) ? x : __int_as_float(0x7fc00000);  // the row becomes NaN, as its softmax is
                o[r][i] = 0.0f;
            }
        }
        const int steps = s.c1 - s.c0;
        GroupRun gr;
        gr.begin(a, s, min(n, top), warp, lane, &found);
        int issued = 0;
        for (; issued < kSimtStages - 1; ++issued) {
            const int g0 = gr.get(issued, 0), g1 = gr.get(issued, 1);
            if (issued < steps)
                stage_step<D>(cache, ring_addr + issued * 2 * L::kBytes, g0, g1, lane);
            else
                copy_commit();
            gr.advance(a, s, min(n, top), warp, lane, issued, &found);
        }
        for (int i = 0; i < steps; ++i) {
            const int nx = i + kSimtStages - 1;
            const int g0 = gr.get(nx, 0), g1 = gr.get(nx, 1);
            __syncwarp();
            if (nx < steps)
                stage_step<D>(cache, ring_addr + (nx % kSimtStages) * 2 * L::kBytes, g0, g1, lane);
            else
                copy_commit();
            gr.advance(a, s, min(n, top), warp, lane, nx, &found);
            copy_wait<kSimtStages - 1>();
            __syncwarp();
            const int base = (s.c0 + i) * kChunk + warp * kStep;
            if (base >= top) continue;
            const uint8_t* st = ring + (i % kSimtStages) * 2 * L::kBytes;
            float z[8][R];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int tok = (4 * u + sub) & 15;
                const uint8_t* g = st + (u >> 2) * L::kBytes;
                const int blk = D == 128 ? ch : ch >> 1;
                uint32_t w8[D / 64];
#pragma unroll
                for (int i2 = 0; i2 < D / 64; ++i2)
                    w8[i2] = reinterpret_cast<const uint32_t*>(g + tok * L::kRow)[ch * (D / 64) + i2];
                const uint32_t sb = g[L::k_scale(tok, blk)];
                const uint32_t s2 = e4m3x2_to_half2(sb | sb << 8);
                float acc[R];
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r] = 0.0f;
#pragma unroll
                for (int i2 = 0; i2 < D / 64; ++i2) {
                    uint32_t h[4];
                    e2m1x8_to_half2(w8[i2], h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 k2 = half2_to_float2(hmul2(h[j], s2));
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            acc[r] = fmaf(q[r][8 * i2 + 2 * j], k2.x, acc[r]);
                            acc[r] = fmaf(q[r][8 * i2 + 2 * j + 1], k2.y, acc[r]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int x = 4; x; x >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], x);
                    z[u][r] = base + 4 * u + sub < lim[r] ? acc[r] * kscale : -INFINITY;
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mx = m[r];
#pragma unroll
                for (int u = 0; u < 8; ++u) mx = fmaxf(mx, z[u][r]);
                const float ref = mx == -INFINITY ? 0.0f : mx;  // no key seen yet
                const float alpha = exp2f(m[r] - ref);
                m[r] = mx;
                l[r] *= alpha;
#pragma unroll
                for (int i2 = 0; i2 < E; ++i2) o[r][i2] *= alpha;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    z[u][r] = exp2f(z[u][r] - ref);
                    l[r] += z[u][r];
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int tok = (4 * u + sub) & 15;
                const uint8_t* g = st + (u >> 2) * L::kBytes;
                const int blk = D == 128 ? ch : ch >> 1, j0 = base + 4 * u + sub;
                const uint32_t* vp = reinterpret_cast<const uint32_t*>(g + L::v_chunk(L::v_row(tok), ch));
                const uint32_t sb = g[L::v_scale(tok, blk)];
                const uint32_t s2 = e4m3x2_to_half2(sb | sb << 8);
#pragma unroll
                for (int i2 = 0; i2 < D / 64; ++i2) {
                    uint32_t h[4];
                    e2m1x8_to_half2(vp[i2], h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 v2 = half2_to_float2(hmul2(h[j], s2));
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            // a key a row does not see adds nothing, whatever its bytes are
                            const bool seen = j0 < lim[r];
                            o[r][8 * i2 + 2 * j] = fmaf(z[u][r], seen ? v2.x : 0.0f, o[r][8 * i2 + 2 * j]);
                            o[r][8 * i2 + 2 * j + 1] = fmaf(z[u][r], seen ? v2.y : 0.0f, o[r][8 * i2 + 2 * j + 1]);
                        }
                    }
                }
            }
        }
        copy_wait<0>();
        __syncthreads();
        // join the 16 sets: (maximum, sum) first, then the sums of values
        float* ml = reinterpret_cast<float*>(smem);
        float* os = ml + 16 * R * 2;
        const int set = warp * 4 + sub;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (ch == 0) {
                ml[(set * R + r) * 2] = m[r];
                ml[(set * R + r) * 2 + 1] = l[r];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) os[(set * R + r) * D + ch * E + i] = o[r][i];
        }
        __syncthreads();
        const bool whole = s.whole();
        const int slot = s.slot(piece);
        for (int x = threadIdx.x; x < s.rows * D; x += kThreads) {
            const int r = x / D, c = x - r * D;
            float mx = -INFINITY;
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, ml[(i * R + r) * 2]);
            const float ref = mx == -INFINITY ? 0.0f : mx;
            float sum = 0.0f, acc = 0.0f;
            for (int i = 0; i < 16; ++i) {
                const float f = exp2f(ml[(i * R + r) * 2] - ref);
                sum = fmaf(f, ml[(i * R + r) * 2 + 1], sum);
                acc = fmaf(f, os[(i * R + r) * D + c], acc);
            }
            acc *= vscale;
            if (whole) {
                int t;
                const long long at = row_offset(a, b, s.h, s.row0 + r, &t);
                reinterpret_cast<T*>(out.O)[at * D + c] = from_f<T>(sum == 0.0f ? 0.0f : acc / sum);
                if (out.lse && c == 0) out.lse[at] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
            } else {
                out.part[((long long)slot * R + r) * D + c] = acc;
                if (c == 0) out.ml[(long long)slot * R + r] = make_float2(mx, sum);
            }
        }
    } while (walk.next(a));
    end_piece(a, out, piece, found);
}

// --------------------------------------------------------- tensor cores

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// 8 x 8 halves, lane (g, t) holding row g, columns 2 t and 2 t + 1: transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void store4(float* p, float x, float y, float z, float w) {
    *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float x, float y, float z, float w) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x, y), b = __floats2bfloat162_rn(z, w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

constexpr int kStages = 2;
constexpr float kLow = 4096.0f;  // lo is at most 8 where its number is below 2^15
// Blocks per SM that the registers allow without spills (but 4 to 8 registers of float32
// rows of 128 channels, at a segment's start). (16 rows of 128 channels: 3 blocks 48.6 us,
// 4 at 128 registers 51.2; 16 rows of 64: 33.0 and 30.9.)
constexpr int mma_blocks(int d, int NR) { return NR == 1 ? 4 : d == 64 ? (NR == 2 ? 4 : 3) : (NR == 2 ? 3 : 2); }

// Q's halves: float rows are two of them
template <typename T, int D, int NR> constexpr int mma_q_bytes() { return (sizeof(T) == 4 ? 2 : 1) * NR * (D / 16) * 256; }
template <typename T, int D, int NR> constexpr int mma_smem() {
    constexpr int ring = 4 * kStages * 2 * Grp<D>::kBytes, merge = 4 * 8 * NR * D * 4;
    return (ring > merge ? ring : merge) + mma_q_bytes<T, D, NR>();
}

// The tensor cores' register form (m16n8k16, halves in, fp32 out), tiles of 8 NR
// rows.
//
// The codes come from shared memory into the registers of the lanes that feed
// them to the step, are widened there and never go back to shared memory: one
// conversion per two codes and one product by the scale, both exact. (tcgen05
// needs the widened operands written first, to shared or tensor memory, 3.5 times the
// cached bytes, which pays with more than 32 rows: cache_tile.cu.)
//
// Tokens and value channels are the 16 side of a step and query rows the 8 side
// (S^T = K Q^T, O^T = V^T P^T): decoding has few rows, and with rows on the 16 side
// half of the steps and exponentials would be for rows that are not there.
//
// A warp takes 32 tokens at a time, each warp its own, with its own maximum and
// sums, so nothing but a segment's end joins the block:
//   S^T   2 token tiles x d/16 steps. Q's rows are scaled by a power of two that puts their
//         largest entry in [2^14, 2^15), so that bf16 is exact as halves down to 2^-31 of
//         it; the power goes into the factor f of the scores.
//   p = 2^(S f - m) in fp32, rounded to halves for the product with V (2^-11 relative; the sum
//         l takes the unrounded p). m starts 7 below a row's first maximum and is moved, to 7
//         below the maximum, when a score exceeds it by more than 15. So 2^7 <= max p <= 2^15,
//         the halves' normal numbers reach 2^-21 of the maximum, and only a move makes lanes
//         compare maxima and rescale sums.
//   O^T   P^T is S^T's register layout transposed 8 x 8; 2 steps of 16 tokens x d/16 channel tiles.
//
// float32 rows are each two halves, x = hi + lo with lo = x - hi rounded (22 bits and
// a sign, 2^-23 of x), p likewise: two products where bf16 has one, with the same
// exact keys and values. The products are summed in fp32 by steps of 16 or 32 tokens
// and by ordinary additions from there. The lower halves are held kLow times as large, and m
// starts 11 below a maximum, so that p keeps its 22 bits down to 2^-26 of the maximum and is
// off by 2^-48 of it below. (Unscaled, weights 2^-24 of the largest had 8 bits and those below
// 2^-32 none: 1e-4 of the result where a key of that weight has no value. The scale takes a
// second sum: over lengths around 16384, 8 x 12 heads, d = 64, 37.0 us against 35.7; 2 x 16 heads
// of about 30,000, d = 128, 40.6 against 40.3; with 12 rows 26.0 against 25.0. On CUDA cores the first
// case takes 49.)
//
// The next segment is found while a segment's first codes are on their way, and its own
// first copies are issued before the warps' sums are joined (3 % of 8 x 12 heads of 16384 tokens
// in float32 and of 32 x 32 of 2048, bf16 batches of short sequences 1 to 2 %).
//
// A warp has about 570 instructions per 32 tokens of 128 channels and 8 rows, 128 of
// them conversions of codes and 128 products by scales (half rate each). Over the
// whole of a 32 us launch under ncu (two 32k prompts, 32 heads) the arithmetic pipe is at
// 52 %, the issue slots at 57 %, DRAM at 0.72 of the copy rate; in the middle of it
// DRAM is near that rate. float32 with d = 64 (8 x 12 heads of 16384 tokens) is at 41 %, 60 % and
// 0.47 and 15 rows of d = 64 at 39 %, 55 % and 0.34: no unit is full there, a warp's steps wait for
// each other's results. Other forms, measured on the first case when this one was at 33 us, 36.7
// with the join: rows on the 16 side 42.7; with the join, 5 blocks per SM at 96 registers 39.8 against
// 39.0 then, three copy stages 37.1, twice as many pieces of half the size 41.1, smaller
// pieces for an SM's later blocks (which run behind the first) 37.2 to 38.6. Steps
// of 64 tokens for d = 64: 131,072 tokens 68.1 to 64.8 us, but 26.8 to 27.9 for the
// ragged drafts of 15 rows.
template <typename T, int D, int NR>
__global__ void __launch_bounds__(kThreads, mma_blocks(D, NR))
k_cache_attn_mma(CacheArgs a, const T* __restrict__ Q, const uint8_t* __restrict__ cache, AttnOut out) {
    using L = Grp<D>;
    constexpr bool F = sizeof(T) == 4;  // float rows
    constexpr int KS = D / 16, NT = D / 8, W = D / 32, RT = 8 * NR, ST = kStages;
    constexpr int GP = NR == 1 ? 2 : 1;  // groups at a time: with more rows the registers hold one
    constexpr int kStage = 2 * L::kBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Walk<RT> walk;
    __shared__ float2 sml[4][RT];
    __shared__ float szf[RT];
    __shared__ int slim[RT];
    __shared__ uint64_t bars[4][ST];
    allow_next();
    int found = 0;
    const int piece = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t* ring = smem + warp * (ST * kStage);
    const uint32_t ring_addr = tc::smem_u32(ring);
    uint2* qs = reinterpret_cast<uint2*>(smem + mma_smem<T, D, NR>() - mma_q_bytes<T, D, NR>());
    if (lane == 0) {
        // (fault test: one more signal for the first step of one warp of the call than come)
        for (int i = 0; i < ST; ++i) tc::mbar_init(&bars[warp][i], a.stall && i + warp + piece == 0 ? 3 : 2);
        tc::fence_mbar_init();
    }
    __shared__ LineScan sums;
    if (!walk.begin(a, piece, out.pieces, sums)) {
        end_piece(a, out, piece, 0);
        return;
    }
    int put = 0, take = 0, phase = 0;  // stages of the ring, and the phase of `take`
    bool dead = false;                 // a wait ran out: the warp goes on without keys
    // A segment's copies. Lane l has the group number of group l & 1 of step l >> 1 in the
    // current run of 16 steps, and issues that copy itself; the next run's table entries are
    // loaded a run ahead.
    const uint8_t *gcur, *gnxt;
    int low, top, steps;  // keys that the first and the last row of the tile see
    auto groups = [&](const Segment& s, int i0) -> const uint8_t* {
        const int gi = GroupRun::load(a, s, top, warp, lane, i0, &found);
        return gi < 0 ? nullptr : cache + (long long)gi * L::kBytes;
    };
    auto enter = [&](const Segment& s) {
        // rows of a tile see more keys the later their token is
        low = row_limit(a, s.n, s.count, s.row0 / a.G);
        top = row_limit(a, s.n, s.count, (s.row0 + s.rows - 1) / a.G);
        steps = dead ? 0 : s.c1 - s.c0;
        gcur = groups(s, 0);
        gnxt = groups(s, 16);
    };
    auto issue = [&](const Segment& s, int i) {
        if (i < steps && (lane >> 1) == (i & 15)) {
            uint64_t* bar = &bars[warp][put];
            if (gcur) {
                tc::mbar_expect_tx(bar, L::kBytes);
                bulk_copy(ring_addr + put * kStage + (lane & 1) * L::kBytes, gcur, L::kBytes, bar);
            } else {
                tc::mbar_arrive(bar);
            }
        }
        if (i < steps) put = put + 1 == ST ? 0 : put + 1;
        if ((i & 15) == 15) {
            gcur = gnxt;
            gnxt = groups(s, i + 17);
        }
    };
    int k = walk.cur;  // the current segment
    enter(walk.segs[k]);
    issue(walk.segs[k], 0);

    for (bool more = true; more; k ^= 1) {
        const Segment& s = walk.segs[k];
        const int n = s.n, count = s.count, b = s.b;
        // Q: warp w has rows 8 w + g, lane (g, t4) channels [t4 d/4, (t4 + 1) d/4) of them
        const float vscale = pow2(cache_exp(a, 1, s.h));
        if (warp < NR) {
            const int r = warp * 8 + g;
            int t = 0;
            const long long at = row_offset(a, b, s.h, s.row0 + min(r, s.rows - 1), &t);
            constexpr int QW = D / 16 * sizeof(T) / 4;  // 16-byte words of a lane's channels
            uint32_t x[4 * QW], amax = 0;
#pragma unroll
            for (int i = 0; i < QW; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < s.rows) v = reinterpret_cast<const uint4*>(Q + at * D + t4 * (D / 4))[i];
                x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 4 * QW; ++i)
                amax = max(amax, F ? x[i] & 0x7fffffffu : max(x[i] << 16 & 0x7fff0000u, x[i] & 0x7fff0000u));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float up, f;
            query_scale(a, s.h, amax >> 23, &up, &f);
            if (t4 == 0) {
                szf[r] = f;
                slim[r] = r < s.rows ? row_limit(a, n, count, t) : 0;
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y0 = __uint_as_float(F ? x[(4 * ks + 2 * e) % (4 * QW)] : x[2 * ks + e] << 16) * up;
                    const float y1 = __uint_as_float(F ? x[(4 * ks + 2 * e + 1) % (4 * QW)] : x[2 * ks + e] & 0xffff0000u) * up;
                    hi[e] = pack_half2(y0, y1);
                    const float2 h = half2_to_float2(hi[e]);
                    lo[e] = pack_half2((y0 - h.x) * kLow, (y1 - h.y) * kLow);
                }
                qs[(ks * NR + warp) * 32 + lane] = make_uint2(hi[0], hi[1]);
                if (F) qs[((KS + ks) * NR + warp) * 32 + lane] = make_uint2(lo[0], lo[1]);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) walk.segment(a);  // the next one, while the first codes are on their way
        constexpr bool kQRegs = NR == 1 && !F;  // Q in registers, else in shared memory
        uint2 qf[kQRegs ? KS : 1];
        if (kQRegs) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[ks % (kQRegs ? KS : 1)] = qs[ks * 32 + lane];
        }
        // of this lane's rows 8 i + 2 t4 and the next
        float zf[NR][2], m[NR][2], l[NR][2], o[NR][NT / 2][4];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                zf[i][e] = szf[8 * i + 2 * t4 + e];
                m[i][e] = kNoKey;
                l[i][e] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < NT / 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] = 0.0f;
        }

        for (int i = 0; i < steps; ++i) {
            __syncwarp();  // the stage that the next copy goes to has been read
            issue(s, i + ST - 1);
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars[warp][take], phase, a.status, a.spin))) {
                // Give up, but not before the copies in flight have landed (or the wait's time has passed
                // for each). The warp takes part in what the block still does, with sums that mean
                // nothing, as the status word will say.
                for (int x = i + 1; x < steps && x < i + ST; ++x) {
                    take = take + 1 == ST ? 0 : take + 1;
                    phase ^= take == 0;
                    tc::mbar_wait(&bars[warp][take], phase, a.status, a.spin);
                }
                dead = true;
                found |= kFoundTimeout;
                break;
            }
            const uint8_t* st = ring + take * kStage;
            take = take + 1 == ST ? 0 : take + 1;
            phase ^= take == 0;
#pragma unroll 1
            for (int h = 0; h < 2; h += GP) {
                const int base = (s.c0 + i) * kChunk + warp * kStep + 16 * h;
                if (base >= top) break;

                // scores of 16 tokens each: [0], [1] token g, rows 2 t4 and the next; [2], [3] token g + 8
                constexpr int NL = F ? NR : 1;
                float z[NR][GP][4], zl[NL][GP][4];  // zl: the lower halves' part
                uint32_t kw[GP][2][W], sc[GP][2][D / 64];  // [group][token g, g + 8]: codes; scales, each in both halves
#pragma unroll
                for (int gi = 0; gi < GP; ++gi) {
                    const uint8_t* kb = st + (h + gi) * L::kBytes;
                    if (D == 128) {
                        const uint32_t sb = *reinterpret_cast<const uint32_t*>(kb + L::kKs + g * 16 + t4 * 4);
                        const uint32_t s0 = e4m3x2_to_half2(sb & 0xffff), s1 = e4m3x2_to_half2(sb >> 16);
                        sc[gi][0][0] = __byte_perm(s0, s0, 0x1010);
                        sc[gi][0][D / 64 - 1] = __byte_perm(s0, s0, 0x3232);
                        sc[gi][1][0] = __byte_perm(s1, s1, 0x1010);
                        sc[gi][1][D / 64 - 1] = __byte_perm(s1, s1, 0x3232);
                    } else {
                        const uint32_t s0 = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(kb + L::kKs + g * 8 + t4 * 2));
                        sc[gi][0][0] = __byte_perm(s0, s0, 0x1010);
                        sc[gi][1][0] = __byte_perm(s0, s0, 0x3232);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint8_t* kr = kb + (8 * x + g) * L::kRow + t4 * (D / 8);
                        if (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(kr);
                            kw[gi][x][0] = v.x; kw[gi][x][1] = v.y; kw[gi][x][W - 2] = v.z; kw[gi][x][W - 1] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(kr);
                            kw[gi][x][0] = v.x; kw[gi][x][1] = v.y;
                        }
                    }
                }
#pragma unroll
                for (int wi = 0; wi < W; ++wi) {
                    uint32_t k8[GP][2][4];
#pragma unroll
                    for (int gi = 0; gi < GP; ++gi)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            e2m1x8_to_half2(kw[gi][x][wi], k8[gi][x]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) k8[gi][x][j] = hmul2(k8[gi][x][j], sc[gi][x][wi >> 1]);
                        }
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                        for (int j = 0; j < NR; ++j) {
                            const int ks = 2 * wi + k2;
                            const uint2 q = kQRegs ? qf[ks % (kQRegs ? KS : 1)] : qs[(ks * NR + j) * 32 + lane];
#pragma unroll
                            for (int gi = 0; gi < GP; ++gi) {
                                if (ks == 0)
                                    mma_f16_first(z[j][gi], k8[gi][0][0], k8[gi][1][0], k8[gi][0][1], k8[gi][1][1], q.x, q.y);
                                else
                                    mma_f16(z[j][gi], k8[gi][0][2 * k2], k8[gi][1][2 * k2], k8[gi][0][2 * k2 + 1],
                                            k8[gi][1][2 * k2 + 1], q.x, q.y);
                            }
                            if (F) {
                                const uint2 ql = qs[((KS + ks) * NR + j) * 32 + lane];
#pragma unroll
                                for (int gi = 0; gi < GP; ++gi) {
                                    if (ks == 0)
                                        mma_f16_first(zl[j % NL][gi], k8[gi][0][0], k8[gi][1][0], k8[gi][0][1], k8[gi][1][1],
                                                      ql.x, ql.y);
                                    else
                                        mma_f16(zl[j % NL][gi], k8[gi][0][2 * k2], k8[gi][1][2 * k2], k8[gi][0][2 * k2 + 1],
                                                k8[gi][1][2 * k2 + 1], ql.x, ql.y);
                                }
                            }
                        }
                }
                if (F) {
#pragma unroll
                    for (int j = 0; j < NR; ++j)
#pragma unroll
                        for (int x = 0; x < GP; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e) z[j][x][e] = fmaf(zl[j % NL][x][e], 1 / kLow, z[j][x][e]);
                }
                const bool edge = base + 16 * GP > low;  // some row does not see all of these tokens
                if (edge) {
#pragma unroll
                    for (int j = 0; j < NR; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int lim = slim[8 * j + 2 * t4 + (e & 1)], tok = base + g + 8 * (e >> 1);
#pragma unroll
                            for (int x = 0; x < GP; ++x)
                                if (tok + 16 * x >= lim) z[j][x][e] = -INFINITY;
                        }
                }
                // against the reference, in log2 units
                float y[NR][GP][4], big = kNoKey;
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int x = 0; x < GP; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[j][x][e] = score_diff(z[j][x][e], zf[j][e & 1], m[j][e & 1]);
                            big = fmaxf(big, y[j][x][e]);
                        }
                if (__any_sync(0xffffffffu, big > 15.0f)) {
#pragma unroll
                    for (int j = 0; j < NR; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = fmaxf(z[j][0][e], z[j][0][e + 2]);
                            if (GP == 2) v = fmaxf(v, fmaxf(z[j][GP - 1][e], z[j][GP - 1][e + 2]));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
                            // (a row's own scores move it, not another's)
                            const float mn = score_diff(v, zf[j][e], m[j][e]) > 15.0f
                                                 ? score_diff(v, zf[j][e], F ? 11.0f : 7.0f)
                                                 : m[j][e];
                            const float f = tc::ex2(m[j][e] - mn);
                            m[j][e] = mn;
                            l[j][e] *= f;
#pragma unroll
                            for (int x = 0; x < NT / 2; ++x) {
                                o[j][x][e] *= f;
                                o[j][x][e + 2] *= f;
                            }
#pragma unroll
                            for (int x = 0; x < GP; ++x) {
                                y[j][x][e] = score_diff(z[j][x][e], zf[j][e], mn);
                                y[j][x][e + 2] = score_diff(z[j][x][e + 2], zf[j][e], mn);
                            }
                        }
                }
                uint32_t p[NR][GP][2], pl[NL][GP][2];  // P^T: [group][tokens 2 t4 and the next, 8 further], row g
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int x = 0; x < GP; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float p0 = tc::ex2(y[j][x][2 * e]), p1 = tc::ex2(y[j][x][2 * e + 1]);
                            l[j][0] += p0;
                            l[j][1] += p1;
                            const uint32_t h2 = pack_half2(p0, p1);
                            p[j][x][e] = transpose8(h2);
                            if (F) {
                                const float2 hf = half2_to_float2(h2);
                                pl[j % NL][x][e] =
                                    transpose8(pack_half2(fmaf(hf.x, -kLow, p0 * kLow), fmaf(hf.y, -kLow, p1 * kLow)));
                            }
                        }
                // groups whose products with V are summed before they go to a float row's o
                constexpr int GS = F ? GP : 1;
#pragma unroll
                for (int g0 = 0; g0 < GP; g0 += GS) {
                    uint32_t s0[GS], s1[GS], vw[GS][4][D / 64];
#pragma unroll
                    for (int gs = 0; gs < GS; ++gs) {
                        const int gi = g0 + gs;
                        const uint8_t* vb = st + (h + gi) * L::kBytes;
                        uint32_t sb = *reinterpret_cast<const uint32_t*>(vb + L::kVs + (D == 128 ? g : g >> 1) * 16 + t4 * 4);
                        if (edge) {
                            // Nothing of a token that a row does not see may reach it: bytes of tokens
                            // that no row sees are made zero here; NaN of a token that only some rows
                            // see is taken out of the product and put into the rows that see it.
                            const int tok = base + 16 * gi + 2 * t4;
                            uint32_t nan = 0;
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint32_t byte = 0xffu << (8 * x);
                                if (tok + 8 * (x >> 1) + (x & 1) >= top) sb &= ~byte;
                                if ((sb >> (8 * x) & 0x7f) == 0x7f) nan |= byte;
                            }
                            if (__any_sync(0xffffffffu, nan != 0)) {
                                sb &= ~nan;
                                const uint32_t one = 0x3c003c00u;  // (1, 1) in halves
                                const uint32_t a0 = __byte_perm(nan, 0, 0x1100) & one, a2 = __byte_perm(nan, 0, 0x3322) & one;
#pragma unroll
                                for (int j = 0; j < NR; ++j) {
                                    const int lim = slim[8 * j + g];
                                    uint32_t see[2];
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
                                        see[x] = (tok + 8 * x < lim ? 0x3c00u : 0u) | (tok + 8 * x + 1 < lim ? 0x3c000000u : 0u);
                                    float hit[4];
                                    mma_f16_first(hit, a0, a0, a2, a2, see[0], see[1]);
#pragma unroll
                                    for (int x = 0; x < NT / 2; ++x)
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (hit[e] > 0.0f) o[j][x][e] = __int_as_float(0x7fc00000);
                                }
                            }
                        }
                        s0[gs] = e4m3x2_to_half2(sb & 0xffff);
                        s1[gs] = e4m3x2_to_half2(sb >> 16);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint8_t* vr = vb + L::v_chunk(t4 + 4 * x, g);
                            if (D == 128) {
                                const uint2 v = *reinterpret_cast<const uint2*>(vr);
                                vw[gs][x][0] = v.x; vw[gs][x][D / 64 - 1] = v.y;
                            } else {
                                vw[gs][x][0] = *reinterpret_cast<const uint32_t*>(vr);
                            }
                        }
                    }
#pragma unroll
                    for (int wi = 0; wi < D / 64; ++wi) {
                        // a byte of both tokens of a pair: even channels, then odd ones
                        constexpr uint32_t lo = 0x0f0f0f0fu;
                        uint32_t v8[GS][2][2][4];  // [group][tokens 8 x + 2 t4 ..][parity of the channel]
#pragma unroll
                        for (int gs = 0; gs < GS; ++gs)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t u0 = vw[gs][2 * x][wi], u1 = vw[gs][2 * x + 1][wi];
                                e2m1x8_to_half2((u0 & lo) | ((u1 << 4) & ~lo), v8[gs][x][0]);
                                e2m1x8_to_half2(((u0 >> 4) & lo) | (u1 & ~lo), v8[gs][x][1]);
                            }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t av[GS][4];
#pragma unroll
                            for (int gs = 0; gs < GS; ++gs)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    av[gs][e] = hmul2(v8[gs][e >> 1][e & 1][x], e < 2 ? s0[gs] : s1[gs]);
#pragma unroll
                            for (int j = 0; j < NR; ++j) {
                                if (!F) {
                                    mma_f16(o[j][4 * wi + x], av[0][0], av[0][1], av[0][2], av[0][3], p[j][g0][0], p[j][g0][1]);
                                    continue;
                                }
                                float c[4], cl[4];
                                mma_f16_first(cl, av[0][0], av[0][1], av[0][2], av[0][3], pl[j % NL][g0][0], pl[j % NL][g0][1]);
                                mma_f16_first(c, av[0][0], av[0][1], av[0][2], av[0][3], p[j][g0][0], p[j][g0][1]);
#pragma unroll
                                for (int gs = 1; gs < GS; ++gs) {
                                    mma_f16(cl, av[gs][0], av[gs][1], av[gs][2], av[gs][3], pl[j % NL][gs][0], pl[j % NL][gs][1]);
                                    mma_f16(c, av[gs][0], av[gs][1], av[gs][2], av[gs][3], p[j][gs][0], p[j][gs][1]);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[j][4 * wi + x][e] += fmaf(cl[e], 1 / kLow, c[e]);
                            }
                        }
                    }
                }
            }
        }
        // the row sums over the lanes of a row
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], x);
        // Join the warps: [warp][row][d] sums, 16 bytes (four channels) at a time. With 8 rows
        // they are in the stage of the warp's ring that the next segment's first copy does not
        // go to, else over all the rings. The lanes that store together have four rows and two
        // chunks apart by d/32; the row's bits exchange chunks so that eight lanes meet eight bank
        // groups.
        constexpr bool kOwn = NR == 1;
        static_assert(!kOwn || (ST == 2 && kStage >= 8 * D * 4 && kStage % 128 == 0), "a stage holds a warp's sums");
        if (!kOwn) __syncthreads();  // every warp is done with its ring
        float4* os = reinterpret_cast<float4*>(smem + (kOwn ? (put ^ 1) * kStage : 0));
        constexpr int C4 = D / 4, kWarpRows = kOwn ? ST * kStage / (D * 4) : RT;  // rows from one warp's to the next's
        static_assert(!kOwn || ST * kStage % (D * 4) == 0, "whole rows");
        auto at4 = [&](int wp, int r, int c) {
            const int t = (r >> 1) & 3;
            return (wp * kWarpRows + r) * C4 + (c ^ (D == 128 ? t : (t & 1) | (t & 2) << 1));
        };
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * j + 2 * t4 + e;
                if (g == 0) sml[warp][r] = make_float2(m[j][e], l[j][e]);
                if (r >= s.rows) continue;
#pragma unroll
                for (int x = 0; x < NT / 4; ++x)
                    os[at4(warp, r, g * (NT / 4) + x)] = make_float4(o[j][2 * x][e], o[j][2 * x][e + 2],
                                                                     o[j][2 * x + 1][e], o[j][2 * x + 1][e + 2]);
            }
        __syncthreads();
        const Segment& next = walk.segs[k ^ 1];
        more = walk.more;
        if (more) {
            enter(next);
            if (kOwn) issue(next, 0);
        }
        const bool whole = s.whole();
        const int slot = s.slot(piece);
        for (int x = threadIdx.x; x < s.rows * C4; x += kThreads) {
            const int r = x / C4, c = x - r * C4;
            float2 v[4];
            float mx = kNoKey;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = sml[i][r];
                mx = fmaxf(mx, v[i].x);
            }
            float sum = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = tc::ex2(v[i].x - mx);
                const float4 u = os[at4(i, r, c)];
                sum = fmaf(f, v[i].y, sum);
                acc.x = fmaf(f, u.x, acc.x); acc.y = fmaf(f, u.y, acc.y);
                acc.z = fmaf(f, u.z, acc.z); acc.w = fmaf(f, u.w, acc.w);
            }
            if (whole) {
                int t;
                const long long at = row_offset(a, b, s.h, s.row0 + r, &t);
                const float inv = sum == 0.0f ? 0.0f : vscale / sum;
                store4(reinterpret_cast<T*>(out.O) + at * D + 4 * c, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                if (out.lse && c == 0) out.lse[at] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
            } else {
                acc.x *= vscale; acc.y *= vscale; acc.z *= vscale; acc.w *= vscale;
                reinterpret_cast<float4*>(out.part + ((long long)slot * RT + r) * D)[c] = acc;
                if (c == 0) out.ml[(long long)slot * RT + r] = make_float2(mx, sum);
            }
        }
        tc::fence_proxy_async();  // the next segment's copies come after these accesses of the ring
        __syncthreads();
        if (!kOwn && more) issue(next, 0);
    }
    end_piece(a, out, piece, found);
}

// ------------------------------------------------------------------ join

// Rows of a block that has W warps for each row.
constexpr int join_rows(int W) { return W >= 8 ? 1 : 8 / W; }
constexpr int kJoinAhead = 4;

// Block (x, y) joins the parts of one cut item, the y-th join_rows(W) rows: item x of
// the call when there are no more items than pieces, else the one that begins in piece x
// and goes on behind it. It finds that from the lengths while the attention runs (loading
// a description of it that the attention left made a call 1.5 us longer). Each of a row's
// W warps adds every W-th part, a lane d/32 channels of it; the first kJoinAhead are
// loaded together with the maxima and sums.
template <typename T, int D, int W>
__global__ void __launch_bounds__(32 * W * join_rows(W)) k_cache_join(CacheArgs a, AttnOut out, bool by_item) {
    constexpr int E = D / 32, R = join_rows(W);
    __shared__ float acc8[R][W][D];
    __shared__ float2 ml8[R][W];
    __shared__ CutItem cut;
    __shared__ LineScan sums;
    const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5, mine = sub / W, warp = sub % W;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y) return;
        wait_previous();
        int found = 0;
        for (int i = threadIdx.x; i < out.pieces; i += blockDim.x) found |= out.found[i];
        const int bounds = __syncthreads_or(found & kFoundBounds), timeout = __syncthreads_or(found & kFoundTimeout);
        if (threadIdx.x == 0) *a.status = timeout ? kStTimeout : bounds ? kStBounds : kStOk;
        return;
    }
    if (threadIdx.x == 0) cut.rows = 0;
    find_cut(a, out, blockIdx.x, by_item, sums, cut);
    __syncthreads();
    const CutItem c = cut;
    if ((int)blockIdx.y * R >= c.rows) return;
    wait_previous();
    const int r = blockIdx.y * R + mine;
    if (r < c.rows) {
        // part p > 0 begins its piece
        auto slot = [&](int p) { return (long long)(2 * (c.piece + p) + (p == 0)) * out.rows + r; };
        auto load = [&](int p, float* v) {
            const float* part = out.part + slot(p) * D;
            if (E == 4) {
                const float4 u = reinterpret_cast<const float4*>(part)[lane];
                v[0] = u.x; v[1] = u.y; v[E - 2] = u.z; v[E - 1] = u.w;
            } else {
                const float2 u = reinterpret_cast<const float2*>(part)[lane];
                v[0] = u.x; v[1] = u.y;
            }
        };
        float mx = kNoKey, sum = 0.0f, acc[E], ahead[kJoinAhead][E];
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
#pragma unroll
            for (int i = 0; i < E; ++i) ahead[j][i] = 0.0f;
            if (warp + j * W < c.parts) load(warp + j * W, ahead[j]);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
        // lane l has the maximum and sum of the l-th of 32 of the warp's parts
        for (int p0 = warp; p0 < c.parts; p0 += 32 * W) {
            const int pl = p0 + lane * W;
            const float2 ml = pl < c.parts ? out.ml[slot(pl)] : make_float2(kNoKey, 0.0f);
            const float m = fmaxf(ml.x, kNoKey), mn = fmaxf(mx, warp_max(m)), old = exp2f(mx - mn), f = exp2f(m - mn);
            sum = sum * old + warp_sum(f * ml.y);
            mx = mn;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] *= old;
            const int n = min(32, (c.parts - p0 + W - 1) / W);
            int j = 0;
            if (p0 == warp) {
#pragma unroll
                for (; j < kJoinAhead; ++j) {
                    const float fj = __shfl_sync(0xffffffffu, f, j);
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (j < n) acc[i] = fmaf(fj, ahead[j][i], acc[i]);
                }
            }
#pragma unroll 8
            for (; j < n; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, j);
                float v[E];
                load(p0 + j * W, v);
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = fmaf(fj, v[i], acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) acc8[mine][warp][lane * E + i] = acc[i];
        if (lane == 0) ml8[mine][warp] = make_float2(mx, sum);
    }
    __syncthreads();
    if (r >= c.rows) return;
    float top = kNoKey, s = 0.0f, f[W];
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, ml8[mine][w].x);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        f[w] = exp2f(ml8[mine][w].x - top);
        s = fmaf(f[w], ml8[mine][w].y, s);
    }
    int t;
    const long long at = row_offset(a, c.b, c.h, c.row0 + r, &t);
    const int i0 = warp * 32 + lane;
    for (int i = i0; i < D; i += 32 * W) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v = fmaf(f[w], acc8[mine][w][i], v);
        reinterpret_cast<T*>(out.O)[at * D + i] = from_f<T>(s == 0.0f ? 0.0f : v / s);
    }
    if (out.lse && i0 == 0) out.lse[at] = s == 0.0f ? -INFINITY : (top + log2f(s)) * kLn2;
}

// ------------------------------------------------------------------ launch

// Units of the line, at most (cache_walk.cuh's Line counts them in 32 bits).
static long long cache_attn_units(const CacheArgs& a, int rtile, int extra) {
    const long long tiles = ((long long)a.G * a.T + rtile - 1) / rtile;
    const long long len = ((long long)a.cols * a.page + kChunk - 1) / kChunk;
    return (long long)a.B * a.Hkv * tiles * (len + extra);
}

CachePlan cache_attn_plan(const CacheArgs& a, int d, int dtype, unsigned flags) {
    CachePlan p{};
    const long long rows = (long long)a.G * a.T;
    // Rows of a tile: the fewest that hold the cache head's rows. Up to 32 rows a tile is
    // in registers; above, 64 rows of 128 channels go to tcgen05. (32 rows over 2 x 16 heads
    // of 32768 tokens: 65 us in registers, 78 on tcgen05; 64 rows over 4 x 8 heads of 9000
    // to 16384 tokens: 57.5 as two tiles in registers, 41.6 on tcgen05.) float32 takes
    // twice the registers, so 16 rows at most.
    p.tensor = !(flags & MITA_FLAG_SIMT);
    int blocks = 4;  // per SM
    if (p.tensor) {
        p.rows = rows <= 8 ? 8 : rows <= 16 || dtype == 0 ? 16 : rows <= 32 || d == 64 ? 32 : 64;
        p.tile = p.rows == 64;
        blocks = p.tile ? 1 : mma_blocks(d, p.rows / 8);
    } else {
        p.rows = rows == 1 ? 1 : 4;
    }
    p.pieces = (int)std::min<long long>((long long)blocks * num_sms(), cache_attn_units(a, p.rows, 0));
    p.fits = cache_attn_units(a, p.rows, kTileExtra) < (1LL << 31);
    p.parts = (size_t)2 * p.pieces * p.rows;
    return p;
}

long long cache_spin(bool stall) { return stall ? tc::kSpinTest : tc::kSpin; }

template <typename T, int D, int W>
static cudaError_t join_w(const CacheArgs& a, const AttnOut& o, long long items, cudaStream_t st) {
    const bool by_item = items <= o.pieces;
    const int rows = (int)std::min<long long>(o.rows, (long long)a.G * a.T);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((by_item ? (int)items : o.pieces) + 1, (rows + join_rows(W) - 1) / join_rows(W));
    c.blockDim = dim3(32 * W * join_rows(W));
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, k_cache_join<T, D, W>, a, o, by_item);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T, int D>
static cudaError_t join_t(const CacheArgs& a, const AttnOut& o, cudaStream_t st) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    prof_mark(st, "cache_join");
    // Warps of a row by the pieces that there are for an item: with 76 of them (8 items) 4, 8
    // and 16 warps 39.1, 37.1 and 35.8 us; with 9.5 (64 items) 2, 4 and 8 warps 37.1, 35.0
    // and 35.0; with 5 (32 items of 64 rows) 41.6, 44.0 and 49.4; with 1.2 (512 items) 63.9,
    // 66.3 and 70.6; with 38 (16 items) 4 and 16 warps 33.6 and 32.3, with 19 both 32.3.
    const long long items = (long long)a.B * o.tiles * a.Hkv;
    if (o.pieces >= 24 * items) return join_w<T, D, 16>(a, o, items, st);
    return o.pieces >= 6 * items ? join_w<T, D, 4>(a, o, items, st) : join_w<T, D, 2>(a, o, items, st);
}

// Sets a kernel's shared memory limit, once per device (`done`: a bit for each of
// the first 64; above those every time).
cudaError_t set_smem_once(const void* f, int bytes, std::atomic<unsigned long long>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ULL << dev : 0;
    if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
    return e;
}

template <typename T, int D, int R>
static cudaError_t simt_t(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st) {
    constexpr int smem = simt_smem<D, R>();
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = set_smem_once((const void*)k_cache_attn_simt<T, D, R>, smem, &done);
    if (e != cudaSuccess) return e;
    k_cache_attn_simt<T, D, R><<<o.pieces, kThreads, smem, st>>>(a, (const T*)Q, cache, o);
    count_launch();
    return join_t<T, D>(a, o, st);
}

template <typename T, int D, int NR>
static cudaError_t mma_t(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st) {
    constexpr int smem = mma_smem<T, D, NR>();
    static_assert(mma_blocks(D, NR) * (smem + 3 * 1024) <= 228 * 1024, "the blocks that a call counts on fit an SM");
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = set_smem_once((const void*)k_cache_attn_mma<T, D, NR>, smem, &done);
    if (e != cudaSuccess) return e;
    k_cache_attn_mma<T, D, NR><<<o.pieces, kThreads, smem, st>>>(a, (const T*)Q, cache, o);
    count_launch();
    return join_t<T, D>(a, o, st);
}

template <int D>
static cudaError_t attn_t(const CacheArgs& a, const CachePlan& p, int dtype, const void* Q, const uint8_t* cache,
                          const AttnOut& o, cudaStream_t st) {
    using bf16 = __nv_bfloat16;
    if (dtype == 0) {
        if (p.tensor) return p.rows == 8 ? mma_t<float, D, 1>(a, Q, cache, o, st) : mma_t<float, D, 2>(a, Q, cache, o, st);
        return p.rows == 1 ? simt_t<float, D, 1>(a, Q, cache, o, st) : simt_t<float, D, 4>(a, Q, cache, o, st);
    }
    if (p.tile) {
        const cudaError_t e = launch_cache_tile(a, Q, cache, o, st);
        return e != cudaSuccess ? e : join_t<bf16, D>(a, o, st);
    }
    if (p.tensor)
        return p.rows == 8    ? mma_t<bf16, D, 1>(a, Q, cache, o, st)
               : p.rows == 16 ? mma_t<bf16, D, 2>(a, Q, cache, o, st)
                              : mma_t<bf16, D, 4>(a, Q, cache, o, st);
    return p.rows == 1 ? simt_t<bf16, D, 1>(a, Q, cache, o, st) : simt_t<bf16, D, 4>(a, Q, cache, o, st);
}

cudaError_t launch_cache_attn(const CacheArgs& a, const CachePlan& p, int d, int dtype, const void* Q,
                              const void* cache, void* O, float* lse, const CacheParts& parts, cudaStream_t st) {
    const int tiles = (int)(((long long)a.G * a.T + p.rows - 1) / p.rows);
    const AttnOut o{O, lse, parts.part, parts.ml, parts.found, p.pieces, p.rows, p.tile ? kTileExtra : kExtra, tiles};
    const uint8_t* c = (const uint8_t*)cache;
    prof_mark(st, "cache_attention");
    return d == 64 ? attn_t<64>(a, p, dtype, Q, c, o, st) : attn_t<128>(a, p, dtype, Q, c, o, st);
}

}  // namespace mita
