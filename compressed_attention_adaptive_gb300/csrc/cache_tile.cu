// Attention over the 4-bit cache for many rows per cache head (drafted tokens of
// grouped queries, parts of prompts): tiles of 64 bf16 rows of 128 channels on
// tcgen05. (cache_attn.cu has the work split and the form for few rows.)
//
// With 64 rows a cached token costs 64 times 4 d = 32,768 flops against 144 bytes.
// The register form of cache_attn.cu needs 17.6 clocks of an SM per token for that
// at its full rate, and widens the codes for each 32 rows anew. Here a chunk of
// 128 tokens is widened once, to halves in tensor memory, for all rows:
//
//   S^T = K Q^T    128 tokens x N rows: K from tensor memory, Q a K-major tile, fp32 in tensor memory
//   P^T = 2^(f S^T - m) as halves, in shared memory (MN-major: a token's N rows are contiguous)
//   O^T += V^T P^T  128 channels x N rows: V^T from tensor memory, O^T fp32 in tensor memory
//
// Tokens and channels are the 128 side: rows would fill only half of it. A softmax
// thread has a token of S^T with 16 of its rows, so a row's maximum would go across
// 128 threads; as in cache_attn.cu the reference m is only moved when a score
// exceeds it by more than 15, and each thread keeps its own part of the rows' sums
// until a segment ends.
//
// Widened operands go to tensor memory, 512 columns in all: keys as rows of 64
// columns, a lane a token; values in the register order of m16n8k16's A, which is
// that of a 16 x 128 bit store and needs no transposition. Lane 32 w + 16 i + 8 o + g
// has channel 16 g + 4 w + 2 i + o. (As tiles in shared memory they were written and
// read there, 160 KB a chunk: 288 us against 269 for the long case below.)
//
// Warps: N / 4 for the softmax and the epilogue, each warpgroup 16 of the rows; one
// copies; one issues the products; four widen keys and four values. Codes have four
// stages, scores and weights three, keys and values two. Every wait is bounded; a
// block that gives up raises its abort flag, lets its copies and products land and
// frees its tensor memory.
//
// Measured, calls in a graph: 64 rows over 2 x 16 heads of 131,072 tokens 261 us (526 TFLOP/s),
// of 32,768 77 us; 4 x 8 heads of 9000 to 16384 tokens 41.6 us (the register form 57.5). A chunk
// takes about 2400 clocks, and no role is busy all of it: softmax 1900, values 1500,
// issuing 1000 (a product of 128 x 64 x 16 takes 51 to 60), copies 1000, keys 800. No unit
// is full (issue slots 58 %, the tensor pipe 16 %): the roles wait for each other's stages.
// The values' 16-bit reads are two-way bank conflicts, all of them. What it took: operands in
// uniform registers (323 us to 288), 16 rows per softmax thread instead of 32 (a softmax chunk
// 2200 clocks to 1450), an epilogue of little code (13 us off every item: cold instructions),
// fewer and longer copies (each takes 180 clocks to issue).
#include <atomic>

#include "cache_tc.cuh"

namespace mita {

namespace {

constexpr int kD = 128, N = 64;  // channels; rows of a tile
constexpr int HN = 16;           // rows of a softmax thread
constexpr int kRaw = 8 * Grp<kD>::kBytes;  // a chunk's codes and scales
constexpr int kRawStages = 4, kSoftStages = 3;  // of codes; of scores and weights
constexpr int kEdge = 64;                  // tokens that only some rows of a tile see, at most

struct TileSmem {
    static constexpr int kSoft = N / 4, kCopy = kSoft, kIssue = kSoft + 1, kWiden = kSoft + 2;  // warps
    static constexpr int kThreads = 32 * (kSoft + 10);
    static constexpr int kP = 128 * 128;  // a token's rows, padded to 128 bytes
    static constexpr int kQ = 0, kPo = kQ + 64 * kD * 2, kRawO = kPo + kSoftStages * kP,
                         kBytes = kRawO + kRawStages * kRaw + 1024;
};

// The four softmax warps with the same rows meet here (barrier 1 + wg), all of them the
// same number of times whatever happened to the waits before.
__device__ __forceinline__ void softmax_sync(int wg) {
    __syncwarp();
    asm volatile("barrier.sync %0, 128;" ::"r"(1 + wg) : "memory");
}
__device__ __forceinline__ bool softmax_any(int wg, bool x) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + wg)
        : "memory");
    return r != 0;
}

// Joins v[0..16) over the 32 lanes: each step a lane keeps half of the values and
// gives the other half away. Lane l ends with value l / 2, in v[0].
template <typename Op> __device__ __forceinline__ void reduce_lanes(float* v, int lane, Op op) {
#pragma unroll
    for (int s = 16, n = HN / 2; s; s >>= 1, n >>= 1) {
        if (n == 0) {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], s));
            continue;
        }
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < HN / 2; ++i) {
            if (i >= n) break;
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, s));
        }
    }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void load_cols(uint32_t taddr, float* v) {  // HN columns
    tmem_ld16(taddr, v);
    tc::tmem_wait_ld();
}
// v, or NaN if a token from `low` on that the row sees (up to `end`) has NaN in this block of its values
__device__ __noinline__ float seen_nan(float v, const uint8_t* nanv, int low, int end, int blk) {
    for (int x = low; x < end; ++x)
        if (nanv[x - low] >> blk & 1) v = __int_as_float(0x7fc00000);
    return v;
}
struct TileBars {
    uint64_t raw_full[kRawStages], raw_empty[kRawStages], k_full[2], v_full[2], v_empty[2];
    uint64_t s_full[kSoftStages], p_full[kSoftStages], q_full, o_full, drain;
};

}  // namespace

__global__ void __launch_bounds__(TileSmem::kThreads, 1)
k_cache_attn_tile(CacheArgs a, const __nv_bfloat16* __restrict__ Q, const uint8_t* __restrict__ cache, AttnOut out) {
    using L = Grp<kD>;
    using S = TileSmem;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sm = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* smp = smem_raw + (sm - tc::smem_u32(smem_raw));
    __shared__ Walk<N, kTileExtra> walk;
    __shared__ TileBars bar;
    __shared__ __align__(16) float2 ref[N];  // the rows' factors of scores, in log2 units, and references
    __shared__ float fac[N], lsum[N], linv[N], part4[4][N];
    __shared__ int lim[N], nan_flag;
    __shared__ long long row_at[N];
    __shared__ __align__(16) uint8_t nanv[kEdge];  // blocks of a token's values that are NaN, tokens from `low` on
    __shared__ uint32_t tmem_slot;
    __shared__ Abort abort;
    volatile Abort* abort_v = &abort;
    allow_next();
    const int piece = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int found = 0;
    // (waits for another kernel's blocks on this SM, which end whatever this one does)
    if (warp == S::kIssue) tc::tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        for (int i = 0; i < kRawStages; ++i) {
            // (fault test: one more signal for the first chunk of one block than comes)
            tc::mbar_init(&bar.raw_full[i], a.stall && i + piece == 0 ? 2 : 1);
            tc::mbar_init(&bar.raw_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.k_full[i], 4);
            tc::mbar_init(&bar.v_full[i], 4);
            tc::mbar_init(&bar.v_empty[i], 1);
        }
        for (int i = 0; i < kSoftStages; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_full[i], S::kSoft);
        }
        tc::mbar_init(&bar.q_full, S::kSoft);
        tc::mbar_init(&bar.o_full, 1);
        tc::mbar_init(&bar.drain, 1);
        tc::fence_mbar_init();
        abort.flag = nan_flag = 0;
        abort.limit = (int)(a.spin / tc::kSpinTest);
    }
    if (tid < kEdge) nanv[tid] = 0;
    tc::fence_before_sync();
    __shared__ LineScan sums;
    bool more = walk.begin(a, piece, out.pieces, sums);
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    constexpr uint32_t kO = 192, kK = 256, kV = 384;  // columns: three S of 64, O, two chunks' keys, two chunks' values

    int done = 0, seg = 0;  // chunks and segments before this one: the barriers' phases go on
    int issued = 0;         // chunks that the copying warp has issued
    bool stop = false;      // a wait of an earlier segment gave up
    for (; more; ++seg) {
        const Segment s = walk.s();
        const int n = s.n, count = s.count;
        const int low = row_limit(a, n, count, s.row0 / a.G), top = row_limit(a, n, count, (s.row0 + s.rows - 1) / a.G);
        // chunks that some row of the tile sees, at least one
        const int nc = max(1, min(s.c1, (top + kChunk - 1) / kChunk) - s.c0);
        if (stop) {
            // what is left of the piece is not computed, and the status word says so
        } else if (warp == S::kCopy) {
            // ---------------------------------------------------- copies
            // Lane l looks after group l % 8 of chunk l / 8 in the current run of four chunks; the next
            // run's table entries are loaded a run ahead. A copy takes the groups that a page and a
            // chunk have together (issuing one takes 180 clocks), and the first one's lane issues it.
            struct Copy {
                const uint8_t* src;
                uint32_t bytes;
            };
            auto copies = [&](int c0) {
                const int c = c0 + (lane >> 3), first = lane & 7, gi = (s.c0 + c) * 8 + first, rem = gi % a.pgroups;
                const int last = (top + kGroup - 1) / kGroup;
                if (c >= nc || gi >= last || (first && rem)) return Copy{nullptr, 0};
                const int g = cache_group(a, s.b, s.h, gi);
                if (g < 0) {
                    found |= kFoundBounds;
                    return Copy{nullptr, 0};
                }
                const int groups = min(min(8 - first, a.pgroups - rem), last - gi);
                return Copy{cache + (long long)g * L::kBytes, (uint32_t)(groups * L::kBytes)};
            };
            Copy cur = copies(0), nxt = copies(4);
            for (int c = 0; c < nc; ++c) {
                const int t = done + c, st = t % kRawStages;
                if (!warp_wait(&bar.raw_empty[st], ((t / kRawStages) & 1) ^ 1, abort_v)) break;
                const bool mine = (lane >> 3) == (c & 3);
                const uint32_t bytes = __reduce_add_sync(0xffffffffu, mine ? cur.bytes : 0u);
                if (elect_one()) tc::mbar_expect_tx(&bar.raw_full[st], bytes);
                __syncwarp();
                if (mine && cur.bytes)
                    bulk_copy(sm + S::kRawO + st * kRaw + (lane & 7) * L::kBytes, cur.src, cur.bytes, &bar.raw_full[st]);
                issued = t + 1;
                if ((c & 3) == 3) {
                    cur = nxt;
                    nxt = copies(c + 5);
                }
            }
            __syncwarp();
        } else if (warp == S::kIssue) {
            // -------------------------------------------------- products
            // Scores are issued two chunks ahead of the values, so that the way from one chunk's
            // weights over the next scores to their weights, which is several waits long, is gone
            // over once for three chunks.
            constexpr uint32_t idS = idesc_half(128, N, 0, 0), idO = idesc_half(128, N, 0, 1);
            bool ok = warp_wait(&bar.q_full, seg & 1, abort_v);
            auto issue_s = [&](int c) {
                const int t = done + c, st = t & 1, ss = t % kSoftStages;
                if (!warp_wait(&bar.k_full[st], (t >> 1) & 1, abort_v)) return false;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // 16 channels each
                        tc::mma_bf16_ts(tmem + ss * 64, tmem + kK + st * 64 + k * 8,
                                        tc::sdesc(sm + S::kQ + (k >> 2) * (64 * 128) + (k & 3) * 32, 16, 1024), idS, k > 0);
                    tc::mma_commit(&bar.s_full[ss]);
                }
                __syncwarp();
                return true;
            };
            for (int c = 0; c < min(2, nc) && ok; ++c) ok = issue_s(c);
            for (int c = 0; c < nc && ok; ++c) {
                // (into the scores of chunk c - 1, whose weights are there)
                if (c + 2 < nc && !(ok = issue_s(c + 2))) break;
                const int t = done + c, st = t & 1, ss = t % kSoftStages;
                if (!(ok = warp_wait(&bar.v_full[st], (t >> 1) & 1, abort_v))) break;
                if (!(ok = warp_wait(&bar.p_full[ss], (t / kSoftStages) & 1, abort_v))) break;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // 16 tokens each
                        tc::mma_bf16_ts(tmem + kO, tmem + kV + st * 64 + k * 8,
                                        tc::sdesc(sm + S::kPo + ss * S::kP + k * 2048, S::kP, 1024), idO, k > 0 || c > 0);
                    tc::mma_commit(&bar.v_empty[st]);
                    if (c == nc - 1) tc::mma_commit(&bar.o_full);
                }
                __syncwarp();
            }
        } else if (warp >= S::kWiden) {
            // -------------------------------------------------- widening
            // Four warps have the keys and four the values, each the quarter of the lanes of tensor
            // memory that it can reach.
            const int quarter = warp & 3;
            const bool keys = warp - S::kWiden < 4;
            const uint32_t lanes = tmem + ((uint32_t)quarter << 21);
            // keys: the lane's token, its four 16-byte words read in an order that meets every bank once
            const int kt = lane & 15, rot = (lane >> 1) & 3;
            // values: lane (g, t) as in cache_attn.cu; of each 16 channels the warp has bytes 2 quarter and the next
            const int g = lane >> 2, t4 = lane & 3;
            for (int c = 0; c < nc; ++c) {
                const int t = done + c, st = t & 1, rs = t % kRawStages;
                if (!warp_wait(&bar.raw_full[rs], (t / kRawStages) & 1, abort_v)) break;
                const uint8_t* raw = smp + S::kRawO + rs * kRaw;
                if (keys) {
                    const uint8_t* gr = raw + (2 * quarter + (lane >> 4)) * L::kBytes;
                    uint4 v[4], w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const uint4*>(gr + kt * L::kRow)[(i + rot) & 3];
                    const uint4 sw = *reinterpret_cast<const uint4*>(gr + L::kKs + (kt & 7) * 16);
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.raw_empty[rs]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = rot & 1 ? v[(i + 3) & 3] : v[i];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = rot & 2 ? w[(i + 2) & 3] : w[i];
                    // the products that read this stage: scores of chunk t - 2
                    const int ts = t - 2;
                    if (ts >= 0 && !warp_wait(&bar.s_full[ts % kSoftStages], (ts / kSoftStages) & 1, abort_v)) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 32 channels, 16 columns
                        const uint32_t s8 = i == 0 ? sw.x : i == 1 ? sw.y : i == 2 ? sw.z : sw.w;
                        const uint32_t s2 = e4m3x2_to_half2(kt < 8 ? s8 & 0xffff : s8 >> 16);
                        const uint32_t cw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                        uint32_t h[16];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t sc = __byte_perm(s2, s2, j < 2 ? 0x1010 : 0x3232);
                            e2m1x8_to_half2(cw[j], h + 4 * j);
#pragma unroll
                            for (int x = 0; x < 4; ++x) h[4 * j + x] = hmul2(h[4 * j + x], sc);
                        }
                        tmem_st16(lanes + kK + st * 64 + 16 * i, reinterpret_cast<const float*>(h));
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.k_full[st]);
                } else {
                    const int tok0 = (s.c0 + c) * kChunk;
                    const bool edge = tok0 + kChunk > low;
                    if (!warp_wait(&bar.v_empty[st], ((t >> 1) & 1) ^ 1, abort_v)) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int gi = 0; gi < 8; gi += 2) {
                        uint32_t h[2][8];  // [lanes 0 .. 15, 16 .. 31]
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint8_t* gr = raw + (gi + y) * L::kBytes;
                            uint32_t sb = *reinterpret_cast<const uint32_t*>(gr + L::kVs + g * 16 + t4 * 4);
                            uint32_t u[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                u[x] = *reinterpret_cast<const uint16_t*>(gr + L::v_chunk(t4 + 4 * x, g) + 2 * quarter);
                            if (edge) {
                                // Nothing of a token that a row does not see may reach it: tokens that no row sees
                                // are zero; NaN of one that some see is zero here and put into those rows' results.
                                const int tok = tok0 + 16 * (gi + y) + 2 * t4;
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const int at = tok + 8 * (x >> 1) + (x & 1);
                                    if (at >= top) {
                                        sb &= ~(0xffu << (8 * x));
                                    } else if (at >= low && (sb >> (8 * x) & 0x7f) == 0x7f) {
                                        sb &= ~(0xffu << (8 * x));
                                        // the byte's other bits belong to other lanes
                                        atomicOr(reinterpret_cast<uint32_t*>(nanv) + ((at - low) >> 2),
                                                 1u << (((at - low) & 3) * 8 + g));
                                        nan_flag = 1;
                                    }
                                }
                            }
                            const uint32_t s0 = e4m3x2_to_half2(sb & 0xffff), s1 = e4m3x2_to_half2(sb >> 16);
                            // a byte of both tokens of a pair: even channels, then odd ones
                            constexpr uint32_t lo = 0x0f0f0f0fu;
                            const uint32_t u0 = __byte_perm(u[0], u[2], 0x5410), u1 = __byte_perm(u[1], u[3], 0x5410);
                            uint32_t e[4], o[4];
                            e2m1x8_to_half2((u0 & lo) | ((u1 << 4) & ~lo), e);
                            e2m1x8_to_half2(((u0 >> 4) & lo) | (u1 & ~lo), o);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                h[i][4 * y] = hmul2(e[i], s0);
                                h[i][4 * y + 1] = hmul2(o[i], s0);
                                h[i][4 * y + 2] = hmul2(e[2 + i], s1);
                                h[i][4 * y + 3] = hmul2(o[2 + i], s1);
                            }
                        }
                        tmem_st_frag(lanes + kV + st * 64 + 8 * gi, h[0]);
                        tmem_st_frag(lanes + (16u << 16) + kV + st * 64 + 8 * gi, h[1]);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive(&bar.raw_empty[rs]);
                        tc::mbar_arrive(&bar.v_full[st]);
                    }
                }
            }
        } else {
            // --------------------------------------------------- softmax
            const float vscale = pow2(cache_exp(a, 1, s.h));
            // Q: thread (r, part) has 16 channels of row r, scaled as in cache_attn.cu.
            {
                const int r = tid >> 3, part = tid & 7;
                int t = 0;
                const long long at = row_offset(a, s.b, s.h, s.row0 + min(r, s.rows - 1), &t);
                uint32_t x[8], amax = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (r < s.rows) v = reinterpret_cast<const uint4*>(Q + at * kD + part * 16)[i];
                    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max(amax, max(x[i] & 0x7fffu, x[i] >> 16 & 0x7fffu));
#pragma unroll
                for (int i = 1; i < 8; i <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, i));
                float up, f;
                query_scale(a, s.h, amax >> 7, &up, &f);
                if (part == 0) {
                    ref[r] = make_float2(f, kNoKey);
                    lim[r] = r < s.rows ? row_limit(a, n, count, t) : 0;
                    row_at[r] = at;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[j] = pack_half2(__uint_as_float(x[4 * i + j] << 16) * up,
                                          __uint_as_float(x[4 * i + j] & 0xffff0000u) * up);
                    st_shared16(sm + S::kQ + tc::sw_off(r, part * 2 + i, 64), h[0], h[1], h[2], h[3]);
                }
                tc::fence_proxy_async();
                softmax_sync(warp >> 2);
                if (lane == 0) tc::mbar_arrive(&bar.q_full);
            }
            // thread: token (then channel) tl, rows r0 to r0 + HN - 1
            const int tl = tid & 127, wg = warp >> 2, r0 = wg * HN, quarter = warp & 3;
            const uint32_t cols = tmem + ((uint32_t)(tid & 96) << 16) + r0;
            float l[HN];
#pragma unroll
            for (int r = 0; r < HN; ++r) l[r] = 0.0f;
            bool ok = true;
            for (int c = 0; c < nc; ++c) {
                const int t = done + c, st = t % kSoftStages, tok = (s.c0 + c) * kChunk + tl;
                // after a wait that gave up the warp goes on without waiting, for the others' sake
                ok &= warp_wait(&bar.s_full[st], (t / kSoftStages) & 1, abort_v);
                tc::fence_after_sync();
                const bool edge = (s.c0 + c + 1) * kChunk > low;  // some row does not see all of the chunk
                float y[HN], big = kNoKey;
                // again after references have moved, which happens once
#pragma unroll 1
                for (int again = 0;; ++again) {
                    load_cols(cols + st * 64, y);
#pragma unroll
                    for (int r = 0; r < HN; r += 2) {
                        const float4 m = *reinterpret_cast<const float4*>(ref + r0 + r);
                        y[r] = score_diff(y[r], m.x, m.y);
                        y[r + 1] = score_diff(y[r + 1], m.z, m.w);
                    }
                    if (edge) {
#pragma unroll
                        for (int r = 0; r < HN; ++r)
                            if (tok >= lim[r0 + r]) y[r] = -INFINITY;
                    }
                    if (again) break;
#pragma unroll
                    for (int r = 0; r < HN; ++r) big = fmaxf(big, y[r]);
                    if (!softmax_any(wg, big > 15.0f)) break;
                    load_cols(cols + st * 64, y);
#pragma unroll
                    for (int r = 0; r < HN; ++r)
                        y[r] = edge && tok >= lim[r0 + r] ? -INFINITY : __fmul_rn(y[r], ref[r0 + r].x);
                    reduce_lanes(y, lane, [](float p, float q) { return fmaxf(p, q); });
                    part4[quarter][r0 + HN * lane / 32] = y[0];
                    softmax_sync(wg);
                    if (tl < HN) {
                        const int r = r0 + tl;
                        const float mx = fmaxf(fmaxf(part4[0][r], part4[1][r]), fmaxf(part4[2][r], part4[3][r]));
                        // (a row's own scores move it, not another's)
                        const float old = ref[r].y, mn = mx - old > 15.0f ? mx - 7.0f : old;
                        fac[r] = tc::ex2(old - mn);
                        ref[r].y = mn;
                    }
                    softmax_sync(wg);
#pragma unroll
                    for (int r = 0; r < HN; ++r) l[r] *= fac[r0 + r];
                    if (c > 0) {
                        // the last products with V (those up to chunk c - 3 were issued before S of this one)
                        ok &= warp_wait(&bar.v_empty[(t - 1) & 1], ((t - 1) >> 1) & 1, abort_v);
                        tc::fence_after_sync();
                        load_cols(cols + kO, y);
#pragma unroll
                        for (int r = 0; r < HN; ++r) y[r] *= fac[r0 + r];
                        tmem_st16(cols + kO, y);
                        tc::tmem_wait_st();
                    }
                }
                const uint32_t pd = sm + S::kPo + st * S::kP;
#pragma unroll
                for (int j = 0; j < HN / 8; ++j) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * j + 2 * i;
                        const float p0 = tc::ex2(y[r]), p1 = tc::ex2(y[r + 1]);
                        l[r] += p0;
                        l[r + 1] += p1;
                        h[i] = pack_half2(p0, p1);
                    }
                    st_shared16(pd + tc::sw_off(tl, r0 / 8 + j, 128), h[0], h[1], h[2], h[3]);
                }
                tc::fence_proxy_async();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.p_full[st]);
            }
            ok &= warp_wait(&bar.o_full, seg & 1, abort_v);
            tc::fence_after_sync();
            if (!softmax_any(wg, !ok)) {
                reduce_lanes(l, lane, [](float p, float q) { return p + q; });
                part4[quarter][r0 + HN * lane / 32] = l[0];
                softmax_sync(wg);
                if (tl < HN) {
                    const int r = r0 + tl;
                    const float sum = (part4[0][r] + part4[1][r]) + (part4[2][r] + part4[3][r]);
                    lsum[r] = sum;
                    linv[r] = sum == 0.0f ? 0.0f : 1.0f / sum;
                }
                softmax_sync(wg);
                const bool whole = s.whole(), nans = nan_flag;
                const long long slot = (long long)s.slot(piece) * N;
                // lane tl of the thread's rows, eight at a time (little code: it runs once a segment)
                const int ch = 16 * (tl & 7) + 4 * (tl >> 5) + ((tl >> 3) & 2) + ((tl >> 3) & 1);
#pragma unroll 1
                for (int i0 = 0; i0 < HN && r0 + i0 < s.rows; i0 += 8) {
                    float o[8];
                    tmem_ld8(cols + kO + i0, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + i0 + i;
                        float v = o[i] * vscale;
                        if (r < s.rows) {
                            if (nans) v = seen_nan(v, nanv, low, min(top, lim[r]), ch >> 4);
                            if (whole)
                                reinterpret_cast<__nv_bfloat16*>(out.O)[row_at[r] * kD + ch] = __float2bfloat16_rn(v * linv[r]);
                            else
                                out.part[(slot + r) * kD + ch] = v;
                        }
                    }
                }
                if (tl < HN && r0 + tl < s.rows) {
                    const int r = r0 + tl;
                    const float sum = lsum[r], m = ref[r].y;
                    if (!whole)
                        out.ml[slot + r] = make_float2(m, sum);
                    else if (out.lse)
                        out.lse[row_at[r]] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
                }
            }
            tc::fence_before_sync();
        }
        done += nc;
        // every warp is through the segment, so that all see the same and meet at the same barriers
        stop = __syncthreads_or(abort.flag);
        if (tid < kEdge) nanv[tid] = 0;
        if (tid == 0) nan_flag = 0;
        more = walk.next(a);
        tc::fence_after_sync();
    }
    // what is in flight lands before the block frees its tensor memory and ends
    if (warp == S::kCopy && lane == 0)
        for (int t = max(0, issued - kRawStages); t < issued; ++t)
            drain(&bar.raw_full[t % kRawStages], (t / kRawStages) & 1, a.status, a.spin);
    if (warp == S::kIssue && lane == 0) {
        tc::mma_commit(&bar.drain);
        drain(&bar.drain, 0, a.status, a.spin);
    }
    tc::fence_before_sync();
    if (abort.flag) found |= kFoundTimeout;
    end_piece(a, out, piece, found);
    tc::fence_after_sync();
    if (warp == S::kIssue) tc::tmem_dealloc(tmem, 512);
}

cudaError_t launch_cache_tile(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st) {
    constexpr int smem = TileSmem::kBytes;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = set_smem_once((const void*)k_cache_attn_tile, smem, &done);
    if (e != cudaSuccess) return e;
    k_cache_attn_tile<<<o.pieces, TileSmem::kThreads, smem, st>>>(a, (const __nv_bfloat16*)Q, cache, o);
    count_launch();
    return cudaGetLastError();
}

}  // namespace mita
