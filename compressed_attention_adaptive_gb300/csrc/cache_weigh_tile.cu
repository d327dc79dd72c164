// The attention weight of cached tokens for many rows per cache head (a prompt's last
// tokens, drafted tokens of grouped queries): tiles of 128 tokens by up to 128 rows on tcgen05.
// (cache_weigh.cu has the mathematics and the form for few rows.)
//
//   S = K Q^T    128 tokens x N rows: K widened to halves in tensor memory, Q a K-major tile in
//                shared memory, fp32 in tensor memory
//
// A lane of tensor memory is a token, so a thread has a token's scores with all rows: it adds up their weights
// by itself. What a token costs is then one exponential per row and the four or so instructions around it; keys are
// widened once for all rows of a pass.
//
// Keys go from memory to registers in the order of m16n8k16's A (the cache's own order: neighbouring lanes
// read neighbouring bytes) and from there to tensor memory by 16 x 128 bit stores, which puts the
// channels of a token in the order {t d/4 + 2 m, t d/4 + 2 m + 1 : t = 0 .. 3} for m = 0, 1, ...; Q's rows are stored in
// the same order.
//
// Warps: four warpgroups for the weights, each with a quarter of a tile's rows, which take turns at joining the four parts of
// a chunk's sums (for up to 64 rows two, each with every other chunk to itself). Four warps widen keys, each the quarter of
// the lanes that it can reach; one issues the products.
// Every wait is bounded; a block that gives up raises its abort flag, lets its products land, frees its
// tensor memory and says so in the status word.
//
// Measured, in a graph: 256 rows over 2 x 8 heads of 32768 tokens 55.1 us (598 TFLOP/s; the register form 221), 32 rows 22.7;
// calls of a decayed sum 59.1 and 22.6, float32 66.1 and 23.5. Up to 64 rows leave 72 registers a thread and spill 56 to 120 bytes:
// 2.6 % of the executed instructions with 32 rows.
// A tile of 128 x 128 takes about 1400 clocks: the exponentials 512 of them, the products 450, what
// four warps of each scheduler issue 800; none is full, the steps wait for each other.
//   - Three warpgroups with a stage of scores and chunks of their own: 72 us; eight widening warps, at whose cost the
//     weights have 72 registers instead of 80: 59.5.
//   - Not kept: half a tile's scores loaded while the other half is weighed, across tiles (68.6); two warpgroups for every
//     second tile (65); two blocks an SM with one stage of 128 rows each (71); warps that only copy (57.8).
#include <algorithm>
#include <type_traits>

#include "cache_tc.cuh"
#include "cache_weigh.cuh"

namespace mita {

namespace {

constexpr int kTok = 128;                        // tokens of a chunk
constexpr int kRaw = 3;                          // stages of codes of a widening warp: copies are kRaw - 1 chunks ahead

// SPLIT: warpgroups that share a tile, with a part of its rows each. Without a split (up to 64 rows, one tile) each has
// chunks to itself, and two smaller blocks share an SM: one's items begin and end while the other's go on.
template <int SPLIT> struct Tiles {
    static constexpr int kBlocks = SPLIT == 1 ? 2 : 1;              // of an SM
    static constexpr int kCols = SPLIT == 1 ? 64 : 128;             // rows of a tile
    static constexpr int kStages = 2;                               // of scores
    static constexpr int kKeys = SPLIT == 1 ? 2 : 4;                // stages of keys
    static constexpr int kSoft = SPLIT == 1 ? kStages : SPLIT;      // warpgroups for the weights
    static constexpr int kWiden = 4 * kSoft, kIssue = kWiden + 4;   // first warps of the other roles
    static constexpr int kThreads = 32 * (kIssue + 1);
    static constexpr uint32_t kK = kStages * kCols, kTmem = 512 / kBlocks;  // columns: of the first stage of keys, in all
    static_assert(kK + kKeys * 64 == kTmem, "tensor memory");
};

// Parts of a chunk's sums, for the warpgroup whose number the chunk's is modulo kSoft; it joins them behind its own part
// of the next chunk. A buffer is used again eight chunks later: a warpgroup comes there only after all have
// released the scores of a chunk kStages before it, which the joining one does after its join.
constexpr int kParts = 8;
static_assert(kParts % Tiles<4>::kSoft == 0 && kParts > Tiles<4>::kStages + 1, "parts would be overwritten");
struct WeighBars {
    uint64_t k_full[4], k_empty[4], s_full[2], s_empty[2], p_full[kParts], drain;
};

// Bytes of a tile's rows: as halves (two for float rows); log sums, factors, limits.
template <typename T, int D, int COLS> constexpr int tile_bytes() { return COLS * (D * 2 * (sizeof(T) == 4 ? 2 : 1) + 12); }

// Rows whose largest entry is in [2^-4, 2^7) (or 0) are all scaled by 2^8, others each as in cache_weigh.cu. Where all rows
// of a pass are of the first kind, which queries are, they share a factor of the scores, and a weight
// takes one number of its row from shared memory instead of two. Entries of 2^-24 and more are exact as halves then, the others
// within 2^-33.
constexpr int kUsual = 8;
__device__ __forceinline__ bool usual_row(uint32_t amax) { return amax == 0 || (amax >> 23 >= 123 && amax >> 23 < 134); }

// Groups of a role's own chunks: lane l looks up group 2 quarter + l % 2 of its own chunk i + l / 2.
struct Groups {
    int cur, nxt;
    template <typename Look> __device__ __forceinline__ void start(Look look) {
        cur = look(0);
        nxt = look(16);
    }
    // called for every i in turn
    __device__ __forceinline__ int get(int i, int y) const { return __shfl_sync(0xffffffffu, cur, 2 * (i & 15) + y); }
    template <typename Look> __device__ __forceinline__ void step(int i, Look look) {
        if ((i & 15) != 15) return;
        cur = nxt;
        nxt = look(i + 17);
    }
};

// Bytes of the widening warps' codes and scales: two groups' keys of each stage.
template <int D> constexpr int raw_bytes() { return 4 * kRaw * 2 * 9 * D; }

// Whether any thread but the widening ones has x; they all meet here.
template <int WARPS> __device__ __forceinline__ bool any_but_widening(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(32 * WARPS)
        : "memory");
    return r != 0;
}

// The loads into v have arrived.
__device__ __forceinline__ void wait_cols(float* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}

}  // namespace

// The call's status word, before the weights' kernel may add to it.
__global__ void __launch_bounds__(256) k_cache_weigh_begin(CacheArgs a) {
    allow_next();
    const bool bad = __syncthreads_or(bad_call<true>(a));
    if (threadIdx.x == 0) *a.status = bad ? kStBounds : kStOk;
}

template <typename T, int D, int SPLIT>
__global__ void __launch_bounds__(Tiles<SPLIT>::kThreads, Tiles<SPLIT>::kBlocks)
k_cache_weigh_tile(CacheArgs a, WeighArgs w, const T* __restrict__ Q, const uint8_t* __restrict__ cache, int tiles) {
    using L = Grp<D>;
    constexpr bool F = sizeof(T) == 4;  // float rows: two halves, hi + lo
    using S = Tiles<SPLIT>;
    constexpr int kCols = S::kCols, kStages = S::kStages, kKeys = S::kKeys, kSoft = S::kSoft, kWiden = S::kWiden,
                  kIssue = S::kIssue, kThreads = S::kThreads;
    constexpr uint32_t kK = S::kK;
    constexpr int KS = D / 16, W = D / 32, kHalf = kCols * D * 2, kTile = (F ? 2 : 1) * kHalf;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sm = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* smp = smem_raw + (sm - tc::smem_u32(smem_raw));
    float* mlse = reinterpret_cast<float*>(smp + tiles * kTile);  // of a row: its log sum, negated;
    float* fac = mlse + tiles * kCols;                            // the factor of its scores;
    int* lim = reinterpret_cast<int*>(fac + tiles * kCols);       // the keys that it sees
    const uint32_t raw = tc::smem_u32(lim + tiles * kCols);
    __shared__ LineStart<kThreads> start;
    __shared__ WeighBars bar;
    __shared__ float parts[SPLIT == 1 ? 1 : kParts][kSoft][kTok];  // [chunk][warpgroup]
    __shared__ uint32_t tmem_slot;
    __shared__ Abort abort;
    volatile Abort* abort_v = &abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
    // (waits for another kernel's blocks on this SM, which end whatever this one does)
    if (warp == kIssue) tc::tmem_alloc(&tmem_slot, S::kTmem);
    if (tid == 0) {
        for (int i = 0; i < kKeys; ++i) {
            // (fault test: one more signal for one block's keys than comes)
            tc::mbar_init(&bar.k_full[i], a.stall && blockIdx.x == 0 ? 5 : 4);
            tc::mbar_init(&bar.k_empty[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.s_empty[i], 4 * SPLIT);
        }
        for (int i = 0; i < kParts; ++i) tc::mbar_init(&bar.p_full[i], 4 * kSoft);
        tc::mbar_init(&bar.drain, 1);
        tc::fence_mbar_init();
        abort.flag = 0;
        abort.limit = (int)(a.spin / tc::kSpinTest);
    }
    tc::fence_before_sync();
    Place<kTok, kThreads> at;
    at.begin<false>(a, start, blockIdx.x, gridDim.x);  // (with barriers: the others' start, and the address of the tensor memory)
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    int done = 0, units = 0;  // chunks and tiles before this pass: the stages and their phases go on
    for (bool more = at.left > 0; more;) {
        const int cnt = (int)min(at.left, (long long)(at.steps - at.at)), n = at.n, c0 = at.at;
        const int rows = at.count * a.G;
        // Rows in passes: the first starts from what the tokens had, the others add to what is there.
        bool stop = false;
        for (int row0 = 0; row0 < max(rows, 1) && !stop; row0 += tiles * kCols) {
            const int here = max(0, min(rows - row0, tiles * kCols));     // rows of the pass
            const int padded = max(32, (here + 31) & ~31), nt = (padded + kCols - 1) / kCols;
            constexpr int PER = D / 16;
            auto factor = [&](int qe) { return fminf(a.scale * pow2(cache_exp(a, 0, at.h)) * pow2(-qe), 3.4028235e38f); };
            bool unusual = false;
            // Q, by the weights' warps: a thread has channels 4 x .. 4 x + 3 of each quarter of a row's
            for (int r = tid / PER; r < padded && warp < kWiden; r += 32 * kWiden / PER) {  // (a warp's rows: all or none)
                const int x = tid % PER;
                int t = 0;
                const bool in = r < here;
                const long long row = row_offset(a, at.b, at.h, row0 + min(r, max(here - 1, 0)), &t);
                uint32_t v[4][F ? 4 : 2], amax = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const T* p = Q + row * D + i * (D / 4) + 4 * x;
                    if (F) {
                        const uint4 u = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
                        v[i][0] = u.x; v[i][1] = u.y; v[i][F ? 2 : 0] = u.z; v[i][F ? 3 : 1] = u.w;
                        if (!F) continue;
                    } else {
                        const uint2 u = in ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
                        v[i][0] = u.x; v[i][1] = u.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < (F ? 4 : 2); ++j)
                        amax = max(amax, F ? v[i][j] & 0x7fffffffu
                                           : max(v[i][j] << 16 & 0x7fff0000u, v[i][j] & 0x7fff0000u));
#pragma unroll
                for (int i = 1; i < PER; i <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, i));
                float up = pow2(kUsual);
                int qe = kUsual;
                if (!usual_row(amax)) {
                    qe = query_exp(amax >> 23, &up);
                    unusual = true;
                }
                if (x == 0) {
                    fac[r] = factor(qe);
                    mlse[r] = in ? -w.lse[row] : -INFINITY;  // (a row that is not there: weights of 0)
                    lim[r] = in ? row_limit(a, n, at.count, t) : 0;
                }
                const uint32_t to = sm + (r / kCols) * kTile;
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // channels 4 x + 2 j and the next of each quarter
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y0 = __uint_as_float(F ? v[i][(2 * j) % (F ? 4 : 2)] : v[i][j] << 16) * up;
                        const float y1 = __uint_as_float(F ? v[i][(2 * j + 1) % (F ? 4 : 2)] : v[i][j] & 0xffff0000u) * up;
                        hi[i] = pack_half2(y0, y1);
                        const float2 h = half2_to_float2(hi[i]);
                        lo[i] = pack_half2(y0 - h.x, y1 - h.y);
                    }
                    const uint32_t off = tc::sw_off(r % kCols, 2 * x + j, kCols);
                    st_shared16(to + off, hi[0], hi[1], hi[2], hi[3]);
                    if (F) st_shared16(to + kHalf + off, lo[0], lo[1], lo[2], lo[3]);
                }
            }
            if (warp < kWiden || warp == kIssue) {
                tc::fence_proxy_async();
                unusual = any_but_widening<kWiden + 1>(unusual);
            }

            if (warp < kWiden) {
                // ------------------------------------------------ weights
                const int wg = warp >> 2, tl = 32 * quarter + lane;
                const int own0 = (wg - done) & (kSoft - 1);  // chunks whose sums the warpgroup stores: from here on, each kSoft-th
                const int low = here ? row_limit(a, n, at.count, row0 / a.G) : 0;  // keys that all rows of the pass see
                const long long sums = ((long long)at.b * a.Hkv + at.h) * w.cap + (long long)c0 * kTok + tl;
                const float* had = (row0 ? w.acc_out : w.acc) + sums;
                const float decay = row0 ? 1.0f : w.decay;
                // the thread's tokens with a sum, from the first chunk's on
                const int olds = (row0 ? n : w.decay != 0.0f ? n - at.count : 0) - (c0 * kTok + tl);
                auto look = [&](int i) {
                    const int c = own0 + kSoft * (i + (lane >> 1)), gi = 8 * (c0 + c) + 2 * quarter + (lane & 1);
                    return c < cnt && gi * kGroup < n ? cache_group(a, at.b, at.h, gi) : -1;
                };
                Groups groups;
                groups.start(look);
                const float same = factor(kUsual);
                // Adds to `sum` the weights of the thread's token tok from `share` rows, from r0 on, whose scores are in the
                // columns from `from` on of stage ss.
                auto weigh = [&](float2& sum, int ss, uint32_t from, int r0, int share, int tok, bool each) {
                    const uint32_t cols = tmem + ((uint32_t)quarter << 21) + ss * kCols + from;
#pragma unroll 1
                    for (int b0 = 0; b0 < share; b0 += 32, r0 += 32) {
                        const int here = min(32, share - b0);
                        float y[32];
                        if (here == 32) {
                            tc::tmem_ld32(cols + b0, y);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                if (i < here) tmem_ld8(cols + b0 + i, y + i);
                        }
                        wait_cols(y);
                        if (b0 + 32 >= share) {  // all are in registers
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&bar.s_empty[ss]);
                        }
                        auto some = [&](auto by_row, int i0, auto count) {
                            constexpr int kRows = decltype(count)::value;
                            float2 p[kRows / 2];
#pragma unroll
                            for (int j = 0; j < kRows; j += 4) {
                                const float4 l = *reinterpret_cast<const float4*>(mlse + r0 + i0 + j);
                                float4 f = make_float4(same, same, same, same);
                                if (decltype(by_row)::value) f = *reinterpret_cast<const float4*>(fac + r0 + i0 + j);
                                const float* z = y + i0 + j;
                                p[j / 2] = weight2(make_float2(z[0], z[1]), make_float2(f.x, f.y), make_float2(l.x, l.y));
                                p[j / 2 + 1] = weight2(make_float2(z[2], z[3]), make_float2(f.z, f.w), make_float2(l.z, l.w));
                                if (decltype(by_row)::value) {
                                    const int4 m = *reinterpret_cast<const int4*>(lim + r0 + i0 + j);
                                    if (tok >= m.x) p[j / 2].x = 0.0f;
                                    if (tok >= m.y) p[j / 2].y = 0.0f;
                                    if (tok >= m.z) p[j / 2 + 1].x = 0.0f;
                                    if (tok >= m.w) p[j / 2 + 1].y = 0.0f;
                                }
                            }
#pragma unroll
                            for (int o = kRows / 4; o; o >>= 1)
#pragma unroll
                                for (int j = 0; j < o; ++j) p[j] = add2(p[j], p[j + o]);
                            sum = add2(sum, p[0]);
                        };
                        if (here == 32 && !each) {
                            some(std::false_type(), 0, std::integral_constant<int, 16>());
                            some(std::false_type(), 16, std::integral_constant<int, 16>());
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                if (i >= here) continue;
                                if (each)
                                    some(std::true_type(), i, std::integral_constant<int, 8>());
                                else
                                    some(std::false_type(), i, std::integral_constant<int, 8>());
                            }
                        }
                    }
                };
                auto base_of = [&](int c) { return c < cnt && c * kTok < olds ? had[(long long)c * kTok] : 0.0f; };
                // some row does not see all of the chunk, or has a factor of its own
                auto each = [&](int c) { return unusual || (c0 + c + 1) * kTok > low; };
                auto store = [&](int c, int group, float base, float sum) {
                    if ((c0 + c) * kTok + tl < n && group >= 0) w.acc_out[sums + (long long)c * kTok] = fmaf(decay, base, sum);
                };
                if (SPLIT == 1) {
                    float base = base_of(own0);
                    for (int c = own0, i = 0; c < cnt; c += kSoft, ++i) {
                        const float next = base_of(c + kSoft);
                        const int group = groups.get(i, lane >> 4);
                        groups.step(i, look);
                        if (!warp_wait(&bar.s_full[wg], (done + c) / kSoft & 1, abort_v)) break;
                        tc::fence_after_sync();
                        float2 sum = make_float2(0.0f, 0.0f);
                        weigh(sum, wg, 0, 0, padded, (c0 + c) * kTok + tl, each(c));
                        store(c, group, base, sum.x + sum.y);
                        base = next;
                    }
                } else {
                    float base = 0.0f;  // of the chunk that the warpgroup will join
                    int u = units, joined = 0;
                    bool ok = true;
                    for (int c = 0; c <= cnt && ok; ++c) {  // (the last one only joins)
                        const int t = done + c;
                        if (c < cnt) {
                            float2 sum = make_float2(0.0f, 0.0f);
                            for (int ti = 0; ti < nt; ++ti, ++u) {
                                const int ss = u % kStages;
                                if (!(ok = warp_wait(&bar.s_full[ss], u / kStages & 1, abort_v))) break;
                                tc::fence_after_sync();
                                const int share = min(kCols, padded - ti * kCols) / SPLIT;
                                weigh(sum, ss, wg * share, ti * kCols + wg * share, share, (c0 + c) * kTok + tl, each(c));
                            }
                            if (!ok) break;
                            parts[t & (kParts - 1)][wg][tl] = sum.x + sum.y;
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&bar.p_full[t & (kParts - 1)]);
                        }
                        if (c > 0 && ((t - 1) & (kSoft - 1)) == wg) {
                            const int pb = (t - 1) & (kParts - 1), group = groups.get(joined, lane >> 4);
                            groups.step(joined++, look);
                            if (!(ok = warp_wait(&bar.p_full[pb], (t - 1) / kParts & 1, abort_v))) break;
                            const float* x = &parts[pb][0][tl];
                            store(c - 1, group, base, (x[0] + x[kTok]) + (x[2 * kTok] + x[3 * kTok]));
                        }
                        if ((t & (kSoft - 1)) == wg) base = base_of(c);
                    }
                }
            } else if (warp < kIssue) {
                // ----------------------------------------------- widening
                const int g = lane >> 2, t4 = lane & 3;
                const int codes = g * L::kRow + t4 * (D / 8), scales = L::kKs + g * (D / 8) + t4 * (D / 32);
                const uint32_t ring = raw + (warp - kWiden) * (kRaw * 18 * D);
                auto look = [&](int i) {
                    const int c = i + (lane >> 1), gi = 8 * (c0 + c) + 2 * quarter + (lane & 1);
                    return c < cnt && gi * kGroup < n ? cache_group(a, at.b, at.h, gi) : -1;
                };
                Groups groups;
                groups.start(look);
                // A lane copies what it will read itself (of d = 64 scales, what it and its neighbour will).
                auto copy = [&](int i) {  // called for every i in turn
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int grp = groups.get(i, y);
                        if (grp < 0) continue;
                        const uint8_t* src = cache + (unsigned long long)(unsigned)grp * L::kBytes;
                        const uint32_t dst = ring + (i % kRaw) * (18 * D) + y * (9 * D);
#pragma unroll
                        for (int x = 0; x < 2; ++x) copy_async<D / 8>(dst + codes + 8 * x * L::kRow, src + codes + 8 * x * L::kRow);
                        if (D == 128 || (t4 & 1) == 0) copy_async<4>(dst + scales, src + scales);
                    }
                    groups.step(i, look);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
#pragma unroll
                for (int i = 0; i < kRaw - 1; ++i) copy(i);
                for (int i = 0; i < cnt; ++i) {
                    const int t = done + i, st = t % kKeys;
                    asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 2) : "memory");
                    __syncwarp();
                    uint32_t code[2][2][W], sc[2];  // [group][token g, g + 8]
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t src = ring + (i % kRaw) * (18 * D) + y * (9 * D);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t p = src + codes + 8 * x * L::kRow;
                            if (D == 128)
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(code[y][x][0]), "=r"(code[y][x][1]), "=r"(code[y][x][W - 2]), "=r"(code[y][x][W - 1])
                                             : "r"(p));
                            else
                                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(code[y][x][0]), "=r"(code[y][x][1]) : "r"(p));
                        }
                        if (D == 128)
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc[y]) : "r"(src + scales));
                        else
                            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc[y]) : "r"(src + scales));
                    }
                    copy(i + kRaw - 1);  // (over the stage that all lanes read before the last barrier)
                    if (!warp_wait(&bar.k_empty[st], ((t / kKeys) & 1) ^ 1, abort_v)) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t s2[2][2];  // [token g, g + 8][16 of the lane's channels]: scales, each in both halves
                        if (D == 128) {
                            const uint32_t a0 = e4m3x2_to_half2(sc[y] & 0xffff), a1 = e4m3x2_to_half2(sc[y] >> 16);
                            s2[0][0] = __byte_perm(a0, a0, 0x1010);
                            s2[0][1] = __byte_perm(a0, a0, 0x3232);
                            s2[1][0] = __byte_perm(a1, a1, 0x1010);
                            s2[1][1] = __byte_perm(a1, a1, 0x3232);
                        } else {
                            const uint32_t a0 = e4m3x2_to_half2(sc[y]);
                            s2[0][0] = __byte_perm(a0, a0, 0x1010);
                            s2[1][0] = __byte_perm(a0, a0, 0x3232);
                        }
                        const uint32_t to = tmem + ((uint32_t)quarter << 21) + ((uint32_t)y << 20) + kK + st * 64;
#pragma unroll
                        for (int wi = 0; wi < W; ++wi) {
                            uint32_t h[8];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                uint32_t k4[4];
                                e2m1x8_to_half2(code[y][x][wi], k4);
#pragma unroll
                                for (int j = 0; j < 4; ++j) h[2 * j + x] = hmul2(k4[j], s2[x][wi / 2]);
                            }
                            tmem_st_frag(to + 16 * wi, h);
                        }
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.k_full[st]);
                }
                tc::cp_async_wait_all();
            } else {
                // ----------------------------------------------- products
                bool ok = true;
                for (int c = 0; c < cnt && ok; ++c) {
                    const int t = done + c, st = t % kKeys;
                    if (!(ok = warp_wait(&bar.k_full[st], (t / kKeys) & 1, abort_v))) break;
                    for (int ti = 0; ti < nt; ++ti) {
                        const int u = units + c * nt + ti, ss = u % kStages;
                        if (!(ok = warp_wait(&bar.s_empty[ss], u / kStages & 1 ^ 1, abort_v))) break;
                        tc::fence_after_sync();
                        const uint32_t id = idesc_half(kTok, min(kCols, padded - ti * kCols), 0, 0);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < (F ? 2 : 1) * KS; ++k)  // 16 channels each; lower halves first: sums are cut to 24 bits
                                tc::mma_bf16_ts(tmem + ss * kCols, tmem + kK + st * 64 + (k % KS) * 8,
                                                tc::sdesc(sm + ti * kTile + (F && k < KS) * kHalf + (k % KS >> 2) * (kCols * 128) +
                                                              (k & 3) * 32,
                                                          16, 1024),
                                                id, k > 0);
                            tc::mma_commit(&bar.s_full[ss]);
                            if (ti == nt - 1) tc::mma_commit(&bar.k_empty[st]);
                        }
                        __syncwarp();
                    }
                }
            }
            done += cnt;
            units += cnt * nt;
            // every warp is through the pass, so that all see the same and the rows' memory is free
            tc::fence_before_sync();
            stop = __syncthreads_or(abort.flag);
            tc::fence_after_sync();
        }
        if (stop) break;
        more = at.next(a, cnt);
    }
    wait_previous();  // the status word is there
    // what is in flight lands before the block frees its tensor memory and ends
    if (warp == kIssue && lane == 0) {
        tc::mma_commit(&bar.drain);
        drain(&bar.drain, 0, a.status, a.spin);
        if (abort.flag) set_status(a.status, kStTimeout);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kIssue) tc::tmem_dealloc(tmem, S::kTmem);
}

// ------------------------------------------------------------------ launch

template <typename T, int D, int SPLIT>
static cudaError_t split_t(const CacheArgs& a, const WeighArgs& w, const void* Q, const uint8_t* cache, cudaStream_t st) {
    // rows of a pass: as many as there are, as far as they fit (24 KB are static)
    using S = Tiles<SPLIT>;
    constexpr int kCols = S::kCols, kBytes = tile_bytes<T, D, kCols>();
    constexpr int kMost = SPLIT == 1 ? 1 : ((227 - 24) * 1024 - 1024 - raw_bytes<D>()) / kBytes;
    const long long rows = (long long)a.G * a.T;
    const int tiles = (int)std::min<long long>(kMost, (rows + kCols - 1) / kCols);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = set_smem_once((const void*)k_cache_weigh_tile<T, D, SPLIT>, kMost * kBytes + raw_bytes<D>() + 1024, &done);
    if (e != cudaSuccess) return e;
    k_cache_weigh_begin<<<1, 256, 0, st>>>(a);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long chunks = (long long)a.B * a.Hkv * ((w.cap + kTok - 1) / kTok);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    // (one SM has the kernel before it)
    c.gridDim = dim3((unsigned)std::min<long long>(chunks, S::kBlocks * num_sms() - 1));
    c.blockDim = dim3(S::kThreads);
    c.dynamicSmemBytes = tiles * kBytes + raw_bytes<D>() + 1024;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, k_cache_weigh_tile<T, D, SPLIT>, a, w, (const T*)Q, cache, tiles);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T, int D>
static cudaError_t tile_t(const CacheArgs& a, const WeighArgs& w, const void* Q, const uint8_t* cache, cudaStream_t st) {
    return (long long)a.G * a.T <= Tiles<1>::kCols ? split_t<T, D, 1>(a, w, Q, cache, st) : split_t<T, D, 4>(a, w, Q, cache, st);
}

cudaError_t launch_cache_weigh_tile(const CacheArgs& a, const WeighArgs& w, int d, int dtype, const void* Q,
                                    const uint8_t* cache, cudaStream_t st) {
    if (dtype == 0) return d == 64 ? tile_t<float, 64>(a, w, Q, cache, st) : tile_t<float, 128>(a, w, Q, cache, st);
    return d == 64 ? tile_t<__nv_bfloat16, 64>(a, w, Q, cache, st) : tile_t<__nv_bfloat16, 128>(a, w, Q, cache, st);
}

}  // namespace mita
