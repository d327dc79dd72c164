// The attention weight of cached tokens for many rows per cache head (a prompt's last
// tokens, drafted tokens of grouped queries): tiles of 128 tokens by up to 128 rows on tcgen05.
// (cache_weigh.cu has the mathematics and the form for few rows.)
//
//   S = K Q^T    128 tokens x N rows: K widened to halves in tensor memory, Q a K-major tile in
//                shared memory, fp32 in tensor memory
//
// A lane of tensor memory is a token, so a thread has a token's scores with all rows: it adds up their weights
// by itself, and nothing is exchanged between threads. What a token costs is then one exponential per row
// and the four or so instructions around it; keys are widened once for all rows of a pass.
//
// Keys go from memory to registers in the order of m16n8k16's A (the cache's own order: neighbouring lanes
// read neighbouring bytes) and from there to tensor memory by 16 x 128 bit stores, which puts the
// channels of a token in the order {t d/4 + 2 m, t d/4 + 2 m + 1 : t = 0 .. 3} for m = 0, 1, ...; Q's rows are stored in
// the same order.
//
// Warps: three warpgroups for the weights, each with a stage of scores and every third chunk of 128 tokens; eight
// warps widen keys, four at a time a chunk, each the quarter of the lanes that it can reach; one issues the products.
// Every wait is bounded; a block that gives up raises its abort flag, lets its products land, frees its
// tensor memory and says so in the status word.
#include <algorithm>
#include <type_traits>

#include "cache_tc.cuh"
#include "cache_weigh.cuh"

namespace mita {

namespace {

constexpr int kTok = 128, kCols = 128;           // tokens of a chunk; rows of a tile
constexpr int kSoft = 3;                         // warpgroups for the weights, and stages of scores
constexpr int kWiden = 4 * kSoft, kIssue = kWiden + 8;  // first warps of the other roles
constexpr int kThreads = 32 * (kIssue + 1);
constexpr int kAhead = 2;                        // chunks of its own that a widening warp's loads are ahead
constexpr uint32_t kK = kSoft * kCols;           // column of the first of two stages of keys

// Scores are announced to the warpgroup that waits for them, not by stage: a warpgroup does not use every stage in
// turn, and a barrier that it had not looked at for two phases would look done. It has at
// most kSoft tiles to come, so that of kReady barriers in turn each is at most one phase ahead.
constexpr int kReady = 4;
static_assert(kReady > kSoft, "a barrier would be two phases ahead");
struct WeighBars {
    uint64_t k_full[2], k_empty[2], s_full[kSoft][kReady], s_empty[kSoft], drain;
};

// Bytes of a tile's rows: as halves (two for float rows), factors and log sums, limits.
template <typename T, int D> constexpr int tile_bytes() { return kCols * (D * 2 * (sizeof(T) == 4 ? 2 : 1) + 8 + 4); }

// Groups of a role's own chunks, `every` apart: lane l looks up group 2 quarter + l % 2 of chunk i + l / 2.
struct Groups {
    int cur, nxt;
    template <typename Look> __device__ __forceinline__ void start(Look look) {
        cur = look(0);
        nxt = look(16);
    }
    // called for every i in turn
    template <typename Look> __device__ __forceinline__ int get(int i, int y, Look look) {
        const int g = __shfl_sync(0xffffffffu, cur, 2 * (i & 15) + y);
        return g;
    }
    template <typename Look> __device__ __forceinline__ void step(int i, Look look) {
        if ((i & 15) != 15) return;
        cur = nxt;
        nxt = look(i + 17);
    }
};

// The loads into v have arrived.
__device__ __forceinline__ void wait_cols(float* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_cache_weigh_tile(CacheArgs a, WeighArgs w, const T* __restrict__ Q, const uint8_t* __restrict__ cache, int tiles) {
    using L = Grp<D>;
    constexpr bool F = sizeof(T) == 4;  // float rows: two halves, hi + lo
    constexpr int KS = D / 16, W = D / 32, KW = D / 64, kHalf = kCols * D * 2, kTile = (F ? 2 : 1) * kHalf;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sm = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* smp = smem_raw + (sm - tc::smem_u32(smem_raw));
    // of two rows each: factors of the scores, log sums negated
    float4* ref = reinterpret_cast<float4*>(smp + tiles * kTile);
    int* lim = reinterpret_cast<int*>(ref + tiles * (kCols / 2));  // keys that a row sees
    __shared__ LineStart<kThreads> start;
    __shared__ WeighBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ Abort abort;
    volatile Abort* abort_v = &abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
    // (waits for another kernel's blocks on this SM, which end whatever this one does)
    if (warp == kIssue) tc::tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            // (fault test: one more signal for one block's keys than comes)
            tc::mbar_init(&bar.k_full[i], a.stall && blockIdx.x == 0 ? 5 : 4);
            tc::mbar_init(&bar.k_empty[i], 1);
        }
        for (int i = 0; i < kSoft; ++i) {
            for (int j = 0; j < kReady; ++j) tc::mbar_init(&bar.s_full[i][j], 1);
            tc::mbar_init(&bar.s_empty[i], 4);
        }
        tc::mbar_init(&bar.drain, 1);
        tc::fence_mbar_init();
        abort.flag = 0;
        abort.limit = (int)(a.spin / tc::kSpinTest);
    }
    tc::fence_before_sync();
    Place<kTok, kThreads> at;
    at.begin(a, start, blockIdx.x, gridDim.x);
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    int done = 0, units = 0;  // chunks and tiles before this pass: the stages and their phases go on
    uint32_t turn = 0;        // tiles that a warpgroup has had; of the issuing warp: a byte for each warpgroup
    for (bool more = at.left > 0; more;) {
        const int cnt = (int)min(at.left, (long long)(at.steps - at.at)), n = at.n, c0 = at.at;
        const int rows = at.count * a.G;
        // Rows in passes: the first starts from what the tokens had, the others add to what is there.
        bool stop = false;
        for (int row0 = 0; row0 < max(rows, 1) && !stop; row0 += tiles * kCols) {
            const int here = max(0, min(rows - row0, tiles * kCols));     // rows of the pass
            const int padded = max(16, (here + 15) & ~15), nt = (padded + kCols - 1) / kCols;
            // Q: a thread has channels 4 x .. 4 x + 3 of each quarter of a row's
            constexpr int PER = D / 16;
            for (int r = tid / PER; r < padded; r += kThreads / PER) {  // (a warp's rows: all or none)
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
                float up;
                const int qe = query_exp(amax >> 23, &up);
                if (x == 0) {
                    float* f = reinterpret_cast<float*>(ref + (r >> 1)) + (r & 1);
                    f[0] = fminf(a.scale * pow2(cache_exp(a, 0, at.h)) * pow2(-qe), 3.4028235e38f);
                    f[2] = in ? -w.lse[row] : -INFINITY;  // (a row that is not there: weights of 0)
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
            tc::fence_proxy_async();
            __syncthreads();

            if (warp < kWiden) {
                // ------------------------------------------------ weights
                const int wg = warp >> 2, first = ((wg - done) % kSoft + kSoft) % kSoft, tl = 32 * quarter + lane;
                const int low = here ? row_limit(a, n, at.count, row0 / a.G) : 0;  // keys that all rows of the pass see
                const long long sums = ((long long)at.b * a.Hkv + at.h) * w.cap + (long long)c0 * kTok + tl;
                const float* had = (row0 ? w.acc_out : w.acc) + sums;
                const float decay = row0 ? 1.0f : w.decay;
                // the thread's tokens with a sum, from the first chunk's on
                const int olds = (row0 ? n : w.decay != 0.0f ? n - at.count : 0) - (c0 * kTok + tl);
                auto base_of = [&](int c) { return c < cnt && c * kTok < olds ? had[(long long)c * kTok] : 0.0f; };
                auto look = [&](int i) {
                    const int c = first + kSoft * (i + (lane >> 1)), gi = 8 * (c0 + c) + 2 * quarter + (lane & 1);
                    return c < cnt && gi * kGroup < n ? cache_group(a, at.b, at.h, gi) : -1;
                };
                const uint32_t cols = tmem + ((uint32_t)quarter << 21);
                Groups groups;
                groups.start(look);
                float base = base_of(first);
                for (int c = first, i = 0; c < cnt; c += kSoft, ++i) {
                    const float next = base_of(c + kSoft);
                    const int group = groups.get(i, lane >> 4, look);
                    groups.step(i, look);
                    const int tok = (c0 + c) * kTok + tl;
                    const bool edge = (c0 + c + 1) * kTok > low;  // some row does not see all of the chunk
                    float2 sum = make_float2(0.0f, 0.0f);
                    bool ok = true;
                    for (int ti = 0; ti < nt; ++ti) {
                        const int ss = (units + c * nt + ti) % kSoft;
                        if (!(ok = warp_wait(&bar.s_full[wg][turn % kReady], turn / kReady & 1, abort_v))) break;
                        ++turn;
                        tc::fence_after_sync();
                        const int nb = min(kCols, padded - ti * kCols) / 16;  // blocks of 16 columns
                        const float4* rf = ref + ti * (kCols / 2);
                        float y[2][16];
                        tmem_ld16(cols + ss * kCols, y[0]);
                        auto block = [&](auto masked, int bi, float* now, float* then) {
                            wait_cols(now);
                            if (bi + 1 < nb) {
                                tmem_ld16(cols + ss * kCols + 16 * (bi + 1), then);
                            } else {  // all of the stage is in registers
                                tc::fence_before_sync();
                                __syncwarp();
                                if (lane == 0) tc::mbar_arrive(&bar.s_empty[ss]);
                            }
                            float2 p[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 r = rf[8 * bi + j];
                                p[j] = weight2(make_float2(now[2 * j], now[2 * j + 1]), make_float2(r.x, r.y),
                                               make_float2(r.z, r.w));
                            }
                            if (decltype(masked)::value) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const int2 m = reinterpret_cast<const int2*>(lim)[ti * (kCols / 2) + 8 * bi + j];
                                    if (tok >= m.x) p[j].x = 0.0f;
                                    if (tok >= m.y) p[j].y = 0.0f;
                                }
                            }
#pragma unroll
                            for (int o = 4; o; o >>= 1)
#pragma unroll
                                for (int j = 0; j < o; ++j) p[j] = add2(p[j], p[j + o]);
                            sum = add2(sum, p[0]);
                        };
                        auto tile = [&](auto masked) {
#pragma unroll 1
                            for (int bi = 0; bi < nb; bi += 2) {
                                block(masked, bi, y[0], y[1]);
                                if (bi + 1 < nb) block(masked, bi + 1, y[1], y[0]);
                            }
                        };
                        if (edge)
                            tile(std::true_type());
                        else
                            tile(std::false_type());
                    }
                    if (!ok) break;
                    if (tok < n && group >= 0) w.acc_out[sums + (long long)c * kTok] = fmaf(decay, base, sum.x + sum.y);
                    base = next;
                }
            } else if (warp < kIssue) {
                // ----------------------------------------------- widening
                const int st = (warp - kWiden) >> 2, first = (st - done) & 1, g = lane >> 2, t4 = lane & 3;
                const uint8_t* codes = cache + g * L::kRow + t4 * (D / 8);
                const uint8_t* scales = cache + L::kKs + g * (D / 8) + t4 * (D / 32);
                auto look = [&](int i) {
                    const int c = first + 2 * (i + (lane >> 1)), gi = 8 * (c0 + c) + 2 * quarter + (lane & 1);
                    return c < cnt && gi * kGroup < n ? cache_group(a, at.b, at.h, gi) : -1;
                };
                Groups groups;
                groups.start(look);
                uint2 kc[kAhead][2][2][KW];  // [chunk][group][token g, g + 8]
                uint32_t sc[kAhead][2];
                auto load = [&](int u, int i) {  // called for every i in turn
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int grp = groups.get(i, y, look);
                        sc[u][y] = 0;  // (tokens that are not there: zeros)
                        if (grp < 0) continue;
                        const unsigned long long to = (unsigned long long)(unsigned)grp * L::kBytes;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint8_t* r = codes + to + 8 * x * L::kRow;
                            if (D == 128) {
                                const uint4 v = *reinterpret_cast<const uint4*>(r);
                                kc[u][y][x][0] = make_uint2(v.x, v.y);
                                kc[u][y][x][KW - 1] = make_uint2(v.z, v.w);
                            } else {
                                kc[u][y][x][0] = *reinterpret_cast<const uint2*>(r);
                            }
                        }
                        sc[u][y] = D == 128 ? *reinterpret_cast<const uint32_t*>(scales + to)
                                            : *reinterpret_cast<const uint16_t*>(scales + to);
                    }
                    groups.step(i, look);
                };
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int k = 0; k < KW; ++k) kc[u][y][x][k] = make_uint2(0, 0);
                    load(u, u);
                }
                bool ok = true;
                for (int c = first, i = 0; c < cnt && ok; i += kAhead) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u, c += 2) {
                        if (c >= cnt || !ok) continue;
                        const int t = done + c;
                        if (!(ok = warp_wait(&bar.k_empty[st], ((t >> 1) & 1) ^ 1, abort_v))) continue;
                        tc::fence_after_sync();
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t s2[2][KW];  // [token g, g + 8]: scales, each in both halves
                            if (D == 128) {
                                const uint32_t a0 = e4m3x2_to_half2(sc[u][y] & 0xffff), a1 = e4m3x2_to_half2(sc[u][y] >> 16);
                                s2[0][0] = __byte_perm(a0, a0, 0x1010);
                                s2[0][KW - 1] = __byte_perm(a0, a0, 0x3232);
                                s2[1][0] = __byte_perm(a1, a1, 0x1010);
                                s2[1][KW - 1] = __byte_perm(a1, a1, 0x3232);
                            } else {
                                const uint32_t a0 = e4m3x2_to_half2(sc[u][y]);
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
                                    e2m1x8_to_half2(wi & 1 ? kc[u][y][x][wi / 2].y : kc[u][y][x][wi / 2].x, k4);
#pragma unroll
                                    for (int j = 0; j < 4; ++j) h[2 * j + x] = hmul2(k4[j], s2[x][wi / 2]);
                                }
                                tmem_st_frag(to + 16 * wi, h);
                            }
                        }
                        load(u, i + u + kAhead);
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&bar.k_full[st]);
                    }
                }
            } else {
                // ----------------------------------------------- products
                bool ok = true;
                for (int c = 0; c < cnt && ok; ++c) {
                    const int t = done + c, st = t & 1;
                    if (!(ok = warp_wait(&bar.k_full[st], (t >> 1) & 1, abort_v))) break;
                    for (int ti = 0; ti < nt; ++ti) {
                        const int u = units + c * nt + ti, ss = u % kSoft;
                        if (!(ok = warp_wait(&bar.s_empty[ss], u / kSoft & 1 ^ 1, abort_v))) break;
                        tc::fence_after_sync();
                        const uint32_t id = idesc_half(kTok, min(kCols, padded - ti * kCols), 0, 0);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < (F ? 2 : 1) * KS; ++k)  // 16 channels each
                                tc::mma_bf16_ts(tmem + ss * kCols, tmem + kK + st * 64 + (k % KS) * 8,
                                                tc::sdesc(sm + ti * kTile + (k / KS) * kHalf + (k % KS >> 2) * (kCols * 128) +
                                                              (k & 3) * 32,
                                                          16, 1024),
                                                id, k > 0);
                            tc::mma_commit(&bar.s_full[t % kSoft][turn >> 8 * (t % kSoft) & (kReady - 1)]);
                            if (ti == nt - 1) tc::mma_commit(&bar.k_empty[st]);
                        }
                        __syncwarp();
                        turn = __vadd4(turn, 1u << 8 * (t % kSoft));
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
    if (warp == kIssue) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ launch

template <typename T, int D>
static cudaError_t tile_t(const CacheArgs& a, const WeighArgs& w, const void* Q, const uint8_t* cache, cudaStream_t st) {
    // rows of a pass: as many as there are, within 150 KB
    constexpr int kMost = 150 * 1024 / tile_bytes<T, D>();
    const long long rows = (long long)a.G * a.T;
    const int tiles = (int)std::min<long long>(kMost, (rows + kCols - 1) / kCols);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = set_smem_once((const void*)k_cache_weigh_tile<T, D>, kMost * tile_bytes<T, D>() + 1024, &done);
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
    c.gridDim = dim3((unsigned)std::min<long long>(chunks, num_sms() - 1));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = tiles * tile_bytes<T, D>() + 1024;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, k_cache_weigh_tile<T, D>, a, w, (const T*)Q, cache, tiles);
    if (e == cudaSuccess) count_launch();
    return e;
}

cudaError_t launch_cache_weigh_tile(const CacheArgs& a, const WeighArgs& w, int d, int dtype, const void* Q,
                                    const uint8_t* cache, cudaStream_t st) {
    if (dtype == 0) return d == 64 ? tile_t<float, 64>(a, w, Q, cache, st) : tile_t<float, 128>(a, w, Q, cache, st);
    return d == 64 ? tile_t<__nv_bfloat16, 64>(a, w, Q, cache, st) : tile_t<__nv_bfloat16, 128>(a, w, Q, cache, st);
}

}  // namespace mita
