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
// row and key, so with few rows per cache head it is bound by HBM.
//
// Work split. An item is one (sequence, tile of query rows, cache head); it is
// cut into chunks of 128 tokens. The chunks of all items form one line, and the
// line is cut into equal pieces, one per block: lengths that differ from
// sequence to sequence balance by themselves, and one long sequence spreads
// over the whole GPU. A block that has all of an item's chunks writes its rows;
// one that has a part writes the unnormalized sums, and k_cache_join adds the
// parts. Everything is derived from the lengths on the device, so a captured
// call follows them when it is replayed.
#include <limits.h>

#include <algorithm>

#include "cache.cuh"

namespace mita {

constexpr int kChunk = 128;    // tokens of a block's step
constexpr int kStep = 32;      // tokens of a warp's step (4 warps)
constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnOut {
    void* O;
    float* lse;    // or null
    float* part;   // [2 * pieces][rows][d]
    float2* ml;    // [2 * pieces][rows] (maximum in log2 units, sum)
    int pieces;
};

// Chunks of sequence b: (row tiles) * Hkv * (chunks of its length).
struct SeqWork {
    int rows, tiles, chunks;
    long long total;
};
__device__ __forceinline__ SeqWork seq_work(const CacheArgs& a, int b, int rtile) {
    SeqWork s;
    s.rows = cache_count(a, b) * a.G;
    s.tiles = (s.rows + rtile - 1) / rtile;
    s.chunks = max(1, (cache_len(a, b) + kChunk - 1) / kChunk);
    s.total = (long long)s.tiles * a.Hkv * s.chunks;
    return s;
}

// The line of chunks: piece c is [at(c), at(c + 1)).
struct Line {
    long long total;
    __device__ __forceinline__ long long at(long long c, int pieces) const { return c * total / pieces; }
};

// Block-wide: the sequence that holds chunk w of the line and the chunks before
// that sequence. All threads call it and get the same answer; *total is set
// when asked for (w < 0 asks for the total only).
__device__ __forceinline__ void line_find(const CacheArgs& a, int rtile, long long w, long long* tmp, long long* total,
                                          int* seq, long long* before) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        const long long mine = b < a.B ? seq_work(a, b, rtile).total : 0;
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();  // the previous tile's tmp has been read
        if (lane == 31) tmp[wid] = x;
        __syncthreads();
        long long off = base;
        for (int i = 0; i < wid; ++i) off += tmp[i];
        x += off;  // inclusive
        if (w >= 0 && mine > 0 && w < x && w >= x - mine) {
            tmp[5] = x - mine;
            tmp[6] = b;
        }
        for (int i = 0; i < kThreads / 32; ++i) base += tmp[i];
    }
    __syncthreads();
    if (w < 0) {
        *total = base;
    } else {
        *before = tmp[5];
        *seq = (int)tmp[6];
    }
    __syncthreads();
}

// One block's part of an item.
struct Segment {
    int b, h, row0, rows;  // sequence, cache head, first row and rows of the tile
    int c0, c1, chunks;    // chunks [c0, c1) of the item's `chunks`
    long long start;       // the item's first chunk on the line
};

// Segment that begins at chunk w (in sequence b, `before` chunks before it) and ends
// at w1 or at the item's end.
__device__ __forceinline__ Segment segment_at(const CacheArgs& a, int rtile, const SeqWork& s, int b, long long before,
                                              long long w, long long w1) {
    Segment g;
    const long long rel = w - before, item = rel / s.chunks;
    g.b = b;
    g.start = before + item * s.chunks;
    const int tile = (int)(item / a.Hkv);
    g.h = (int)(item - (long long)tile * a.Hkv);
    g.row0 = tile * rtile;
    g.rows = min(rtile, s.rows - g.row0);
    g.chunks = s.chunks;
    g.c0 = (int)(rel - item * s.chunks);
    g.c1 = (int)min((long long)s.chunks, w1 - g.start);
    return g;
}

// Row r of a sequence: token r / G of the call, query head h G + r % G.
__device__ __forceinline__ long long row_offset(const CacheArgs& a, int b, int h, int r, int* t) {
    *t = r / a.G;
    return ((long long)(b * a.H + h * a.G + (r - *t * a.G)) * a.T + *t);
}
// Keys that token t of the call sees.
__device__ __forceinline__ int row_limit(const CacheArgs& a, int n, int count, int t) {
    return a.causal ? max(n - (count - 1 - t), 0) : n;
}

// ------------------------------------------------------ staging of groups

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The groups of a warp's steps in a segment: step i is the 32 tokens from
// (c0 + i) * 128 + 32 * warp on, two groups. Lane l holds the group number of
// group l & 1 of step l >> 1 in the current run of 16 steps; the next run's
// table entries are loaded a run ahead.
struct GroupRun {
    int cur, nxt;
    __device__ __forceinline__ static int load(const CacheArgs& a, const Segment& s, int n, int warp, int lane, int i0) {
        const int step = i0 + (lane >> 1);
        const int gi = ((s.c0 + step) * kChunk + warp * kStep) / kGroup + (lane & 1);
        return s.c0 + step < s.c1 && gi * kGroup < n ? cache_group(a, s.b, s.h, gi) : -1;
    }
    __device__ __forceinline__ void begin(const CacheArgs& a, const Segment& s, int n, int warp, int lane) {
        cur = load(a, s, n, warp, lane, 0);
        nxt = load(a, s, n, warp, lane, 16);
    }
    // group g of step i; called once per step, in order
    __device__ __forceinline__ int get(int i, int g) const { return __shfl_sync(0xffffffffu, cur, 2 * (i & 15) + g); }
    __device__ __forceinline__ void advance(const CacheArgs& a, const Segment& s, int n, int warp, int lane, int i) {
        if ((i & 15) == 15) {
            cur = nxt;
            nxt = load(a, s, n, warp, lane, i + 17);
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
            copy16(dst + k * 16, cache + (long long)max(g, 0) * Grp<D>::kBytes + (k < N ? k : k - N) * 16, g >= 0);
        }
    }
    copy_commit();
}

// ------------------------------------------------------------ CUDA cores

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

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
    __shared__ long long tmp[8];
    if (blockIdx.x == 0) {
        cache_check_call(a, false);
        return;
    }
    const int piece = blockIdx.x - 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> 3, ch = lane & 7;  // token of four, chunk
    long long total, before;
    line_find(a, R, -1, tmp, &total, nullptr, nullptr);
    const Line line{total};
    long long w = line.at(piece, out.pieces);
    const long long w_begin = w, w_end = line.at(piece + 1, out.pieces);
    if (w >= w_end) return;
    int b;
    line_find(a, R, w, tmp, &total, &b, &before);
    SeqWork sw = seq_work(a, b, R);
    uint8_t* ring = smem + warp * (kSimtStages * 2 * L::kBytes);
    const uint32_t ring_addr = smem_addr(ring);

    while (w < w_end) {
        while (w >= before + sw.total) {  // next sequence with work
            before += sw.total;
            sw = seq_work(a, ++b, R);
        }
        const Segment s = segment_at(a, R, sw, b, before, w, w_end);
        const int n = cache_len(a, b), count = cache_count(a, b);
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
                q[r][i] = to_float(Q[at + i]);
                o[r][i] = 0.0f;
            }
        }
        const int steps = s.c1 - s.c0;
        GroupRun gr;
        gr.begin(a, s, min(n, top), warp, lane);
        int issued = 0;
        for (; issued < kSimtStages - 1; ++issued) {
            const int g0 = gr.get(issued, 0), g1 = gr.get(issued, 1);
            if (issued < steps) stage_step<D>(cache, ring_addr + issued * 2 * L::kBytes, g0, g1, lane); else copy_commit();
            gr.advance(a, s, min(n, top), warp, lane, issued);
        }
        for (int i = 0; i < steps; ++i) {
            const int nx = i + kSimtStages - 1;
            const int g0 = gr.get(nx, 0), g1 = gr.get(nx, 1);
            __syncwarp();
            if (nx < steps) stage_step<D>(cache, ring_addr + (nx % kSimtStages) * 2 * L::kBytes, g0, g1, lane); else copy_commit();
            gr.advance(a, s, min(n, top), warp, lane, nx);
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
        const bool whole = s.c0 == 0 && s.c1 == s.chunks;
        const int slot = 2 * piece + (w == w_begin ? 0 : 1);
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
        __syncthreads();
        w = s.start + s.c1;
    }
}

// ------------------------------------------------------------------ join

// Block (c, y), c >= 1: if piece c's first chunk lies inside an item and is the
// first such cut of it, joins that item's parts; each of the four warps takes a
// row of the four rows from 4 y on. Piece c - 1 has the item's first chunk.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads) k_cache_join(CacheArgs a, AttnOut out) {
    __shared__ long long tmp[8];
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long total, before;
    line_find(a, R, -1, tmp, &total, nullptr, nullptr);
    const Line line{total};
    const long long w = line.at(c, out.pieces), wp = line.at(c - 1, out.pieces);
    if (w >= total) return;
    int b;
    line_find(a, R, w, tmp, &total, &b, &before);
    const SeqWork sw = seq_work(a, b, R);
    const Segment s = segment_at(a, R, sw, b, before, w, total);
    if (s.c0 == 0 || wp > s.start) return;
    const int r = blockIdx.y * 4 + warp;
    if (r >= s.rows) return;
    const long long end = s.start + s.chunks;
    float mx = -INFINITY, sum = 0.0f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
    for (int p = c - 1; p < out.pieces && line.at(p, out.pieces) < end; ++p) {
        const long long wb = line.at(p, out.pieces);
        if (wb == line.at(p + 1, out.pieces)) continue;  // an empty piece
        const long long at = (2LL * p + (wb >= s.start ? 0 : 1)) * R + r;
        const float2 ml = out.ml[at];
        const float mn = fmaxf(mx, ml.x), ref = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2f(mx - ref), fp = exp2f(ml.x - ref);
        mx = mn;
        sum = sum * f + ml.y * fp;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = acc[i] * f + out.part[at * D + lane * (D / 32) + i] * fp;
    }
    int t;
    const long long at = row_offset(a, b, s.h, s.row0 + r, &t);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        reinterpret_cast<T*>(out.O)[at * D + lane * (D / 32) + i] = from_f<T>(sum == 0.0f ? 0.0f : acc[i] * inv);
    if (out.lse && lane == 0) out.lse[at] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ launch

// Rows of a tile: one (a single row per cache head) or four.
static int simt_rows(const CacheArgs& a) { return (long long)a.G * a.T == 1 ? 1 : 4; }

static long long max_chunks(const CacheArgs& a, int rtile) {
    const long long tiles = ((long long)a.G * a.T + rtile - 1) / rtile;
    const long long len = ((long long)a.cols * a.page + kChunk - 1) / kChunk;
    return (long long)a.B * a.Hkv * tiles * len;
}

CachePlan cache_attn_plan(const CacheArgs& a, int d, int dtype, unsigned flags) {
    CachePlan p;
    p.rows = simt_rows(a);
    // four blocks per SM, one of them the check of the call's indexes
    p.pieces = (int)std::min<long long>(4LL * num_sms() - 1, max_chunks(a, p.rows));
    p.parts = (size_t)2 * p.pieces * p.rows;
    return p;
}

template <typename T, int D, int R>
static cudaError_t simt_t(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st) {
    constexpr int smem = simt_smem<D, R>();
    cudaError_t e = cudaFuncSetAttribute(k_cache_attn_simt<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_cache_attn_simt<T, D, R><<<o.pieces + 1, kThreads, smem, st>>>(a, (const T*)Q, cache, o);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess || o.pieces == 1) return e;
    prof_mark(st, "cache_join");
    k_cache_join<T, D, R><<<dim3(o.pieces - 1, (R + 3) / 4), kThreads, 0, st>>>(a, o);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t attn_t(const CacheArgs& a, const CachePlan& p, const void* Q, const uint8_t* cache,
                          const AttnOut& o, cudaStream_t st) {
    return p.rows == 1 ? simt_t<T, D, 1>(a, Q, cache, o, st) : simt_t<T, D, 4>(a, Q, cache, o, st);
}

cudaError_t launch_cache_attn(const CacheArgs& a, const CachePlan& p, int d, int dtype, const void* Q,
                              const void* cache, void* O, float* lse, float* part, float2* ml, cudaStream_t st) {
    const AttnOut o{O, lse, part, ml, p.pieces};
    const uint8_t* c = (const uint8_t*)cache;
    prof_mark(st, "cache_attention");
    if (dtype == 0) return d == 64 ? attn_t<float, 64>(a, p, Q, c, o, st) : attn_t<float, 128>(a, p, Q, c, o, st);
    return d == 64 ? attn_t<__nv_bfloat16, 64>(a, p, Q, c, o, st) : attn_t<__nv_bfloat16, 128>(a, p, Q, c, o, st);
}

}  // namespace mita
