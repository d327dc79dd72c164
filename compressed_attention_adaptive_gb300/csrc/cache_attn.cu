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
#include "tc.cuh"

namespace mita {

constexpr int kChunk = 128;    // tokens of a block's step
constexpr int kStep = 32;      // tokens of a warp's step (4 warps)
constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// An item that is cut: the join's work. rows = 0: nothing to join here.
struct CutItem {
    int b, h, row0, rows;
    int slot, parts;  // the first part's slot, and the pieces it goes over
};

static_assert(sizeof(CutItem) == kCutBytes, "the workspace holds CutItems");

struct AttnOut {
    void* O;
    float* lse;    // or null
    float* part;   // [2 * pieces][rows][d]
    float2* ml;    // [2 * pieces][rows] (maximum in log2 units, sum)
    CutItem* cut;  // [pieces]: the item that starts in a piece and ends behind it
    int pieces, rows;  // pieces of the line, rows of a tile
};

// Division of numbers that nearly always fit 32 bits.
__device__ __forceinline__ long long quot(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// One sequence's share of the line: (row tiles) * Hkv * (chunks of its length).
struct SeqWork {
    int n, count, rows, chunks;
    long long total;
};
__device__ __forceinline__ SeqWork seq_work(const CacheArgs& a, int b, int rtile) {
    SeqWork s;
    s.n = cache_len(a, b);
    s.count = cache_count(a, b);
    s.rows = s.count * a.G;
    s.chunks = max(1, (s.n + kChunk - 1) / kChunk);
    s.total = (long long)((s.rows + rtile - 1) / rtile) * a.Hkv * s.chunks;
    return s;
}

// The line of chunks, cut into `pieces` pieces that differ by one chunk at most.
struct Line {
    long long total, q, r;
    int pieces;
    __device__ __forceinline__ void set(long long t, int max_pieces) {
        total = t;
        pieces = (int)min((long long)max_pieces, t);
        q = pieces ? quot(t, pieces) : 0;
        r = t - q * pieces;
    }
    __device__ __forceinline__ long long at(int c) const { return c * q + min((long long)c, r); }
    __device__ __forceinline__ int piece_of(long long x) const {
        const long long head = r * (q + 1);
        return (int)(x < head ? quot(x, q + 1) : r + quot(x - head, q));
    }
};

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The line and, if `piece` has any of it, the sequence *b that piece starts in
// and the chunks *before it. Each warp finds it by itself, from one load of 32
// lengths at a time.
__device__ __forceinline__ bool line_start(const CacheArgs& a, int rtile, int piece, int max_pieces, int lane,
                                           Line* line, int* b, long long* before, SeqWork* sw) {
    SeqWork mine{};
    long long x = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        mine.total = 0;
        if (b0 + lane < a.B) mine = seq_work(a, b0 + lane, rtile);
        x += mine.total;
    }
    x = warp_scan(x, lane);
    line->set(__shfl_sync(0xffffffffu, x, 31), max_pieces);
    if (piece >= line->pieces) return false;
    const long long w = line->at(piece);
    long long base = 0;
    for (int b0 = 0;; b0 += 32) {
        if (a.B > 32) {
            mine.total = 0;
            if (b0 + lane < a.B) mine = seq_work(a, b0 + lane, rtile);
            x = base + warp_scan(mine.total, lane);
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w < x);
        if (hit) {  // the first sequence whose share ends behind w
            const int l = __ffs(hit) - 1;
            *b = b0 + l;
            *before = __shfl_sync(0xffffffffu, x - mine.total, l);
            sw->n = __shfl_sync(0xffffffffu, mine.n, l);
            sw->count = __shfl_sync(0xffffffffu, mine.count, l);
            sw->rows = __shfl_sync(0xffffffffu, mine.rows, l);
            sw->chunks = __shfl_sync(0xffffffffu, mine.chunks, l);
            sw->total = __shfl_sync(0xffffffffu, mine.total, l);
            return true;
        }
        base = __shfl_sync(0xffffffffu, x, 31);
    }
}

// One block's part of an item.
struct Segment {
    int b, h, row0, rows;  // sequence, cache head, first row and rows of the tile
    int c0, c1, chunks;    // chunks [c0, c1) of the item's `chunks`
    long long start;       // the item's first chunk on the line
};

// Segment that begins at chunk w (in sequence b, `before` chunks before it) and
// ends at w1 or at the item's end.
__device__ __forceinline__ Segment segment_at(const CacheArgs& a, int rtile, const SeqWork& s, int b, long long before,
                                              long long w, long long w1) {
    Segment g;
    const long long rel = w - before, item = quot(rel, s.chunks);
    g.b = b;
    g.start = before + item * s.chunks;
    const int tile = (int)quot(item, a.Hkv);
    g.h = (int)(item - (long long)tile * a.Hkv);
    g.row0 = tile * rtile;
    g.rows = min(rtile, s.rows - g.row0);
    g.chunks = s.chunks;
    g.c0 = (int)(rel - item * s.chunks);
    g.c1 = (int)min((long long)s.chunks, w1 - g.start);
    return g;
}

// A block's walk along its piece, in shared memory: registers are for the sums.
// Thread 0 (at first its warp) moves it; begin() and next() are called by the
// whole block and leave the next segment in `s`.
struct Walk {
    Line line;
    long long w, w_begin, w_end, before;
    SeqWork sw;
    Segment s;
    int b, slot;
    bool more;

    __device__ __forceinline__ void segment(const CacheArgs& a, const AttnOut& out, int piece) {
        while (w >= before + sw.total) {  // next sequence with work
            before += sw.total;
            sw = seq_work(a, ++b, out.rows);
        }
        s = segment_at(a, out.rows, sw, b, before, w, w_end);
        slot = 2 * piece + (w == w_begin ? 0 : 1);
        w = s.start + s.c1;
        if (w == w_end) note_cut(out, piece, s.c0 == 0 && s.c1 < s.chunks);
    }
    // The item that starts in this piece and ends behind it, if there is one.
    __device__ __forceinline__ void note_cut(const AttnOut& out, int piece, bool cut) {
        CutItem c{};
        if (cut) {
            c.b = s.b; c.h = s.h; c.row0 = s.row0; c.rows = s.rows;
            c.slot = slot;
            c.parts = line.piece_of(s.start + s.chunks - 1) - piece + 1;
        }
        out.cut[piece] = c;
    }
    __device__ __forceinline__ bool begin(const CacheArgs& a, const AttnOut& out, int piece) {
        if (threadIdx.x < 32) {
            Line l;
            SeqWork q;
            long long bf;
            int sb;
            const bool any = line_start(a, out.rows, piece, out.pieces, threadIdx.x, &l, &sb, &bf, &q);
            if (threadIdx.x == 0) {
                note_cut(out, piece, false);
                more = any;
                if (any) {
                    line = l; sw = q; before = bf; b = sb;
                    w = w_begin = l.at(piece);
                    w_end = l.at(piece + 1);
                    segment(a, out, piece);
                }
            }
        }
        __syncthreads();
        return more;
    }
    __device__ __forceinline__ bool next(const CacheArgs& a, const AttnOut& out, int piece) {
        __syncthreads();  // the block is done with the segment and its shared memory
        if (threadIdx.x == 0) {
            more = w < w_end;
            if (more) segment(a, out, piece);
        }
        __syncthreads();
        return more;
    }
};

// A kernel that this one's launch may be followed by can be set up meanwhile;
// it waits for this one's end before it reads anything.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
    allow_next();
    if (blockIdx.x == 0) {
        cache_check_call(a, false);
        return;
    }
    const int piece = blockIdx.x - 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> 3, ch = lane & 7;  // token of four, chunk
    __shared__ Walk walk;
    if (!walk.begin(a, out, piece)) return;
    uint8_t* ring = smem + warp * (kSimtStages * 2 * L::kBytes);
    const uint32_t ring_addr = smem_addr(ring);

    do {
        const Segment& s = walk.s;
        const int n = walk.sw.n, count = walk.sw.count, b = s.b;
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
        const int slot = walk.slot;
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
    } while (walk.next(a, out, piece));
}

// --------------------------------------------------------- tensor cores

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 8 x 8 halves, lane (g, t) holding row g, columns 2 t and 2 t + 1: transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// One group of a step: a bulk copy that `bar` counts, or nothing.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

constexpr float kNoKey = -1.7e38f;  // a row's maximum before it has seen a key: finite, so that differences are

constexpr int kStages = 2;
// Blocks per SM that the registers allow without spills. (16 rows of 128 channels: 3 blocks 48.6 us,
// 4 at 128 registers 51.2; 16 rows of 64: 33.0 and 30.9.)
constexpr int mma_blocks(int d, int NR) { return NR == 1 ? 4 : d == 64 ? (NR == 2 ? 4 : 3) : (NR == 2 ? 3 : 2); }

template <int D, int NR> constexpr int mma_smem() {
    constexpr int ring = 4 * kStages * 2 * Grp<D>::kBytes, merge = 4 * 8 * NR * D * 4;
    return (ring > merge ? ring : merge) + NR * (D / 16) * 256;
}

// bf16 rows on the tensor cores' register form (m16n8k16, halves in, fp32 out),
// tiles of 8 NR rows.
//
// The codes come from shared memory into the registers of the lanes that feed
// them to the step, are widened there and never go back to shared memory: one
// conversion per two codes and one product by the scale, both exact. (The
// tcgen05 form would need the widened operands in shared memory, 3.5 times the
// cached bytes written and read again, for tiles of 128 rows of which decoding
// fills 1 to 64.)
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
//         l takes the unrounded p). m is only moved when a score exceeds it by more than 8,
//         so p <= 2^8, and only then do lanes compare maxima and are the sums rescaled.
//   O^T   P^T is S^T's register layout transposed 8 x 8; 2 steps of 16 tokens x d/16 channel tiles.
template <int D, int NR>
__global__ void __launch_bounds__(kThreads, mma_blocks(D, NR))
k_cache_attn_mma(CacheArgs a, const __nv_bfloat16* __restrict__ Q, const uint8_t* __restrict__ cache, AttnOut out) {
    using L = Grp<D>;
    constexpr int KS = D / 16, NT = D / 8, W = D / 32, RT = 8 * NR, ST = kStages;
    constexpr int GP = NR == 1 ? 2 : 1;  // groups at a time: with more rows the registers hold one
    constexpr int kStage = 2 * L::kBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Walk walk;
    __shared__ float2 sml[4][RT];
    __shared__ float szf[RT];
    __shared__ int slim[RT];
    __shared__ uint64_t bars[4][ST];
    allow_next();
    if (blockIdx.x == 0) {
        cache_check_call(a, false);
        return;
    }
    const int piece = blockIdx.x - 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t* ring = smem + warp * (ST * kStage);
    const uint32_t ring_addr = smem_addr(ring);
    uint2* qs = reinterpret_cast<uint2*>(smem + mma_smem<D, NR>() - NR * KS * 256);
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) tc::mbar_init(&bars[warp][i], 2);
        tc::fence_mbar_init();
    }
    if (!walk.begin(a, out, piece)) return;
    int put = 0, take = 0, phase = 0;  // stages of the ring, and the phase of `take`
    bool dead = false;                 // a wait ran out

    do {
        const Segment& s = walk.s;
        const int n = walk.sw.n, count = walk.sw.count, b = s.b;
        // rows of a tile see more keys the later their token is
        const int low = row_limit(a, n, count, s.row0 / a.G), top = row_limit(a, n, count, (s.row0 + s.rows - 1) / a.G);
        const int steps = s.c1 - s.c0;
        // Lane l has the group number of group l & 1 of step l >> 1 in the current run of 16
        // steps, and issues that copy itself; the next run's table entries are loaded a run ahead.
        auto groups = [&](int i0) -> const uint8_t* {
            const int gi = GroupRun::load(a, s, top, warp, lane, i0);
            return gi < 0 ? nullptr : cache + (long long)gi * L::kBytes;
        };
        const uint8_t *gcur = groups(0), *gnxt = groups(16);
        auto issue = [&](int i) {
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
                gnxt = groups(i + 17);
            }
        };
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue(i);

        // Q: warp w has rows 8 w + g, lane (g, t4) channels [t4 d/4, (t4 + 1) d/4) of them
        const float vscale = pow2(cache_exp(a, 1, s.h));
        if (warp < NR) {
            const int r = warp * 8 + g;
            int t = 0;
            const long long at = row_offset(a, b, s.h, s.row0 + min(r, s.rows - 1), &t);
            uint32_t x[D / 8], amax = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < s.rows) v = reinterpret_cast<const uint4*>(Q + at * D + t4 * (D / 4))[i];
                x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) amax = max(amax, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int ex = (int)(amax >> 7);  // biased exponent of the row's largest entry
            const int qe = ex == 255 ? 0 : min(141 - ex, 120);
            const float up = pow2(qe), kf = a.scale * kLog2e * pow2(cache_exp(a, 0, s.h));
            if (t4 == 0) {
                // kept away from 0 and infinity: a masked score is -infinity times it
                szf[r] = fminf(fmaxf(kf * pow2(-qe), 1.1754944e-38f), 3.4028235e38f);
                slim[r] = r < s.rows ? row_limit(a, n, count, t) : 0;
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t h[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t y = x[2 * ks + e];
                    h[e] = pack_half2(__uint_as_float(y << 16) * up, __uint_as_float(y & 0xffff0000u) * up);
                }
                qs[(ks * NR + warp) * 32 + lane] = make_uint2(h[0], h[1]);
            }
        }
        __syncthreads();
        uint2 qf[NR == 1 ? KS : 1];
        if (NR == 1) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[ks] = qs[ks * 32 + lane];
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
            issue(i + ST - 1);
            if (!tc::mbar_wait(&bars[warp][take], phase, a.status)) {
                // give up, but not before the copies in flight have landed (or a second has passed for each)
                for (int x = i + 1; x < steps && x < i + ST; ++x) {
                    take = take + 1 == ST ? 0 : take + 1;
                    phase ^= take == 0;
                    tc::mbar_wait(&bars[warp][take], phase, a.status);
                }
                dead = true;
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
                float z[NR][GP][4];
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int x = 0; x < GP; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[j][x][e] = 0.0f;
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
                            const uint2 q = NR == 1 ? qf[(2 * wi + k2) % (NR == 1 ? KS : 1)] : qs[((2 * wi + k2) * NR + j) * 32 + lane];
#pragma unroll
                            for (int gi = 0; gi < GP; ++gi)
                                mma_f16(z[j][gi], k8[gi][0][2 * k2], k8[gi][1][2 * k2], k8[gi][0][2 * k2 + 1],
                                        k8[gi][1][2 * k2 + 1], q.x, q.y);
                        }
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
                            y[j][x][e] = fmaf(z[j][x][e], zf[j][e & 1], -m[j][e & 1]);
                            big = fmaxf(big, y[j][x][e]);
                        }
                if (__any_sync(0xffffffffu, big > 8.0f)) {
#pragma unroll
                    for (int j = 0; j < NR; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = fmaxf(z[j][0][e], z[j][0][e + 2]);
                            if (GP == 2) v = fmaxf(v, fmaxf(z[j][GP - 1][e], z[j][GP - 1][e + 2]));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
                            const float mn = fmaxf(m[j][e], v * zf[j][e]), f = ex2(m[j][e] - mn);
                            m[j][e] = mn;
                            l[j][e] *= f;
#pragma unroll
                            for (int x = 0; x < NT / 2; ++x) {
                                o[j][x][e] *= f;
                                o[j][x][e + 2] *= f;
                            }
#pragma unroll
                            for (int x = 0; x < GP; ++x) {
                                y[j][x][e] = fmaf(z[j][x][e], zf[j][e], -mn);
                                y[j][x][e + 2] = fmaf(z[j][x][e + 2], zf[j][e], -mn);
                            }
                        }
                }
                uint32_t p[NR][GP][2];  // P^T: [group][tokens 2 t4 and the next, 8 further], row g
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int x = 0; x < GP; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float p0 = ex2(y[j][x][2 * e]), p1 = ex2(y[j][x][2 * e + 1]);
                            l[j][0] += p0;
                            l[j][1] += p1;
                            p[j][x][e] = transpose8(pack_half2(p0, p1));
                        }
#pragma unroll
                for (int gi = 0; gi < GP; ++gi) {
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
                                float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma_f16(hit, a0, a0, a2, a2, see[0], see[1]);
#pragma unroll
                                for (int x = 0; x < NT / 2; ++x)
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (hit[e] > 0.0f) o[j][x][e] = __int_as_float(0x7fc00000);
                            }
                        }
                    }
                    const uint32_t s0 = e4m3x2_to_half2(sb & 0xffff), s1 = e4m3x2_to_half2(sb >> 16);
                    uint32_t vw[4][D / 64];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint8_t* vr = vb + L::v_chunk(t4 + 4 * x, g);
                        if (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(vr);
                            vw[x][0] = v.x; vw[x][D / 64 - 1] = v.y;
                        } else {
                            vw[x][0] = *reinterpret_cast<const uint32_t*>(vr);
                        }
                    }
#pragma unroll
                    for (int wi = 0; wi < D / 64; ++wi) {
                        // a byte of both tokens of a pair: even channels, then odd ones
                        constexpr uint32_t lo = 0x0f0f0f0fu;
                        uint32_t v8[2][2][4];  // [tokens 8 x + 2 t4 ..][parity of the channel]
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t u0 = vw[2 * x][wi], u1 = vw[2 * x + 1][wi];
                            e2m1x8_to_half2((u0 & lo) | ((u1 << 4) & ~lo), v8[x][0]);
                            e2m1x8_to_half2(((u0 >> 4) & lo) | (u1 & ~lo), v8[x][1]);
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t a0 = hmul2(v8[0][0][x], s0), a1 = hmul2(v8[0][1][x], s0);
                            const uint32_t a2 = hmul2(v8[1][0][x], s1), a3 = hmul2(v8[1][1][x], s1);
#pragma unroll
                            for (int j = 0; j < NR; ++j) mma_f16(o[j][4 * wi + x], a0, a1, a2, a3, p[j][gi][0], p[j][gi][1]);
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
        __syncthreads();  // every warp is done with its ring
        // Join the warps: [warp][row][d] sums, 16 bytes (four channels) at a time. The
        // lanes that store together have four rows and two chunks apart by d/32; the
        // row's bits exchange chunks so that eight lanes meet eight bank groups.
        float4* os = reinterpret_cast<float4*>(smem);
        constexpr int C4 = D / 4;
        auto at4 = [&](int wp, int r, int c) {
            const int t = (r >> 1) & 3;
            return (wp * RT + r) * C4 + (c ^ (D == 128 ? t : (t & 1) | (t & 2) << 1));
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
        const bool whole = s.c0 == 0 && s.c1 == s.chunks;
        const int slot = walk.slot;
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
                const float f = ex2(v[i].x - mx);
                const float4 u = os[at4(i, r, c)];
                sum = fmaf(f, v[i].y, sum);
                acc.x = fmaf(f, u.x, acc.x); acc.y = fmaf(f, u.y, acc.y);
                acc.z = fmaf(f, u.z, acc.z); acc.w = fmaf(f, u.w, acc.w);
            }
            if (whole) {
                int t;
                const long long at = row_offset(a, b, s.h, s.row0 + r, &t);
                const float inv = sum == 0.0f ? 0.0f : vscale / sum;
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                                     h1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(out.O) + at * D)[c] =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
                if (out.lse && c == 0) out.lse[at] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
            } else {
                acc.x *= vscale; acc.y *= vscale; acc.z *= vscale; acc.w *= vscale;
                reinterpret_cast<float4*>(out.part + ((long long)slot * RT + r) * D)[c] = acc;
                if (c == 0) out.ml[(long long)slot * RT + r] = make_float2(mx, sum);
            }
        }
        tc::fence_proxy_async();  // the next segment's copies come after these accesses of the ring
    } while (!__syncthreads_or(dead) && walk.next(a, out, piece));
}

// ------------------------------------------------------------------ join

constexpr int kJoinRows = 4, kJoinWarps = 8;

// Block (c, y) joins the parts of the item that starts in piece c and ends
// behind it, rows 4 y to 4 y + 3 at once: each warp adds every eighth part, a lane
// d/32 channels of each row. It is a chain of loads (the item, the maxima, the
// sums), so the rows and parts are in flight together.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) k_cache_join(CacheArgs a, AttnOut out) {
    constexpr int E = D / 32;
    __shared__ float acc8[kJoinWarps][kJoinRows][D];
    __shared__ float sum8[kJoinWarps][kJoinRows];
    wait_previous();
    const CutItem c = out.cut[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = out.rows;
    const int r0 = blockIdx.y * kJoinRows, rows = min(c.rows - r0, kJoinRows);
    if (rows <= 0) return;
    // part p > 0 begins its piece
    auto slot = [&](int p) { return (long long)(p == 0 ? c.slot : 2 * (blockIdx.x + p)) * R + r0; };
    float mx[kJoinRows], sum[kJoinRows], acc[kJoinRows][E];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        mx[r] = -INFINITY;
        sum[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[r][i] = 0.0f;
    }
    for (int p = lane; p < c.parts; p += 32) {
        const float2* ml = out.ml + slot(p);
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r)
            if (r < rows) mx[r] = fmaxf(mx[r], ml[r].x);
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        mx[r] = warp_max(mx[r]);
        if (mx[r] == -INFINITY) mx[r] = 0.0f;  // no part has a key of this row
    }
#pragma unroll 2
    for (int p = warp; p < c.parts; p += kJoinWarps) {
        const long long at = slot(p);
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            if (r >= rows) continue;
            const float2 ml = out.ml[at + r];
            float v[E];
            if (E == 4) {
                const float4 u = reinterpret_cast<const float4*>(out.part + (at + r) * D)[lane];
                v[0] = u.x; v[1] = u.y; v[E - 2] = u.z; v[E - 1] = u.w;
            } else {
                const float2 u = reinterpret_cast<const float2*>(out.part + (at + r) * D)[lane];
                v[0] = u.x; v[1] = u.y;
            }
            const float f = exp2f(ml.x - mx[r]);
            sum[r] = fmaf(f, ml.y, sum[r]);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[r][i] = fmaf(f, v[i], acc[r][i]);
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
#pragma unroll
        for (int i = 0; i < E; ++i) acc8[warp][r][lane * E + i] = acc[r][i];
        if (lane == 0) sum8[warp][r] = sum[r];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * D; x += 32 * kJoinWarps) {
        const int r = x / D, i = x - r * D;
        float s = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            s += sum8[w][r];
            v += acc8[w][r][i];
        }
        int t;
        const long long at = row_offset(a, c.b, c.h, c.row0 + r0 + r, &t);
        reinterpret_cast<T*>(out.O)[at * D + i] = from_f<T>(s == 0.0f ? 0.0f : v / s);
        if (out.lse && i == 0) {
            float top = mx[0];
#pragma unroll
            for (int q = 1; q < kJoinRows; ++q) top = q == r ? mx[q] : top;
            out.lse[at] = s == 0.0f ? -INFINITY : (top + log2f(s)) * kLn2;
        }
    }
}

// ------------------------------------------------------------------ launch

static long long max_chunks(const CacheArgs& a, int rtile) {
    const long long tiles = ((long long)a.G * a.T + rtile - 1) / rtile;
    const long long len = ((long long)a.cols * a.page + kChunk - 1) / kChunk;
    return (long long)a.B * a.Hkv * tiles * len;
}

CachePlan cache_attn_plan(const CacheArgs& a, int d, int dtype, unsigned flags) {
    CachePlan p;
    const long long rows = (long long)a.G * a.T;
    p.tensor = dtype == 1 && !(flags & MITA_FLAG_SIMT);
    int blocks = 4;  // per SM
    if (p.tensor) {
        p.rows = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
        blocks = mma_blocks(d, p.rows / 8);
    } else {
        p.rows = rows == 1 ? 1 : 4;
    }
    // one of the resident blocks checks the call's indexes
    p.pieces = (int)std::min<long long>((long long)blocks * num_sms() - 1, max_chunks(a, p.rows));
    p.parts = (size_t)2 * p.pieces * p.rows;
    return p;
}

template <typename T, int D>
static cudaError_t join_t(const CacheArgs& a, const AttnOut& o, cudaStream_t st) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || o.pieces == 1) return e;
    prof_mark(st, "cache_join");
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(o.pieces, (o.rows + kJoinRows - 1) / kJoinRows);
    c.blockDim = dim3(32 * kJoinWarps);
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, k_cache_join<T, D>, a, o);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T, int D, int R>
static cudaError_t simt_t(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st) {
    constexpr int smem = simt_smem<D, R>();
    const cudaError_t e = cudaFuncSetAttribute(k_cache_attn_simt<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_cache_attn_simt<T, D, R><<<o.pieces + 1, kThreads, smem, st>>>(a, (const T*)Q, cache, o);
    count_launch();
    return join_t<T, D>(a, o, st);
}

template <int D, int NR>
static cudaError_t mma_t(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st) {
    constexpr int smem = mma_smem<D, NR>();
    static_assert(mma_blocks(D, NR) * (smem + 3 * 1024) <= 228 * 1024, "the blocks that a call counts on fit an SM");
    const cudaError_t e = cudaFuncSetAttribute(k_cache_attn_mma<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_cache_attn_mma<D, NR><<<o.pieces + 1, kThreads, smem, st>>>(a, (const __nv_bfloat16*)Q, cache, o);
    count_launch();
    return join_t<__nv_bfloat16, D>(a, o, st);
}

template <int D>
static cudaError_t attn_t(const CacheArgs& a, const CachePlan& p, int dtype, const void* Q, const uint8_t* cache,
                          const AttnOut& o, cudaStream_t st) {
    if (p.tensor)
        return p.rows == 8 ? mma_t<D, 1>(a, Q, cache, o, st)
               : p.rows == 16 ? mma_t<D, 2>(a, Q, cache, o, st) : mma_t<D, 4>(a, Q, cache, o, st);
    if (dtype == 0) return p.rows == 1 ? simt_t<float, D, 1>(a, Q, cache, o, st) : simt_t<float, D, 4>(a, Q, cache, o, st);
    return p.rows == 1 ? simt_t<__nv_bfloat16, D, 1>(a, Q, cache, o, st) : simt_t<__nv_bfloat16, D, 4>(a, Q, cache, o, st);
}

cudaError_t launch_cache_attn(const CacheArgs& a, const CachePlan& p, int d, int dtype, const void* Q,
                              const void* cache, void* O, float* lse, const CacheParts& parts, cudaStream_t st) {
    const AttnOut o{O, lse, parts.part, parts.ml, (CutItem*)parts.cut, p.pieces, p.rows};
    const uint8_t* c = (const uint8_t*)cache;
    prof_mark(st, "cache_attention");
    return d == 64 ? attn_t<64>(a, p, dtype, Q, c, o, st) : attn_t<128>(a, p, dtype, Q, c, o, st);
}

}  // namespace mita
