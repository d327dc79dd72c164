// What the attention kernels over the 4-bit cache share (cache_attn.cu,
// cache_tile.cu): how a call's work is cut into pieces, how a block walks along its
// piece, and how it reports what it found.
#pragma once

#include <atomic>

#include "cache.cuh"
#include "tc.cuh"

namespace mita {

constexpr int kChunk = 128;  // tokens of a block's step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnOut {
    void* O;
    float* lse;    // or null
    float* part;   // [2 * pieces][rows][d]
    float2* ml;    // [2 * pieces][rows] (maximum in log2 units, sum)
    int* found;        // [pieces]: what a piece found wrong, for the call's status word
    int pieces, rows;  // pieces of the line, rows of a tile
    int extra, tiles;  // Walk's EXTRA; tiles of a sequence with T rows
};

// One sequence's share of the line. Its items are cut into chunks, and each item
// takes `extra` units more than its chunks: what starting and ending an item costs
// a block (loading Q, the first copies' latency, joining the warps), so that
// blocks with many short items get fewer chunks.
struct SeqWork {
    int n, count, rows, chunks, items;
};
__device__ __forceinline__ SeqWork seq_work(const CacheArgs& a, int b, int rtile) {
    SeqWork s;
    s.n = cache_len(a, b);
    s.count = cache_count(a, b);
    s.rows = s.count * a.G;
    s.chunks = max(1, (s.n + kChunk - 1) / kChunk);
    s.items = (s.rows + rtile - 1) / rtile * a.Hkv;
    return s;
}

// With fewer than kFew chunks per block an item's start is not counted: chunks run
// side by side then, and what counts is that no block has one more of them.
// Measured with 64 sequences of 33 to 8191 tokens (16,400 chunks, 512 items): the
// slowest block ended at 69 us without `extra` and at 56 with it, the median at 49.
// cache_tile.cu's items cost more to start and end (kTileExtra 2, 4, 6, 9, 14:
// 47.3, 45.2, 45.2, 45.3, 46.2 us for 32 items of 64 rows over 9000 to 16384 tokens).
constexpr int kExtra = 2, kTileExtra = 4, kFew = 8;

// The line of units, cut into `pieces` pieces that differ by one unit at most.
struct Line {
    int pieces, q, r, extra, total;
    __device__ __forceinline__ int at(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int piece_of(int x) const {
        const int head = r * (q + 1);
        return x < head ? x / (q + 1) : r + (x - head) / q;
    }
};

__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The line of a call, by a whole warp. `mine` is left with the lane's sequence of the last 32.
__device__ __forceinline__ Line call_line(const CacheArgs& a, int rtile, int extra, int max_pieces, int lane, SeqWork* mine) {
    unsigned items = 0, chunks = 0;
#pragma unroll 8
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        mine->items = 0;
        if (b0 + lane < a.B) *mine = seq_work(a, b0 + lane, rtile);
        items += mine->items;
        chunks += mine->items * mine->chunks;
    }
    items = __reduce_add_sync(0xffffffffu, items);
    chunks = __reduce_add_sync(0xffffffffu, chunks);
    Line l;
    l.extra = chunks >= (unsigned)max_pieces * kFew ? extra : 0;
    l.total = (int)(chunks + items * l.extra);
    l.pieces = min(max_pieces, l.total);
    l.q = l.pieces ? l.total / l.pieces : 0;
    l.r = l.total - l.q * l.pieces;
    return l;
}
// The sequence whose share holds unit w, by the same warp after call_line(): one lane
// returns true, with the sequence, its work and the units before it.
__device__ __forceinline__ bool find_unit(const CacheArgs& a, const Line& l, int rtile, int w, int lane, SeqWork* mine,
                                          int* b, int* before) {
    int base = 0, x = 0, share = 0;
    unsigned hit = 0;
    int b0 = 0;
    for (; b0 < a.B && !hit; b0 += 32) {
        if (a.B > 32) {
            mine->items = 0;
            if (b0 + lane < a.B) *mine = seq_work(a, b0 + lane, rtile);
        }
        share = mine->items * (mine->chunks + l.extra);
        x = base + warp_scan(share, lane);
        hit = __ballot_sync(0xffffffffu, w < x);  // the first whose share ends behind w
        base = __shfl_sync(0xffffffffu, x, 31);
    }
    *before = x - share;
    *b = b0 - 32 + lane;
    return hit && lane == __ffs(hit) - 1;
}

// One block's part of an item.
struct Segment {
    int b, h, row0, rows;  // sequence, cache head, first row and rows of the tile
    int c0, c1, chunks;    // chunks [c0, c1) of the item's `chunks`
    int first;             // the item's chunk 0 on the line
};

// A block's walk along its piece, in shared memory: registers are for the sums.
// The first warp finds the start, thread 0 moves it; begin() and next() are called
// by the whole block and leave the next segment in `s`. A piece holds at most one
// segment of an item that began before it (the first) and one of an item that goes
// on behind it (the last).
template <int RT, int EXTRA = kExtra> struct Walk {
    Line line;
    int w, w_end, before, b;  // position; units before sequence b
    SeqWork sw;
    Segment s;
    bool more;

    // The next segment from w on, if there is one.
    __device__ __forceinline__ void segment(const CacheArgs& a) {
        more = false;
        while (w < w_end) {
            const int len = sw.chunks + line.extra;
            if (w - before >= sw.items * len) {  // next sequence with work
                before += sw.items * len;
                if (++b >= a.B) return;
                sw = seq_work(a, b, RT);
                continue;
            }
            const int item = (w - before) / len, start = before + item * len;
            const int tile = item / a.Hkv;
            s.b = b;
            s.h = item - tile * a.Hkv;
            s.row0 = tile * RT;
            s.rows = min(RT, sw.rows - s.row0);
            s.chunks = sw.chunks;
            s.first = start + line.extra;
            s.c0 = max(w - s.first, 0);
            s.c1 = min(s.chunks, w_end - s.first);
            w = start + len;
            if (s.c0 < s.c1) {
                more = true;
                return;
            }
        }
    }
    __device__ __forceinline__ bool begin(const CacheArgs& a, int piece, int max_pieces) {
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            SeqWork mine{};
            const Line l = call_line(a, RT, EXTRA, max_pieces, lane, &mine);
            if (lane == 0) more = false;
            __syncwarp();
            int b1, before1;
            if (piece < l.pieces && find_unit(a, l, RT, l.at(piece), lane, &mine, &b1, &before1)) {
                line = l;
                w = l.at(piece);
                w_end = l.at(piece + 1);
                before = before1;
                b = b1;
                sw = mine;
                segment(a);
            }
        }
        __syncthreads();
        return more;
    }
    __device__ __forceinline__ bool next(const CacheArgs& a) {
        __syncthreads();  // the block is done with the segment and its shared memory
        if (threadIdx.x == 0) segment(a);
        __syncthreads();
        return more;
    }
    __device__ __forceinline__ bool whole() const { return s.c0 == 0 && s.c1 == s.chunks; }
    // Where the sums of a part of an item go: the part that starts the item, or another.
    __device__ __forceinline__ int slot(int piece) const { return 2 * piece + (s.c0 == 0); }
};

// What a piece finds wrong; the join makes the call's status word of it. Between
// them the pieces read every table entry that the call uses; the first also
// checks the lengths, counts and exponents.
enum : int { kFoundBounds = 1, kFoundTimeout = 2 };
__device__ __forceinline__ int first_piece(const CacheArgs& a) {
    bool bad = bad_exps(a);
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) bad |= bad_len(a, b);
    return bad ? kFoundBounds : 0;
}
// The end of a piece, by the whole block.
__device__ __forceinline__ void end_piece(const CacheArgs& a, const AttnOut& out, int piece, int found) {
    if (piece == 0) found |= first_piece(a);
    const int bounds = __syncthreads_or(found & kFoundBounds), timeout = __syncthreads_or(found & kFoundTimeout);
    if (threadIdx.x == 0) out.found[piece] = (bounds ? kFoundBounds : 0) | (timeout ? kFoundTimeout : 0);
}

// An item that is cut, for the join.
struct CutItem {
    int b, h, row0, rows;  // rows = 0: not cut
    int piece, parts;      // the first part's piece, and the pieces it goes over
};
// Item i of the call (of all tiles of T rows), by a whole warp.
__device__ __forceinline__ CutItem cut_item(const CacheArgs& a, const AttnOut& out, int i, int lane) {
    SeqWork sw{};
    const Line l = call_line(a, out.rows, out.extra, out.pieces, lane, &sw);
    CutItem c{};
    c.b = i / (out.tiles * a.Hkv);
    const int j = i - c.b * (out.tiles * a.Hkv), tile = j / a.Hkv;
    int before = 0;  // units before the sequence
    for (int b0 = 0; b0 < c.b; b0 += 32)
        if (b0 + lane < c.b) {
            const SeqWork x = seq_work(a, b0 + lane, out.rows);
            before += x.items * (x.chunks + l.extra);
        }
    before = __reduce_add_sync(0xffffffffu, before);
    sw = seq_work(a, c.b, out.rows);
    if (j >= sw.items) return c;
    const int first = before + j * (sw.chunks + l.extra) + l.extra;
    c.piece = l.piece_of(first);
    c.parts = l.piece_of(first + sw.chunks - 1) - c.piece + 1;
    c.h = j - tile * a.Hkv;
    c.row0 = tile * out.rows;
    if (c.parts > 1) c.rows = min(out.rows, sw.rows - c.row0);
    return c;
}
// The item that begins in piece p and goes on behind it (there is at most one), by a
// whole warp; the lane that returns true has it.
__device__ __forceinline__ bool cut_item_of_piece(const CacheArgs& a, const AttnOut& out, int p, int lane, CutItem* c) {
    SeqWork sw{};
    const Line l = call_line(a, out.rows, out.extra, out.pieces, lane, &sw);
    if (p + 1 >= l.pieces) return false;
    const int w = l.at(p + 1);  // the first unit behind the piece
    int before;
    if (!find_unit(a, l, out.rows, w, lane, &sw, &c->b, &before)) return false;
    const int len = sw.chunks + l.extra, j = (w - before) / len, first = before + j * len + l.extra;
    if (first >= w || first < l.at(p)) return false;
    const int tile = j / a.Hkv;
    c->h = j - tile * a.Hkv;
    c->row0 = tile * out.rows;
    c->rows = min(out.rows, sw.rows - c->row0);
    c->piece = p;
    c->parts = l.piece_of(first + sw.chunks - 1) - p + 1;
    return true;
}

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

// --------------------------------------------------------------- helpers

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// One group of a step: a bulk copy that `bar` counts, or nothing.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Query rows go to halves scaled by a power of two (`up`) that puts the row's
// largest entry, of biased exponent ex, in [2^14, 2^15); f: the factor of the
// scores for it, in log2 units. A row with an infinity or a NaN becomes NaN
// altogether, as its softmax is (infinite scores have no differences).
__device__ __forceinline__ void query_scale(const CacheArgs& a, int h, int ex, float* up, float* f) {
    const int qe = min(141 - ex, 120);
    *up = ex == 255 ? __int_as_float(0x7fc00000) : pow2(qe);
    // kept away from 0 and infinity: a masked score is -infinity times it
    *f = fminf(fmaxf(a.scale * kLog2e * pow2(cache_exp(a, 0, h)) * pow2(-qe), 1.1754944e-38f), 3.4028235e38f);
}

// z f - m, with the product rounded: the reference m was made of a rounded product
// too, so that the difference to its own score stays 7 (or less) when scores are so
// large that 7 is lost in them. One rounding would leave up to 2^-24 of m.
__device__ __forceinline__ float score_diff(float z, float f, float m) { return __fadd_rn(__fmul_rn(z, f), -m); }

constexpr float kNoKey = -1.7e38f;  // a row's maximum before it has seen a key: finite, so that differences are

// cache_attn.cu
cudaError_t set_smem_once(const void* f, int bytes, std::atomic<unsigned long long>* done);
// cache_tile.cu: tiles of 64 bf16 rows of 128 channels
cudaError_t launch_cache_tile(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st);

}  // namespace mita
