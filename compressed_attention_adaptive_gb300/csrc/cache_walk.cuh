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
__host__ __device__ __forceinline__ SeqWork seq_work(const CacheArgs& a, int b, int rtile) {
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
    __host__ __device__ __forceinline__ int at(int c) const { return c * q + min(c, r); }
    __host__ __device__ __forceinline__ int piece_of(int x) const {
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

// Finds the line of a call, by a whole block: a thread takes B / blockDim sequences, its
// own few or one. `at(line, s0, s1, first, before, share)` is then called by each thread
// that has sequences [s0, s1), with the work of s0, the units before them and theirs. (One warp that went over
// the sequences 32 at a time, twice, made a call of 1024 sequences 46 us longer.)
struct LineScan {
    unsigned items[32], chunks[32];  // of each warp
};
template <typename At>
__device__ __forceinline__ void scan_line(const CacheArgs& a, int rtile, int extra, int max_pieces, LineScan& sums, At at) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = a.B <= blockDim.x ? 1 : (a.B + blockDim.x - 1) / blockDim.x;
    const int warps = per == 1 ? (a.B + 31) / 32 : (a.B + 32 * per - 1) / (32 * per);
    const int s0 = threadIdx.x * per, s1 = min(s0 + per, a.B);
    unsigned items = 0, chunks = 0, items0 = 0, chunks0 = 0;  // the thread's; of the warps before
    SeqWork first{};
    if (warp < warps && s0 < s1) {
        first = seq_work(a, s0, rtile);
        items = first.items;
        chunks = first.items * first.chunks;
#pragma unroll 4
        for (int b = s0 + 1; b < s1; ++b) {
            const SeqWork w = seq_work(a, b, rtile);
            items += w.items;
            chunks += w.items * w.chunks;
        }
    }
    unsigned all_items = __reduce_add_sync(0xffffffffu, items), all_chunks = __reduce_add_sync(0xffffffffu, chunks);
    if (warps > 1) {
        if (lane == 0) {
            sums.items[warp] = all_items;
            sums.chunks[warp] = all_chunks;
        }
        __syncthreads();
        all_items = all_chunks = 0;
        for (int w = 0; w < warps; ++w) {
            if (w == warp) {
                items0 = all_items;
                chunks0 = all_chunks;
            }
            all_items += sums.items[w];
            all_chunks += sums.chunks[w];
        }
    } else {
        __syncwarp();
    }
    if (warp >= warps) return;
    Line l;
    l.extra = all_chunks >= (unsigned)max_pieces * kFew ? extra : 0;
    l.total = (int)(all_chunks + all_items * l.extra);
    l.pieces = min(max_pieces, l.total);
    l.q = l.pieces ? l.total / l.pieces : 0;
    l.r = l.total - l.q * l.pieces;
    const int share = (int)(chunks + items * l.extra);
    const int before = (int)(chunks0 + items0 * l.extra) + warp_scan(share, lane) - share;
    if (s0 < s1) at(l, s0, s1, first, before, share);
}
// A sequence may be read more than once in a call. Lengths that change meanwhile leave the
// results undefined, but no search goes past the sequences and no part past the pieces.
//
// The sequence of [s0, s1) whose share holds unit w, with its work (first that of s0) and
// the units before it; -1 if it is none of them.
__host__ __device__ __forceinline__ int find_unit(const CacheArgs& a, const Line& l, int rtile, int w, int s0, int s1,
                                                  int* before, SeqWork* sw) {
    for (;;) {
        const int share = sw->items * (sw->chunks + l.extra);
        if (w < *before + share) return s0;
        *before += share;
        if (++s0 >= s1) return -1;
        *sw = seq_work(a, s0, rtile);
    }
}
// The pieces of item j of a sequence with `before` units before it: the first and their
// number, 0 if the item is not on the line.
__host__ __device__ __forceinline__ int item_pieces(const Line& l, const SeqWork& sw, int before, int j, int* piece) {
    const int first = before + j * (sw.chunks + l.extra) + l.extra, last = first + sw.chunks - 1;
    if (last >= l.total) return 0;
    *piece = l.piece_of(first);
    return l.piece_of(last) - *piece + 1;
}

// One block's part of an item.
struct Segment {
    int b, h, row0, rows;  // sequence, cache head, first row and rows of the tile
    int c0, c1, chunks;    // chunks [c0, c1) of the item's `chunks`
    int first;             // the item's chunk 0 on the line
    int n, count;          // the sequence's
    __device__ __forceinline__ bool whole() const { return c0 == 0 && c1 == chunks; }
    // Where the sums of a part of an item go: the part that starts the item, or another.
    __device__ __forceinline__ int slot(int piece) const { return 2 * piece + (c0 == 0); }
};

// A block's walk along its piece, in shared memory: registers are for the sums.
// The thread with the first sequence finds the start, thread 0 moves it; begin() and
// next() are called by the whole block and leave the next segment in s(). (A kernel may
// call segment() ahead instead, by thread 0: the segment before stays as it was.) A
// piece holds at most one segment of an item that began before it (the first) and
// one of an item that goes on behind it (the last).
template <int RT, int EXTRA = kExtra> struct Walk {
    Line line;
    int w, w_end, before, b;  // position; units before sequence b
    SeqWork sw;
    Segment segs[2];  // the current one and another
    int cur;
    bool more;

    __device__ __forceinline__ const Segment& s() const { return segs[cur]; }
    // The next segment from w on, if there is one.
    __device__ __forceinline__ void segment(const CacheArgs& a) {
        more = false;
        cur ^= 1;
        Segment& s = segs[cur];
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
            s.n = sw.n;
            s.count = sw.count;
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
    __device__ __forceinline__ bool begin(const CacheArgs& a, int piece, int max_pieces, LineScan& sums) {
        if (threadIdx.x == 0) more = false;
        scan_line(a, RT, EXTRA, max_pieces, sums, [&](const Line& l, int s0, int s1, SeqWork first, int before0, int share) {
            if (piece >= l.pieces) return;
            const int w0 = l.at(piece);
            if (w0 < before0 || w0 >= before0 + share) return;
            b = find_unit(a, l, RT, w0, s0, s1, &before0, &first);
            if (b < 0) return;
            line = l;
            w = w0;
            w_end = l.at(piece + 1);
            before = before0;
            sw = first;
            cur = 0;
            segment(a);
        });
        __syncthreads();
        return more;
    }
    __device__ __forceinline__ bool next(const CacheArgs& a) {
        __syncthreads();  // the block is done with the segment and its shared memory
        if (threadIdx.x == 0) segment(a);
        __syncthreads();
        return more;
    }
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
// Fills in `c` (rows = 0 so far) for item i of the call (of all tiles of T rows) or, with
// by_item false, for the item that begins in piece i and goes on behind it (there is at
// most one). By a whole block; visible after its next barrier.
__device__ __forceinline__ void find_cut(const CacheArgs& a, const AttnOut& out, int i, bool by_item, LineScan& sums,
                                         CutItem& c) {
    scan_line(a, out.rows, out.extra, out.pieces, sums, [&](const Line& l, int s0, int s1, SeqWork sw, int before, int share) {
        int b, j;  // the sequence, and the item's number in it
        if (by_item) {
            b = i / (out.tiles * a.Hkv);
            if (b < s0 || b >= s1) return;
            j = i - b * (out.tiles * a.Hkv);
            for (int x = s0; x < b; sw = seq_work(a, ++x, out.rows)) before += sw.items * (sw.chunks + l.extra);
            if (j >= sw.items) return;
        } else {
            if (i + 1 >= l.pieces) return;
            const int w = l.at(i + 1);  // the first unit behind the piece
            if (w < before || w >= before + share) return;
            b = find_unit(a, l, out.rows, w, s0, s1, &before, &sw);
            if (b < 0) return;
            j = (w - before) / (sw.chunks + l.extra);
        }
        const int tile = j / a.Hkv;
        int piece;
        const int parts = item_pieces(l, sw, before, j, &piece);
        if (parts < 2 || (!by_item && piece != i)) return;
        c.b = b;
        c.h = j - tile * a.Hkv;
        c.row0 = tile * out.rows;
        c.rows = min(out.rows, sw.rows - c.row0);
        c.piece = piece;
        c.parts = parts;
    });
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

// One group of a step: a bulk copy that `bar` counts, or nothing.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}
// An m16n8k16 step of the tensor cores, halves in and fp32 sums.
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
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Query rows go to halves scaled by a power of two (`up`) that puts the row's
// largest entry, of biased exponent ex, in [2^14, 2^15); f: the factor of the
// scores for it, in log2 units. A row with an infinity or a NaN becomes NaN
// altogether, as its softmax is (infinite scores have no differences).
__device__ __forceinline__ int query_exp(int ex, float* up) {
    const int qe = min(141 - ex, 120);
    *up = ex == 255 ? __int_as_float(0x7fc00000) : pow2(qe);
    return qe;
}
__device__ __forceinline__ void query_scale(const CacheArgs& a, int h, int ex, float* up, float* f) {
    const int qe = query_exp(ex, up);
    // kept away from 0 and infinity: a masked score is -infinity times it
    *f = fminf(fmaxf(a.scale * kLog2e * pow2(cache_exp(a, 0, h)) * pow2(-qe), 1.1754944e-38f), 3.4028235e38f);
}

// z f - m, with the product rounded: the reference m was made of a rounded product
// too, so that the difference to its own score stays 7 (or less) when scores are so
// large that 7 is lost in them. One rounding would leave up to 2^-24 of m.
__device__ __forceinline__ float score_diff(float z, float f, float m) { return __fadd_rn(__fmul_rn(z, f), -m); }

// A row's maximum before it has seen a key: finite, so that differences to it are not
// NaN, and no finite score is below it (one that is far above gives an infinite difference,
// which moves the maximum like any other).
constexpr float kNoKey = -3.402823466e38f;

// cache_attn.cu
cudaError_t set_smem_once(const void* f, int bytes, std::atomic<unsigned long long>* done);
// cache_tile.cu: tiles of 64 bf16 rows of 128 channels
cudaError_t launch_cache_tile(const CacheArgs& a, const void* Q, const uint8_t* cache, const AttnOut& o, cudaStream_t st);

}  // namespace mita
