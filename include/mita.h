/*
 * mita.h -- C ABI of libmita.so, the GB300 (sm_103a) MiTA attention forward.
 *
 * The operation is the forward pass of "MiTA Attention: Efficient Fast-Weight
 * Scaling via a Mixture of Top-k Activations" as summarized on gist.science:
 *
 *   landmarks    Qt = adaptive average pooling of Q, m rows      (Arabic ed. s2, "mechanism details";
 *                                                                  Dutch ed. "Kernconcepten" 1)
 *   shared       Vt = softmax(scale * Qt K^T) V                  (Arabic ed. s2: Vt = Atten(Qt, K, V))
 *   expert sets  I_i = indices of the k largest k_j . qt_i       (Arabic ed. s2; Dutch ed. "Kernconcepten" 3)
 *   routing      e_1(q) .. e_s(q)                                (Dutch ed. "Wiskundige Formulering")
 *   output       O_q = softmax attention of q over
 *                K* = [Qt, K_(e1), .., K_(es)], V* = [Vt, V_(e1), .., V_(es)]
 *                                                                (Dutch ed. "Wiskundige Formulering")
 *
 * The summaries leave four points open; this library fixes them as follows:
 *   - the shared expert's keys are Qt (its values are Vt);
 *   - a query is routed to the s landmarks with the largest q . qt_i, ties to
 *     the lower landmark index, listed by descending score;
 *   - top-k ranks raw (unscaled) scores, ties to the lower key index, and each
 *     I_i is returned in ascending key order;
 *   - expert sets that overlap are concatenated (a key picked by two routed
 *     experts fills two slots), and one softmax runs over all m + s*k slots.
 *
 * Conventions for every entry point:
 *   - Tensors are DEVICE pointers, contiguous, row-major [B, H, rows, d]
 *     (d fastest). Q, K, V, O use `dtype`; Qt / Vt outputs are float32;
 *     index outputs are int32.
 *   - The caller owns all memory, including the workspace (device memory of at
 *     least mita_workspace_size() bytes, 256-byte aligned). The library never
 *     allocates, frees or synchronizes inside these calls.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream). Outputs are valid once the stream reaches them.
 *   - Argument errors are returned synchronously before anything is enqueued.
 *     A failed launch returns MITA_ERR_CUDA. Errors detected on the device
 *     (an index out of range, a bounded wait that ran out) are written to a
 *     status word inside the workspace and read with mita_device_status().
 *     The first kernel of every call resets that word, so it holds the first
 *     device-side error of the most recent call on the workspace: read it
 *     after each call whose device status matters.
 *   - Calls are reentrant; concurrent calls must use distinct workspaces.
 */
#ifndef MITA_H
#define MITA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MITA_OK = 0,
    MITA_ERR_INVALID_ARG = 1, /* bad shape, pointer, flag or dtype             */
    MITA_ERR_UNSUPPORTED = 2, /* valid MiTA parameters this library cannot run */
    MITA_ERR_WORKSPACE = 3,   /* workspace NULL, misaligned or too small       */
    MITA_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed          */
    MITA_ERR_TIMEOUT = 5,     /* device: a bounded wait gave up                */
    MITA_ERR_BOUNDS = 6       /* device: an index was out of range             */
} mita_status;

typedef enum { MITA_DTYPE_F32 = 0, MITA_DTYPE_BF16 = 1 } mita_dtype;

enum {
    /* Leave the m shared slots out of the output softmax (only the routed
     * experts remain). With k = N and s = 1 the output is plain softmax
     * attention, which tests use as an identity. */
    MITA_FLAG_NO_SHARED = 1u << 0,
    /* Run every step on CUDA cores in fp32 even where the tensor-core path
     * applies (a second GPU implementation for cross-checks). */
    MITA_FLAG_SIMT = 1u << 1,
    /* The causal variant (the summaries describe none; these rules are this
     * library's reading, for 1-D pooling only): the shared expert of landmark
     * i attends to the keys of its prefix, j < hi_i, where [lo_i, hi_i) is
     * its pooling bin; query t has landmark i's shared slot only once that bin
     * is complete (hi_i <= t + 1); expert sets and routes are selected as in
     * the non-causal pass, and of a routed expert's keys query t attends to
     * those with j <= t; a query left with no slot gets a zero output row.
     * Runs on the tensor-core path when m <= 128, k <= 256 and the shared
     * slots are on, and on the CUDA-core path (float32, or MITA_FLAG_SIMT);
     * other shapes return MITA_ERR_UNSUPPORTED. With 2-D pooling it is
     * MITA_ERR_INVALID_ARG. */
    MITA_FLAG_CAUSAL = 1u << 2,
    /* mita_rope only: pairs are neighbouring channels. */
    MITA_FLAG_INTERLEAVED = 1u << 3
};

/* Fault test of the device-side failure detection, not for production: in
 * one CTA of the landmark pass and one of the expert attention, a producer
 * leaves out one of the signals its consumers wait for, and every bounded
 * wait of those two kernels gives up after about a millisecond instead of a
 * second. The call then records MITA_ERR_TIMEOUT in the device status word
 * (read with mita_device_status()); every role of the stalled CTAs leaves its
 * loop, lets its copies and MMAs in flight land and frees its tensor memory,
 * so the next call on the same workspace runs normally. Outputs of the
 * flagged call are undefined. Only the tensor-core path has these waits: on
 * the CUDA-core path the flag has no effect. (A macro, since the bit is
 * outside the int range of a C enum constant.) */
#define MITA_TESTFLAG_STALL_PRODUCER (1u << 31)

typedef struct {
    int B, H, N, d;   /* batch, heads, tokens, head dim (8 <= d <= 256, d % 8 == 0) */
    int m, k, s;      /* landmarks (1..N), top-k width (1..N), routed experts (1..min(m, 8)) */
    int grid_h, grid_w; /* token grid for 2-D pooling (grid_h * grid_w == N);
                           grid_h == 0 means 1-D pooling over N tokens           */
    int lm_h, lm_w;   /* landmark grid (lm_h * lm_w == m); ignored for 1-D      */
    float scale;      /* softmax scale; 0 means 1/sqrt(d)                        */
    unsigned flags;   /* MITA_FLAG_*                                             */
    int dtype;        /* mita_dtype of Q, K, V and O                             */
} mita_params;

/* Bytes of device workspace needed for `p`; 0 if `p` is invalid. On the
 * tensor-core path it holds one bf16 partial output row per (query, routed
 * slot, 256-key sub-expert), so it grows with s * ceil(k / 256): about
 * 2 * B * H * N * d * s * ceil(k / 256) bytes for those rows (2.0 GB in all at
 * B2 H16 N32768 d128, m128, k256, s2). */
size_t mita_workspace_size(const mita_params* p);

/* Landmark queries only. Qt: float32 [B, H, m, d], caller-owned device memory. */
mita_status mita_landmarks(const mita_params* p, const void* Q, float* Qt, void* ws, size_t ws_bytes,
                           void* stream);

/* Landmarks, expert index sets and routes, without the attention outputs.
 * idx: int32 [B, H, m, k], each row ascending; route: int32 [B, H, N, s],
 * descending routing score. Either output may be NULL. */
mita_status mita_select(const mita_params* p, const void* Q, const void* K, int32_t* idx, int32_t* route,
                        void* ws, size_t ws_bytes, void* stream);

/* The whole forward pass. O: [B, H, N, d] in `dtype`. idx_out ([B, H, m, k]),
 * route_out ([B, H, N, s]) and Vt_out (float32 [B, H, m, d]) are optional
 * (NULL to skip) copies of the intermediate index sets, routes and shared
 * expert values. */
mita_status mita_forward(const mita_params* p, const void* Q, const void* K, const void* V, void* O,
                         int32_t* idx_out, int32_t* route_out, float* Vt_out, void* ws, size_t ws_bytes,
                         void* stream);

/* Bytes of DEVICE memory mita_forward_host() needs: room for Q, K, V and O
 * plus the workspace. */
size_t mita_host_buffer_size(const mita_params* p);

/* The forward pass on HOST buffers: Q, K, V, O are host pointers (pinned
 * memory gives full copy speed), `dev` is caller-owned device memory of at
 * least mita_host_buffer_size() bytes. Copies Q, K, V to the device, runs the
 * forward pass, copies O back. The heads are processed in a few groups so that
 * one group's copies overlap another's compute: the copies run on two streams
 * the library keeps per device, ordered after earlier work on `stream` and
 * joined back into it, so all of the call's work is ordered on `stream`
 * (concurrent calls from several host threads enqueue one after another). The
 * call returns without waiting; the host buffers must stay valid until
 * `stream` has passed it. The device status word is the workspace's, at
 * offset 4 * align_up(B*H*N*d*element size, 1024) bytes of `dev`. */
mita_status mita_forward_host(const mita_params* p, const void* Q, const void* K, const void* V, void* O,
                              void* dev, size_t dev_bytes, void* stream);

/* Synchronizes `stream`, returns the device status word of workspace `ws`
 * (MITA_OK if no device-side error was recorded by the most recent call on
 * `ws`) and clears it. */
mita_status mita_device_status(void* ws, void* stream);

/* Static description of a status code. */
const char* mita_status_string(mita_status s);

/* Detail of the last error returned on the calling thread ("" if none). */
const char* mita_last_error(void);

/* ---- backward pass ---------------------------------------------------------
 * The summaries describe the forward pass and report training speed, but print
 * no backward pass; this one is the chain rule through the forward's steps with
 * the expert sets and routes held fixed (a top-k choice is piecewise constant
 * and has no gradient): through each query's softmax over its shared and
 * routed slots, through the shared expert Vt = softmax(scale Qt K^T) V, and
 * through the pooling of the landmarks. Runs on CUDA cores in fp32 (the inputs
 * widened from `dtype`). Non-causal, 1-D pooling only (other settings return
 * MITA_ERR_UNSUPPORTED).
 *
 * Bytes of device workspace mita_backward() needs for `p`; 0 if `p` is invalid
 * or unsupported there. */
size_t mita_backward_workspace_size(const mita_params* p);

/* Gradients of sum(O * dO) with respect to Q, K, V. Q, K, V, dO and the
 * outputs dQ, dK, dV: device [B, H, N, d] in `dtype`; idx [B, H, m, k] and
 * route [B, H, N, s]: the expert sets and routes of the forward pass whose
 * gradient is wanted (mita_forward's idx_out / route_out, or mita_select's).
 * Every output row is written. Asynchronous on `stream`; argument errors are
 * returned before anything is enqueued; an index out of range in idx or route
 * is recorded in the workspace's status word (mita_device_status on `ws`). */
mita_status mita_backward(const mita_params* p, const void* Q, const void* K, const void* V, const void* dO,
                          const int32_t* idx, const int32_t* route, void* dQ, void* dK, void* dV, void* ws,
                          size_t ws_bytes, void* stream);

/* 1 if `p` runs on the tcgen05 tensor-core path, 0 if on CUDA cores, -1 if invalid. */
int mita_uses_tensor_cores(const mita_params* p);

/* ---- forward pass without device allocation --------------------------------
 * Not part of the method (the summaries have no counterpart): an interface
 * for callers that cannot allocate device memory. Some code may not call
 * cudaMalloc at all: it can synchronize the whole device, another framework
 * may own all device memory through its own pool, or the caller is a plugin
 * that only receives the tensors it works on. mita_forward_static() is
 * mita_forward() with its workspace in a library-owned static device array of
 * MITA_STATIC_WORKSPACE_BYTES, so the caller passes only Q, K, V and O.
 *   - Problems whose mita_workspace_size() exceeds the static area are
 *     rejected with MITA_ERR_UNSUPPORTED; nothing is enqueued.
 *   - The call allocates nothing (no cudaMalloc, no allocating library call).
 *     Every GPU on which the library is loaded holds the static area until the
 *     process exits.
 *   - The first call on a device looks up the area's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture. `stream` must belong to the current device.
 *   - All calls share the one area, which keeps the last call's contents; the
 *     pass clears what must start at zero itself. Calls whose work overlaps on
 *     the GPU (different streams, or concurrent host threads) race on the area
 *     and must be serialized by the caller.
 *   - status_out (optional, device int32) receives the call's device status
 *     word (MITA_OK or MITA_ERR_TIMEOUT / MITA_ERR_BOUNDS) once the stream
 *     reaches it. */
#define MITA_STATIC_WORKSPACE_BYTES (64u << 20)
mita_status mita_forward_static(const mita_params* p, const void* Q, const void* K, const void* V, void* O,
                                int32_t* status_out, void* stream);

/* ---- 4-bit key/value cache --------------------------------------------------
 * Not part of the method (the summaries have no counterpart): what a caller
 * needs to generate with a model whose prompts went through mita_forward(). The
 * keys and values of a sequence are kept in 4 bits in pages of one pool;
 * mita_cache_write() stores rows, mita_cache_read() returns them (as contiguous
 * K and V, for another mita_forward()), and mita_cache_attention() is dense
 * softmax attention of a call's new rows over everything cached.
 *
 * Format. Each row of d channels is cut into blocks of 16. With e the exponent
 * of the row's head and y = x * 2^-e:
 *   s    = max |y| / 6, rounded to e4m3 (ties to even, at most 448);
 *   code = y / s, rounded to e2m1: 0, 1/2, 1, 3/2, 2, 3, 4 or 6 with a sign
 *          (ties to the even code, beyond 6 to 6);
 *   the value read back is code * s * 2^e, exact in bf16 and float32.
 * Both roundings are of the exact quotients. A block with s = 0 reads as zeros,
 * one that holds a NaN reads as 16 NaN, an infinity as 6 * 448 * 2^e with its
 * sign. 9/16 of a byte per channel in all. The exponent moves the
 * range that scales cover (2^-9 .. 448, and their precision falls below 2^-6);
 * it costs no accuracy, and 0 suits rows whose largest channels are between
 * about 1/10 and 2688.
 *
 * Pages. `cache` is mita_cache_size() bytes, 16-byte aligned: n_pages pages of
 * `page` tokens for all H_kv heads. Their inner order is the library's own.
 * `table` int32 [B][max_pages] names the pages of each sequence in order;
 * position i is place i % page of page table[b][i / page]. Sequences may share
 * pages that they only read.
 *
 * Rows. len int32 [B] is the number of tokens that sequence b has, the call's
 * own rows included; its rows are the last count[b] of them (count int32 [B], or
 * NULL: T each): row t is position len[b] - count[b] + t. Rows t >= count[b] are
 * padding: not read, and left as they were in outputs. exps int32 [2][H_kv]
 * (first the keys' exponents, then the values'; |e| <= 60), or NULL: all zero.
 * All four arrays are device memory and are read when the stream gets there, so
 * a captured call follows them; they stay as they are until it has ended (the results are
 * undefined otherwise). The same arrays serve all three calls: write a
 * step's rows, then attend.
 *
 * Out of range (a page outside [0, n_pages) among those that the call uses, a
 * length outside [0, max_pages * page], a count outside [0, T], for write and
 * read also count > len, an exponent outside +-60): the status word of `ws`
 * becomes MITA_ERR_BOUNDS, the places concerned are neither read nor written,
 * and what is computed from them is undefined. Every call writes the word, which
 * so holds the last call's verdict: a write's is lost if another call on the same
 * workspace follows before mita_device_status(). (Attention finds a bad page, length, count
 * or exponent again; count > len is no error there, so the rows that the write left out for
 * it then go unreported.) To read both, give the two calls a workspace each. */
typedef struct {
    int B, H, H_kv;  /* sequences, query heads, cache heads (H % H_kv == 0)     */
    int T, d;        /* rows per sequence and call; head dim: 64 or 128         */
    int page;        /* tokens per page: a multiple of 16, 16 .. 4096           */
    int n_pages;     /* pages in the pool                                       */
    int max_pages;   /* columns of the page table                               */
    float scale;     /* softmax scale; 0 means 1/sqrt(d)                        */
    unsigned flags;  /* mita_cache_attention, mita_cache_weights: MITA_FLAG_CAUSAL,
                        MITA_FLAG_SIMT, MITA_TESTFLAG_STALL_PRODUCER (see there; one
                        block of the attention, or of the weights where they run in
                        tiles, waits for a signal that does not come)          */
    int dtype;       /* mita_dtype of K, V, Q and O                             */
} mita_cache_params;

/* Bytes of the pool, and of device workspace that each of the three calls
 * needs; 0 if `p` is invalid. The workspace does not depend on the lengths.
 *
 * Attention counts its work in 32 bits: with R rows to a tile (8, 16, 32 or 64,
 * the fewest that hold T * H / H_kv or else the most: 16 for float32, 32 for
 * bf16 with d = 64, 64 with d = 128; with MITA_FLAG_SIMT 1 or 4),
 *   B * H_kv * ceil(T * H / H_kv / R) * (ceil(max_pages * page / 128) + 4) < 2^31,
 * else it is MITA_ERR_UNSUPPORTED (a prompt is attended in parts then). Storing and reading
 * have no such limit for T <= max_pages * page; for parameters that only they take
 * the workspace is what they need. */
size_t mita_cache_size(const mita_cache_params* p);
size_t mita_cache_workspace_size(const mita_cache_params* p);

/* Stores rows K, V: [B, H_kv, T, d] in `dtype`. No place may be written twice
 * in one call. */
mita_status mita_cache_write(const mita_cache_params* p, const void* K, const void* V, void* cache,
                             const int32_t* table, const int32_t* len, const int32_t* count, const int32_t* exps,
                             void* ws, size_t ws_bytes, void* stream);

/* Reads rows back into K, V: [B, H_kv, T, d] in `dtype`. With T the longest
 * sequence and count = len it returns whole sequences. K and V must not overlap. */
mita_status mita_cache_read(const mita_cache_params* p, const void* cache, const int32_t* table, const int32_t* len,
                            const int32_t* count, const int32_t* exps, void* K, void* V, void* ws, size_t ws_bytes,
                            void* stream);

/* Attention of rows Q [B, H, T, d] over the cache; query head i uses cache head
 * i / (H / H_kv). Row t sees the keys j < len[b], with MITA_FLAG_CAUSAL those up
 * to its own position (j < len[b] - (count[b] - 1 - t)); a row that sees no key
 * gets zeros. A key that a row does not see has no influence on it, whatever its
 * bytes are, and neither have the call's other rows; a row with a NaN or an
 * infinity that sees a key gets NaN. Scores times log2(e) have to be within float32's
 * range. O: [B, H, T, d] in `dtype`. lse_out (float32 [B, H, T], or NULL):
 * ln sum exp(scale q.k) over the seen keys, -infinity without any, with which the
 * rows can be joined with attention over other keys (mita_forward's shared
 * slots, say). count > len is allowed: with MITA_FLAG_CAUSAL rows before the first
 * token see none, without it every row sees all keys.
 * O must not overlap Q, nor lse_out either of them. The same call gives the same bits; how a sequence's keys
 * are divided, and so the last bits, depends on all the call's lengths.
 * Runs on tensor cores with fp32 scores, softmax statistics and sums. The weights of
 * bf16 rows are rounded to halves before they meet the values: 2^-11 each, and
 * 2^-32 of the row's largest for those below 2^-21 of it. Numbers of float32 rows
 * are the sum of two halves: 22 bits, and 2^-48 of the largest for weights below
 * 2^-26 of it. With MITA_FLAG_SIMT on CUDA cores, in fp32 throughout. */
mita_status mita_cache_attention(const mita_cache_params* p, const void* Q, const void* cache, const int32_t* table,
                                 const int32_t* len, const int32_t* count, const int32_t* exps, void* O,
                                 float* lse_out, void* ws, size_t ws_bytes, void* stream);

/* ---- what cached tokens are worth, and eviction ------------------------------
 * Not part of the method (the summaries have no counterpart): keeps the cache of a
 * long generation within a budget. After a call's rows have attended,
 * mita_cache_weights() adds the attention weight that each cached token got from
 * them to its sum; mita_cache_evict() and, for sequences that are cut again and again,
 * mita_cache_evict_aged() keep the tokens of each cache head with the
 * largest sums. Sums are float32 [B][H_kv][max_pages * page], by place.
 *
 * Weights. For each token j < len[b] and cache head h
 *   acc_out[b][h][j] = decay * acc[b][h][j]  (0 for the call's own tokens, j >= len[b] - count[b])
 *                      + sum over the rows t < count[b] and the query heads of h that see j
 *                        of exp(scale q.k_j - lse[b][head][t])
 * with the keys that a row sees, Q, table, len, count and exps as in
 * mita_cache_attention(), and lse what that call returned (any float32 [B, H, T]
 * with the rows' log sums). A token that a row does not see gets nothing of it, so a
 * row that sees no key is harmless; no weight is above 1 (a rounded lse may be below a score);
 * a row with a NaN or an infinity in Q, or whose lse
 * is NaN, makes the sums of the tokens that it sees NaN. Places j >= len[b] are left
 * as they were. acc_out may be acc; no other overlap of acc_out with anything is taken. decay is finite, >= 0; with 0 acc is not read and may be NULL. The sum
 * of an own token starts at 0 whatever its place held before, so sums need no initial value.
 * A sequence with count[b] = 0 has its sums decayed. The same call gives the same bits.
 * Scores, weights and sums are fp32; bf16 rows enter exactly, float32 rows as two halves (22 bits), but for
 * entries far below the row's largest, which are off by at most 2^-29 of it. With MITA_FLAG_SIMT fp32 throughout, on CUDA cores. The workspace is that of
 * mita_cache_workspace_size(). */
mita_status mita_cache_weights(const mita_cache_params* p, const void* Q, const void* cache, const int32_t* table,
                               const int32_t* len, const int32_t* count, const int32_t* exps, const float* lse,
                               float decay, const float* acc, float* acc_out, void* ws, size_t ws_bytes,
                               void* stream);

/* Eviction. keep int32 [B] (device): the tokens that sequence b keeps. A sequence with
 * len[b] <= keep[b] stays as it is. Of the others each cache head keeps the tokens at its first `first` and
 * its last `recent` places and, of those between, the keep[b] - first - recent with the largest
 * acc (ties to the lower place; NaN counts as the largest, -0 as 0). The kept rows at places
 * j >= keep[b] move, in ascending order, to the places that were freed below keep[b], in
 * ascending order; the other kept rows stay where they are. Keys and values move as they are
 * held, without another rounding. (Places are not positions, then: a caller that rotates by
 * position counts positions itself. Heads of one sequence keep different tokens. The last places
 * have the newest tokens the first time that a sequence is cut, and not from then on: calls that cut
 * sequences again and again take mita_cache_evict_aged().)
 *   len_out  int32 [B]: min(len[b], keep[b]). May be len.
 *   acc_out  float32 like acc: the sums of the rows now at j < len_out[b]. May be acc.
 *   src_out  int32 [B][H_kv][max_pages * page] or NULL: the place that the row now at
 *            j < len_out[b] had, to carry anything else along.
 * Places from len_out[b] on keep what they held in acc_out and src_out, and in the cache. Other
 * overlaps of outputs or of the workspace with anything are refused. Pages that the call writes (those of places below
 * keep[b] of a sequence that is cut) must not be shared with another sequence.
 * Uses B, H_kv, d, page, n_pages and max_pages of p. first, recent >= 0. Out of range: as
 * above, and a budget keep[b] below first + recent; a sequence whose length or budget is out of
 * range is left as it was, with len_out[b] = len[b].
 *
 * mita_cache_evict_aged() does the same with `recent` by age: each cache head keeps the tokens at its
 * first `first` places (they never move, so these are the sequence's first tokens if no earlier call
 * had a smaller `first`), of the others the `recent` newest that it still has, and of the rest those with
 * the largest acc, keep[b] in all. What a head has lost of the newest, to a call with a smaller `recent`,
 * others with the largest acc replace. age int32 [B][H_kv][max_pages * page], by place, changed in place, tells how
 * much older a token is than its place says: the token at place j is as old as an unmoved one at place
 * j - age[b][h][j] would be (at most 2^30 either way). Zeros are a sequence in order. The caller sets a
 * sequence's numbers to 0 when it begins and otherwise leaves them to the call: rows appended at len_out[b] and
 * behind find zeros there, and appended rows that are taken back again leave zeros (a len that falls
 * below what the last eviction left has no meaning here). age must not overlap anything. */
size_t mita_cache_evict_workspace_size(const mita_cache_params* p);
mita_status mita_cache_evict(const mita_cache_params* p, void* cache, const int32_t* table, const int32_t* len,
                             const int32_t* keep, int first, int recent, const float* acc, int32_t* len_out,
                             float* acc_out, int32_t* src_out, void* ws, size_t ws_bytes, void* stream);
mita_status mita_cache_evict_aged(const mita_cache_params* p, void* cache, const int32_t* table, const int32_t* len,
                                  const int32_t* keep, int first, int recent, const float* acc, int32_t* age,
                                  int32_t* len_out, float* acc_out, int32_t* src_out, void* ws, size_t ws_bytes,
                                  void* stream);

/* ---- rotary positions ----------------------------------------------------------
 * Not part of the method (the summaries have no counterpart): turns the rows of Q and K by
 * their positions before mita_forward(), mita_cache_write() and mita_cache_attention().
 * Pair i of the first `rot` channels of a row at position t is turned by the angle
 * a = t * freqs[i] and scaled:
 *   y0 = gain (x0 cos a - x1 sin a),  y1 = gain (x0 sin a + x1 cos a);
 * the other channels are copied. Pair i is channels i and i + rot / 2, or with
 * MITA_FLAG_INTERLEAVED 2 i and 2 i + 1. Angles are reduced exactly in 64-bit integers (a
 * position times a frequency in turns, which is off by at most 2^-63 of a turn and 2^-104 of itself), so far
 * positions lose nothing: cos and sin are off by about 2^-23 at every position, for frequencies up to 2^40. Products and sums are fp32, rounded once to `dtype`. */
#define MITA_ROPE_PAIRS 128
typedef struct {
    int B, H, H_kv;   /* sequences, query heads, key heads (H_kv = 0: Q alone)     */
    int T, d;         /* rows per sequence; head dim: even, 2 .. 256               */
    int rot;          /* channels that are rotated: even, 2 .. d                   */
    float gain;       /* 0 means 1                                                 */
    unsigned flags;   /* MITA_FLAG_INTERLEAVED                                     */
    int dtype;        /* mita_dtype of all rows                                    */
    double freqs[MITA_ROPE_PAIRS]; /* radians per position of pair i < rot / 2     */
} mita_rope_params;

enum {
    MITA_ROPE_PLAIN = 0,  /* base^(-2 i / rot)                                                     */
    MITA_ROPE_LINEAR = 1, /* that / factor: positions of a longer context squeezed into the first  */
    MITA_ROPE_NTK = 2,    /* base * factor^(rot / (rot - 2)) in place of base: the slowest pair
                             is slowed by factor, the fastest not (rot = 2: plain)                 */
    MITA_ROPE_PARTS = 3   /* by the turns r = original f / (2 pi) that a pair makes over the
                             original length: f (g + (1 - g) / factor) with
                             g = clamp((r - low) / (high - low), 0, 1)                             */
};

/* Fills p->freqs[0 .. rot / 2) (of p only rot is read). base > 1; factor >= 1 for the scaled
 * forms; original > 0 and low < high for MITA_ROPE_PARTS (ignored otherwise). */
mita_status mita_rope_frequencies(mita_rope_params* p, double base, int scaling, double factor, double original,
                                  double low, double high);

/* Rotates Q [B, H, T, d] into Qo and K [B, H_kv, T, d] into Ko (K and Ko NULL with H_kv = 0).
 * strides: 12 numbers of elements (host memory): batch, head and row stride of Q, K, Qo and Ko in turn;
 * NULL: all contiguous. So a projection's [B, T, heads, d] can be read where it is and written as
 * the other calls want it. Channels are contiguous. Inputs may repeat rows (stride 0), an
 * output's rows must not overlap. Qo may be Q with the same strides (in place), Ko likewise K;
 * an output must not share elements with anything else: what cannot be told apart by its range, or
 * row by row with equal batch and row strides, is refused. pos int32 (device): row t of
 * sequence b is at position pos[b * pos_stride + t] (any int32; pos_stride >= 0, 0 for positions
 * that all sequences share); NULL: at t. Pointers are aligned to their elements; 16-byte aligned
 * rows are faster. No workspace, no device status. */
mita_status mita_rope(const mita_rope_params* p, const void* Q, const void* K, void* Qo, void* Ko,
                      const int64_t* strides, const int32_t* pos, int64_t pos_stride, void* stream);

/* The backward pass: the transposed map (angles negated, the same gain) of gradients dQo, dKo with
 * respect to the rotated rows into dQ, dK. Its arguments are those of mita_rope. */
mita_status mita_rope_backward(const mita_rope_params* p, const void* dQo, const void* dKo, void* dQ, void* dK,
                               const int64_t* strides, const int32_t* pos, int64_t pos_stride, void* stream);

/* ---- measurement hooks (not part of the method) ---------------------------
 * Number of kernels this library has launched in the process so far. */
long long mita_launch_count(void);

/* Opens a phase profile: until mita_profile_end(), every call records a CUDA
 * event on its stream at the start of each phase (landmark pooling, top-k
 * sample and threshold, landmark pass, top-k selection, shared-expert combine,
 * routing, bucketing, the shared slots' own pass when there are more than 128
 * landmarks, expert attention, merge; the cache calls: write, read, attention,
 * join, weights, evict; rope) and at its end; up to max_marks events
 * in total (created here, kept for reuse). Process-wide; not for concurrent
 * calls. */
mita_status mita_profile_begin(int max_marks);

/* Closes the profile: waits for the last event, sums the milliseconds of each
 * phase over all profiled calls into ms[i] and writes the phase names,
 * newline-separated, into `names`. Returns the number of phases (<= max_phases)
 * or -1 on a CUDA error. */
int mita_profile_end(char* names, size_t names_bytes, double* ms, int max_phases);

#ifdef __cplusplus
}
#endif

#endif /* MITA_H */
