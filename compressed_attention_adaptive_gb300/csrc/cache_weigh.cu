// The attention weight that each cached token gets from a call's rows (format and layout of
// the cache: cache.cuh):
//
//   acc'_j = decay acc_j + sum over rows r that see j of exp(scale q_r.k_j - lse_r)
//
// With the rows' log sums given there is no maximum to find and no sum over tokens: a token's sum needs
// its own key alone, so tokens can be cut anywhere and nothing is joined. It reads
// d/2 + d/16 + 4 bytes per token and cache head, writes 4, and does 2 d flops and an exponential
// per row.
//
// Work split. The steps of 32 tokens of all (sequence, cache head) form one line, cut into equal
// parts, one per warp; warps share nothing but the search for their place. A token's sum is
// added in an order of its own, whatever the cut, so the same call gives the same bits.
//
// Measured, in a graph: one row over 2 x 16 heads of 32768 tokens 20.1 us (4.2 TB/s, 0.61 of the copy rate), 64 sequences
// of 33 to 8191 tokens, four rows over 8 heads 40.7. A kernel that only reads the first's 75 MB of keys takes 17.9 us (events
// around it), every other 1152 bytes, as here, or in one run; only more of them come faster (600 MB at 0.91 of the copy
// rate, in one run at 0.95). Float32, one row: 21.4.
#include <algorithm>

#include "cache_weigh.cuh"

namespace mita {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;  // of a block
constexpr int kTok = 2 * kGroup;                       // tokens of a warp's step
constexpr int kRaw = 2;                                // stages of a warp's codes and scales in shared memory

}  // namespace

// The call's first block: its status word.
__device__ __forceinline__ void check(const CacheArgs& a) {
    const bool bad = __syncthreads_or(bad_call<true>(a));
    if (threadIdx.x == 0) *a.status = bad ? kStBounds : kStOk;
}

// ------------------------------------------------------------ CUDA cores

// fp32 throughout: eight lanes share a token, each with the d/8 channels of two blocks' halves or of one
// block, and a warp takes four tokens at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_cache_weigh_simt(CacheArgs a, WeighArgs w, const T* __restrict__ Q, const uint8_t* __restrict__ cache) {
    using L = Grp<D>;
    constexpr int E = D / 8;  // channels of a lane
    __shared__ LineStart<kThreads> start;
    if (blockIdx.x == 0) {
        check(a);
        return;
    }
    const int lane = threadIdx.x & 31, sub = lane >> 3, ch = lane & 7, blk = D == 128 ? ch : ch >> 1;
    Place<kTok, kThreads> at;
    at.begin<true>(a, start, (long long)(blockIdx.x - 1) * kWarps + (threadIdx.x >> 5), (long long)(gridDim.x - 1) * kWarps);
    if (at.left == 0) return;
    do {
        for (int gi = 2 * at.at; gi < 2 * at.at + 2 && gi * kGroup < at.n; ++gi) {
            const int group = cache_group(a, at.b, at.h, gi);
            if (group < 0) continue;
            const uint8_t* gr = cache + (long long)group * L::kBytes;
            const float f = a.scale * pow2(cache_exp(a, 0, at.h));
            float k[4][E], sum[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int tok = 4 * u + sub;
                sum[u] = 0.0f;
                const uint32_t sb = gr[L::k_scale(tok, blk)], s2 = e4m3x2_to_half2(sb | sb << 8);
#pragma unroll
                for (int i = 0; i < E / 8; ++i) {
                    uint32_t r[4];
                    e2m1x8_to_half2(reinterpret_cast<const uint32_t*>(gr + tok * L::kRow)[ch * (E / 8) + i], r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = half2_to_float2(hmul2(r[j], s2));
                        k[u][8 * i + 2 * j] = x.x;
                        k[u][8 * i + 2 * j + 1] = x.y;
                    }
                }
            }
            const int rows = at.count * a.G;
            for (int r = 0; r < rows; ++r) {
                int t;
                const long long row = row_offset(a, at.b, at.h, r, &t);
                const int lim = row_limit(a, at.n, at.count, t);
                if (lim <= gi * kGroup) continue;
                float q[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float x = to_f(Q[row * D + ch * E + i]);
                    q[i] = isfinite(x) ? x : __int_as_float(0x7fc00000);  // the row becomes NaN, as its softmax is
                }
                const float lse = w.lse[row];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float z = 0.0f;
#pragma unroll
                    for (int i = 0; i < E; ++i) z = fmaf(q[i], k[u][i], z);
#pragma unroll
                    for (int x = 4; x; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
                    if (gi * kGroup + 4 * u + sub < lim) sum[u] += weight(z, f, lse);
                }
            }
            const long long base = ((long long)at.b * a.Hkv + at.h) * w.cap;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = gi * kGroup + 4 * u + sub;
                if (ch || j >= at.n) continue;
                if (w.decay != 0.0f && j < at.n - at.count) sum[u] = fmaf(w.decay, w.acc[base + j], sum[u]);
                w.acc_out[base + j] = sum[u];
            }
        }
    } while (at.next(a, 1));
}

// --------------------------------------------------------- tensor cores

// Q's halves of a warp in shared memory (float rows are two of them), or in registers where they are few
template <typename T, int D, int NR, bool FEW> constexpr bool q_regs() { return FEW || (NR == 1 && sizeof(T) == 2); }
template <typename T, int D, int NR, bool FEW> constexpr int q_bytes() {
    return q_regs<T, D, NR, FEW>() ? 0 : (sizeof(T) == 4 ? 2 : 1) * NR * (D / 16) * 256;
}

// Blocks of an SM. (Eight bf16 rows: 64 sequences of 33 to 8191 tokens, 8 cache heads: 47.1 us with two, 41.1 with
// three, 47.6 with four; 2 x 16 heads of 32768: 21.2, 23.0 and 27.6. Float rows lose from three on.) Three leave 80 registers, and
// d = 128 spills 32 bytes for one and two rows, 64 for up to eight: 0.4 % of the executed instructions with the
// first shape, 0.7 % with the second, read back from L1.
template <typename T, int NR> constexpr int weigh_blocks() { return NR == 1 && sizeof(T) == 2 ? 3 : 2; }

// Scores on m16n8k16 steps (halves in, fp32 out), tokens on the 16 side and 8 NR query rows on the 8 side.
//
// The lanes of a warp copy the codes of a group in the order in which they feed the steps, 16
// bytes each for d = 128 and neighbours next to each other, into a part of shared memory that is the warp's own, so that
// the next step, two groups, is on its way without registers, and no warp waits for another. (Loads into registers two
// steps ahead: 24.7 us for 2 x 16 heads of 32768 tokens, 20.2 so; copies two or three steps ahead 23.0 and more, with
// fewer blocks 19.7.) Widening is exact (cache.cuh). Rows are scaled by a power of two that puts the largest entry in
// [2^14, 2^15): bf16 rows are exact as halves down to 2^-31 of it; float32 rows are two halves, hi + lo, in sums of their own
// (a sum is cut to 24 bits at every step; what the lower halves add should not be cut at the size of the whole).
// A lane ends with two tokens of each group and two rows for each eight; four lanes share a token.
//
// FEW: with two rows, of the eight columns of the 8 side a row has four, each with the channels of every fourth block of
// its own and zeros elsewhere. The sums of the blocks of 16 channels come out apart, so that scales are multiplied into them
// (4 d/64 products for two tokens) and not into the codes (32 d/128 for them), and of what the step ends with
// no column is empty: a lane has one score and one exponential for each group.
template <typename T, int D, int NR, bool FEW>
__global__ void __launch_bounds__(kThreads, weigh_blocks<T, NR>())
k_cache_weigh(CacheArgs a, WeighArgs w, const T* __restrict__ Q, const uint8_t* __restrict__ cache) {
    using L = Grp<D>;
    constexpr bool F = sizeof(T) == 4;  // float rows
    constexpr bool kQRegs = q_regs<T, D, NR, FEW>();
    constexpr int KS = D / 16, W = D / 32, RT = (FEW ? 2 : 8) * NR, KW = D / 64;  // KW: 8-byte words of a lane's codes of a token
    constexpr int SW = FEW && D == 128 ? 2 : 1;                                   // words of a lane's scales of a group
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineStart<kThreads> start;
    if (blockIdx.x == 0) {
        check(a);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    uint2* qs = reinterpret_cast<uint2*>(smem + warp * q_bytes<T, D, NR, FEW>());
    const uint32_t ring = tc::smem_u32(smem) + kWarps * q_bytes<T, D, NR, FEW>() + warp * (kRaw * 18 * D);
    Place<kTok, kThreads> at;
    at.begin<true>(a, start, (long long)(blockIdx.x - 1) * kWarps + warp, (long long)(gridDim.x - 1) * kWarps);
    if (at.left == 0) return;
    for (bool more = true; more;) {
        const int cnt = (int)min(at.left, (long long)(at.steps - at.at)), n = at.n, step0 = at.at;
        const int rows = at.count * a.G;
        // the lane's token of step 0
        const long long sums = ((long long)at.b * a.Hkv + at.h) * w.cap + (long long)step0 * kTok + 8 * t4 + g;
        const int codes = g * L::kRow + t4 * (D / 8);
        const int scales = L::kKs + g * (D / 8) + (FEW ? (t4 & 1) * (D / 16) : t4 * (D / 32));
        // lane l: group l % 2 of step i + l / 2
        auto groups = [&](int i) {
            const int gi = 2 * (step0 + i) + lane;
            return i + (lane >> 1) < cnt && gi * kGroup < n ? cache_group(a, at.b, at.h, gi) : -1;
        };
        // Rows in tiles: the first starts from what the tokens had, the others add to what is there
        // (a lane reads what it wrote itself).
        for (int row0 = 0; row0 < max(rows, 1); row0 += RT) {
            const float* had = (row0 ? w.acc_out : w.acc) + sums;
            const float decay = row0 ? 1.0f : w.decay;
            // steps' tokens of the lane with a sum: those before step `olds`
            const int olds = (row0 ? n : w.decay != 0.0f ? n - at.count : 0) - (step0 * kTok + 8 * t4 + g);
            int gcur = groups(0), gnxt = groups(16);
            uint32_t ok = 0;
            float base[kRaw];
            // Step i into stage u (that of i modulo kRaw); called for every i in turn. A lane copies the codes that it will read, and
            // scales for its neighbours.
            auto copy = [&](int u, int i) {
                ok &= ~(3u << 2 * u);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int grp = __shfl_sync(0xffffffffu, gcur, 2 * (i & 15) + y);
                    if (grp < 0) continue;
                    ok |= 1u << (2 * u + y);
                    const uint8_t* src = cache + (unsigned long long)(unsigned)grp * L::kBytes;
                    const uint32_t dst = ring + (u * 2 + y) * (9 * D);
#pragma unroll
                    for (int x = 0; x < 2; ++x) copy_async<D / 8>(dst + codes + 8 * x * L::kRow, src + codes + 8 * x * L::kRow);
                    if (D == 128 || lane < 16) copy_async<4>(dst + L::kKs + 4 * lane, src + L::kKs + 4 * lane);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                base[u] = i < cnt && i * kTok < olds ? had[(long long)i * kTok] : 0.0f;
                if ((i & 15) == 15) {
                    gcur = gnxt;
                    gnxt = groups(i + 17);
                }
            };
#pragma unroll
            for (int u = 0; u < kRaw - 1; ++u) copy(u, u);

            // Q: lane (g, t4) has channels [t4 d/4, (t4 + 1) d/4) of rows g, and what it needs of
            // rows 2 t4 and the next: factor of the scores, lse, keys that they see. (FEW: of row g / 4, if t4 is g % 4,
            // and what it needs of row t4 / 2.)
            constexpr int kParts = F ? 2 : 1;
            uint2 qf[kQRegs ? kParts * KS * NR : 1];
            float2 zf[NR], lse[NR];  // (lse negated)
            int2 lim[NR];
            int low = 0, top = 0;
            __syncwarp();  // all have read the tile before
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const int r = row0 + (FEW ? 2 * j + (g >> 2) : 8 * j + g);
                const bool mine = r < rows && (!FEW || t4 == (g & 3));
                int t = 0;
                const long long row = row_offset(a, at.b, at.h, min(r, max(rows - 1, 0)), &t);
                constexpr int QW = D / 16 * sizeof(T) / 4;  // 16-byte words of a lane's channels
                uint32_t x[4 * QW], amax = 0;
#pragma unroll
                for (int i = 0; i < QW; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (mine) v = reinterpret_cast<const uint4*>(Q + row * D + t4 * (D / 4))[i];
                    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
                }
                // (a row that is not there: weights of 0)
                const float l = r < rows ? w.lse[row] : INFINITY;
                const int m = r < rows ? row_limit(a, n, at.count, t) : 0;
#pragma unroll
                for (int i = 0; i < 4 * QW; ++i)
                    amax = max(amax, F ? x[i] & 0x7fffffffu : max(x[i] << 16 & 0x7fff0000u, x[i] & 0x7fff0000u));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                if (FEW) {
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
                }
                float up;
                const int qe = query_exp(amax >> 23, &up);
                const float f = fminf(a.scale * pow2(cache_exp(a, 0, at.h)) * pow2(-qe), 3.4028235e38f);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y0 = __uint_as_float(F ? x[(4 * ks + 2 * e) % (4 * QW)] : x[2 * ks + e] << 16) * up;
                        const float y1 = __uint_as_float(F ? x[(4 * ks + 2 * e + 1) % (4 * QW)] : x[2 * ks + e] & 0xffff0000u) * up;
                        hi[e] = pack_half2(y0, y1);
                        const float2 h = half2_to_float2(hi[e]);
                        lo[e] = pack_half2(y0 - h.x, y1 - h.y);
                    }
                    if (FEW && t4 != (g & 3)) hi[0] = hi[1] = lo[0] = lo[1] = 0;  // (0 times a NaN would not be)
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        const uint2 q = part ? make_uint2(lo[0], lo[1]) : make_uint2(hi[0], hi[1]);
                        if (kQRegs)
                            qf[((part * KS + ks) * NR + j) % (kQRegs ? kParts * KS * NR : 1)] = q;
                        else
                            qs[((part * KS + ks) * NR + j) * 32 + lane] = q;
                    }
                }
                // lanes with rows 2 t4 and the next (FEW: with row t4 / 2)
                const int r0 = FEW ? 8 * (t4 & 2) : 8 * t4, r1 = FEW ? r0 : r0 + 4;
                zf[j] = make_float2(__shfl_sync(0xffffffffu, f, r0), __shfl_sync(0xffffffffu, f, r1));
                lse[j] = make_float2(-__shfl_sync(0xffffffffu, l, r0), -__shfl_sync(0xffffffffu, l, r1));
                lim[j] = make_int2(__shfl_sync(0xffffffffu, m, r0), __shfl_sync(0xffffffffu, m, r1));
            }
            if (rows) {  // keys that the tile's first and last row see: later tokens see more
                low = row_limit(a, n, at.count, row0 / a.G);
                top = row_limit(a, n, at.count, min(row0 + RT - 1, rows - 1) / a.G);
            }
            __syncwarp();

            for (int i0 = 0; i0 < cnt; i0 += kRaw) {
#pragma unroll
                for (int u = 0; u < kRaw; ++u) {
                    const int i = i0 + u, tok = (step0 + i) * kTok;
                    float sum = 0.0f;
                    const float was = base[u];
                    const bool in = i < cnt && tok + 8 * t4 + g < n && (ok >> (2 * u + (t4 >> 1)) & 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 2) : "memory");
                    __syncwarp();
                    copy((u + kRaw - 1) % kRaw, i + kRaw - 1);  // (over what all lanes read before the barrier)
                    if (i < cnt && tok < top) {
                        uint2 kc[2][2][KW];  // [group][token g, g + 8]
                        uint32_t sc[2][SW];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t src = ring + (u * 2 + y) * (9 * D);
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t p = src + codes + 8 * x * L::kRow;
                                if (D == 128)
                                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                                 : "=r"(kc[y][x][0].x), "=r"(kc[y][x][0].y), "=r"(kc[y][x][KW - 1].x),
                                                   "=r"(kc[y][x][KW - 1].y)
                                                 : "r"(p));
                                else
                                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(kc[y][x][0].x), "=r"(kc[y][x][0].y) : "r"(p));
                            }
                            if (SW == 2)
                                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(sc[y][0]), "=r"(sc[y][SW - 1]) : "r"(src + scales));
                            else if (D == 128 || FEW)
                                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc[y][0]) : "r"(src + scales));
                            else
                                asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc[y][0]) : "r"(src + scales));
                        }
                        const bool edge = tok + kTok > low;  // some row does not see all of these tokens
                        auto rows_of = [&](int part, int ks, int j) {
                            const int at = (part * KS + ks) * NR + j;
                            return kQRegs ? qf[at % (kQRegs ? kParts * KS * NR : 1)] : qs[at * 32 + lane];
                        };
                        const bool odd = t4 & 1, up = t4 & 2;
                        if constexpr (FEW) {
                            float w2[2];  // [group]: of the lane's token and rows
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                constexpr int HF = D / 64;  // blocks of a lane's channels
                                float z[NR][HF][4], zl[F ? NR : 1][HF][4];  // (lower halves in a sum of their own: sums are cut to 24 bits)
#pragma unroll
                                for (int wi = 0; wi < W; ++wi) {
                                    uint32_t k8[2][4];
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
                                        e2m1x8_to_half2(wi & 1 ? kc[y][x][wi / 2].y : kc[y][x][wi / 2].x, k8[x]);
#pragma unroll
                                    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                                        for (int part = 0; part < kParts; ++part)
#pragma unroll
                                            for (int j = 0; j < NR; ++j) {
                                                const int ks = 2 * wi + k2;
                                                const uint2 q = rows_of(part, ks, j);
                                                float* to = part ? zl[F ? j : 0][ks / 4] : z[j][ks / 4];
                                                if (ks % 4 == 0)
                                                    mma_f16_first(to, k8[0][2 * k2], k8[1][2 * k2], k8[0][2 * k2 + 1],
                                                                  k8[1][2 * k2 + 1], q.x, q.y);
                                                else
                                                    mma_f16(to, k8[0][2 * k2], k8[1][2 * k2], k8[0][2 * k2 + 1], k8[1][2 * k2 + 1],
                                                            q.x, q.y);
                                            }
                                }
                                if (F) {
#pragma unroll
                                    for (int i = 0; i < NR * HF * 4; ++i) (&z[0][0][0])[i] += (&zl[0][0][0])[F ? i : 0];
                                }
                                float s[2][2][HF];  // [token g, g + 8][column][block]
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    if (D == 128) {
                                        const uint32_t two = sc[y][c % SW];
                                        const float2 a0 = half2_to_float2(e4m3x2_to_half2(two & 0xffff));
                                        const float2 a1 = half2_to_float2(e4m3x2_to_half2(two >> 16));
                                        s[0][c][0] = a0.x; s[0][c][HF - 1] = a0.y;
                                        s[1][c][0] = a1.x; s[1][c][HF - 1] = a1.y;
                                    } else {
                                        const uint32_t two = sc[y][0] >> 16 * c & 0xffff;
                                        const float2 a0 = half2_to_float2(e4m3x2_to_half2(two));
                                        s[0][c][0] = a0.x;
                                        s[1][c][0] = a0.y;
                                    }
                                }
#pragma unroll
                                for (int j = 0; j < NR; ++j) {
                                    float v[2];
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        v[x] = z[j][0][2 * x] * s[x][0][0];
#pragma unroll
                                        for (int i = 1; i < 2 * HF; ++i)
                                            v[x] = fmaf(z[j][i / 2][2 * x + (i & 1)], s[x][i & 1][i / 2], v[x]);
                                    }
                                    const float mine = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
                                    float p = weight(mine, zf[j].x, -lse[j].x);
                                    if (edge && tok + kGroup * y + 8 * (t4 & 1) + g >= lim[j].x) p = 0.0f;
                                    w2[y] = j ? w2[y] + p : p;
                                }
                            }
                            sum = (up ? w2[1] : w2[0]) + __shfl_xor_sync(0xffffffffu, up ? w2[0] : w2[1], 2);
                        } else {
                            float2 s2t[2][2];  // [group][token g, g + 8], two rows each
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                uint32_t s2[2][KW];  // [token g, g + 8]: scales, each in both halves
                                if (D == 128) {
                                    const uint32_t a0 = e4m3x2_to_half2(sc[y][0] & 0xffff), a1 = e4m3x2_to_half2(sc[y][0] >> 16);
                                    s2[0][0] = __byte_perm(a0, a0, 0x1010);
                                    s2[0][KW - 1] = __byte_perm(a0, a0, 0x3232);
                                    s2[1][0] = __byte_perm(a1, a1, 0x1010);
                                    s2[1][KW - 1] = __byte_perm(a1, a1, 0x3232);
                                } else {
                                    const uint32_t a0 = e4m3x2_to_half2(sc[y][0]);
                                    s2[0][0] = __byte_perm(a0, a0, 0x1010);
                                    s2[1][0] = __byte_perm(a0, a0, 0x3232);
                                }
                                float z[NR][4], zl[F ? NR : 1][4];
#pragma unroll
                                for (int wi = 0; wi < W; ++wi) {
                                    uint32_t k8[2][4];
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        e2m1x8_to_half2(wi & 1 ? kc[y][x][wi / 2].y : kc[y][x][wi / 2].x, k8[x]);
#pragma unroll
                                        for (int j = 0; j < 4; ++j) k8[x][j] = hmul2(k8[x][j], s2[x][wi / 2]);
                                    }
#pragma unroll
                                    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                                        for (int j = 0; j < NR; ++j) {
                                            const int ks = 2 * wi + k2;
                                            const uint2 q = rows_of(0, ks, j);
                                            if (ks == 0)
                                                mma_f16_first(z[j], k8[0][0], k8[1][0], k8[0][1], k8[1][1], q.x, q.y);
                                            else
                                                mma_f16(z[j], k8[0][2 * k2], k8[1][2 * k2], k8[0][2 * k2 + 1], k8[1][2 * k2 + 1],
                                                        q.x, q.y);
                                            if (F) {
                                                const uint2 ql = rows_of(1, ks, j);
                                                if (ks == 0)
                                                    mma_f16_first(zl[F ? j : 0], k8[0][0], k8[1][0], k8[0][1], k8[1][1], ql.x, ql.y);
                                                else
                                                    mma_f16(zl[F ? j : 0], k8[0][2 * k2], k8[1][2 * k2], k8[0][2 * k2 + 1],
                                                            k8[1][2 * k2 + 1], ql.x, ql.y);
                                            }
                                        }
                                }
                                s2t[y][0] = s2t[y][1] = make_float2(0.0f, 0.0f);
                                if (F) {
#pragma unroll
                                    for (int i = 0; i < NR * 4; ++i) (&z[0][0])[i] += (&zl[0][0])[F ? i : 0];
                                }
#pragma unroll
                                for (int j = 0; j < NR; ++j) {
                                    float2 p0 = weight2(make_float2(z[j][0], z[j][1]), zf[j], lse[j]);
                                    float2 p1 = weight2(make_float2(z[j][2], z[j][3]), zf[j], lse[j]);
                                    if (edge) {
                                        const int t0 = tok + kGroup * y + g;
                                        if (t0 >= lim[j].x) p0.x = 0.0f;
                                        if (t0 >= lim[j].y) p0.y = 0.0f;
                                        if (t0 + 8 >= lim[j].x) p1.x = 0.0f;
                                        if (t0 + 8 >= lim[j].y) p1.y = 0.0f;
                                    }
                                    s2t[y][0] = j ? add2(s2t[y][0], p0) : p0;
                                    s2t[y][1] = j ? add2(s2t[y][1], p1) : p1;
                                }
                            }
                            // over the four lanes of a token: lane t4 ends with token 8 t4 + g of the step
                            float2 k0 = up ? s2t[1][0] : s2t[0][0], k1 = up ? s2t[1][1] : s2t[0][1];
                            const float2 g0 = up ? s2t[0][0] : s2t[1][0], g1 = up ? s2t[0][1] : s2t[1][1];
                            float x0 = k0.x + k0.y + __shfl_xor_sync(0xffffffffu, g0.x + g0.y, 2);
                            float x1 = k1.x + k1.y + __shfl_xor_sync(0xffffffffu, g1.x + g1.y, 2);
                            sum = (odd ? x1 : x0) + __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 1);
                        }
                    }
                    if (in) w.acc_out[sums + (long long)i * kTok] = fmaf(decay, was, sum);
                }
            }
            tc::cp_async_wait_all();
            __syncwarp();
        }
        more = at.next(a, cnt);
    }
}

// ------------------------------------------------------------------ launch

// The block that checks, and those with parts of the line: `blocks` on each SM in all.
static unsigned weigh_grid(const CacheArgs& a, const WeighArgs& w, int blocks) {
    const long long steps = (long long)a.B * a.Hkv * ((w.cap + kTok - 1) / kTok);
    return (unsigned)std::min<long long>((steps + kWarps - 1) / kWarps + 1, (long long)blocks * num_sms());
}

template <typename T, int D, int NR, bool FEW = false>
static cudaError_t mma_t(const CacheArgs& a, const WeighArgs& w, const void* Q, const uint8_t* cache, cudaStream_t st) {
    constexpr int smem = kWarps * (q_bytes<T, D, NR, FEW>() + kRaw * 18 * D);
    static std::atomic<unsigned long long> done{0};
    if (smem > 40 * 1024) {
        const cudaError_t e = set_smem_once((const void*)k_cache_weigh<T, D, NR, FEW>, smem, &done);
        if (e != cudaSuccess) return e;
    }
    k_cache_weigh<T, D, NR, FEW><<<weigh_grid(a, w, weigh_blocks<T, NR>()), kThreads, smem, st>>>(a, w, (const T*)Q, cache);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t weigh_t(const CacheArgs& a, const WeighArgs& w, unsigned flags, const void* Q, const uint8_t* cache,
                           cudaStream_t st) {
    if (flags & MITA_FLAG_SIMT) {
        k_cache_weigh_simt<T, D><<<weigh_grid(a, w, 4), kThreads, 0, st>>>(a, w, (const T*)Q, cache);
        count_launch();
        return cudaGetLastError();
    }
    const long long rows = (long long)a.G * a.T;
    // From how many rows on tiles on tcgen05 take less. Microseconds here and there for 8 heads of 1000 tokens, 2 x 8 of
    // 32768, 64 x 8 of 300: bf16, d = 128, 16 rows 5.8/7.1, 16.2/22.7, 10.3/17.7; 32 rows 9.1/7.1, 31.4/22.7, 18.4/17.7;
    // float32, 8 rows 6.1/7.3, 16.6/23.1, 11.1/18.2, 16 rows 8.4/7.3, 27.7/23.0, 17.4/18.1; d = 64, bf16, 32 rows 6.5,
    // 18.2 and 11.6 here, 33 rows 7.8, 22.8 and 18.7 there (two passes here, 64 rows: 10.1, 33.9 and 20.3).
    constexpr int kMost = D == 64 ? 32 : sizeof(T) == 4 ? 8 : 16;
    if (rows > kMost) return launch_cache_weigh_tile(a, w, D, sizeof(T) == 4 ? 0 : 1, Q, cache, st);
    // (2 x 16 heads of 32768 tokens, one row each: 19.7 us, and 21.4 in the form for eight rows; float32 21.4 and 23.2; d = 64 15.3 and
    // 15.9, 17.2 and 17.7. Four rows in two tiles of two: 23.6 against 22.8, and 64 sequences of 33 to 8191 tokens 56.6 against
    // 40.3, as each further step of the tensor cores takes its 17 clocks.)
    if (rows <= 2) return mma_t<T, D, 1, true>(a, w, Q, cache, st);
    if constexpr (kMost > 8) {
        if (rows > 16) return mma_t<T, D, kMost == 32 && sizeof(T) == 2 ? 4 : 2>(a, w, Q, cache, st);  // (float: two tiles of 16)
        if (rows > 8) return mma_t<T, D, 2>(a, w, Q, cache, st);
    }
    return mma_t<T, D, 1>(a, w, Q, cache, st);
}

cudaError_t launch_cache_weigh(const CacheArgs& a, int d, int dtype, unsigned flags, const void* Q, const void* cache,
                               const float* lse, float decay, const float* acc, float* acc_out, cudaStream_t st) {
    const WeighArgs w{lse, acc, acc_out, decay, (long long)a.cols * a.page};
    const uint8_t* c = (const uint8_t*)cache;
    prof_mark(st, "cache_weights");
    if (dtype == 0) return d == 64 ? weigh_t<float, 64>(a, w, flags, Q, c, st) : weigh_t<float, 128>(a, w, flags, Q, c, st);
    return d == 64 ? weigh_t<__nv_bfloat16, 64>(a, w, flags, Q, c, st)
                   : weigh_t<__nv_bfloat16, 128>(a, w, flags, Q, c, st);
}

}  // namespace mita
