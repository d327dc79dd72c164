// Rotary positions: y0 = gain (x0 cos a - x1 sin a), y1 = gain (x0 sin a + x1 cos a) for the pairs of a
// row's first `rot` channels, a = position * frequency; the other channels are copied.
//
// Each row is read and written once, 6 operations per pair, so long calls are bound by HBM
// and calls of a few tokens by the launch. The angle depends on token and pair alone: a thread
// has one place of a row and goes over the heads of Q and K with its cos and sin in registers, so
// that these cost it once per token what a head's row costs.
//
// Angles. A frequency is held in turns per position as a 64-bit fraction (host: in two doubles, to 2^-63 of a turn, so
// 2^-32 of one at the farthest position); position * fraction in integers wraps at whole turns, which is the reduction,
// exactly. The signed fraction goes to sincospi as a float: 2^-24 of the angle in (-pi, pi].
//
// Measured: queries and keys of two prompts of 32768, 16 heads each, d = 128, out of a projection's order
// (1074 MB) 167 us (6.4 TB/s, 0.95 of the copy rate), 131,072 rows of 10 heads in place of
// order 99 us (0.99). One token of 64 sequences, 40 heads: 3.4 us, a launch and three memory latencies.
//   - 16-byte accesses, four heads' loads and then their stores: 253 and 155 us; 16 bytes with the next
//     heads' loads ahead: 235 and 145; 32 bytes with them ahead: 167 and 99.
// Halves that are no multiple of 16 go by narrower accesses: d = 80 in 16 bytes 173 us (0.57 of the copy rate), d = 72 and
// 40 in 4 bytes 366 (0.24) and 178 (0.28); d = 64 in 32 bytes 88 (0.90).
#include <math.h>

#include "rope.cuh"

namespace mita {

constexpr int kRopeThreads = 256;

// V elements of a row, one access of up to 32 bytes.
template <typename T, int V> struct alignas(sizeof(T) * V) Elems {
    T x[V];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (sizeof(T) * V == 32) {
            uint32_t* r = reinterpret_cast<uint32_t*>(x);
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                         : "l"(p));
        } else {
            *this = *reinterpret_cast<const Elems*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (sizeof(T) * V == 32) {
            const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
            asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                         "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "l"(p)
                         : "memory");
        } else {
            *reinterpret_cast<Elems*>(p) = *this;
        }
    }
};

// T: element; IL: interleaved pairs; V: elements of an access. A unit of a rotated place is V pairs (two accesses),
// or one access of V / 2 interleaved pairs.
template <typename T, bool IL, int V>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeArgs a) {
    constexpr bool kOne = IL && V > 1;    // one access holds whole pairs
    constexpr int P = kOne ? V / 2 : V;   // pairs of a unit
    constexpr int N = kOne ? 1 : 2;       // accesses of a unit
    constexpr int kHeads = std::max(1, 64 / (N * V * (int)sizeof(T)));  // heads loaded together, twice over
    using E = Elems<T, V>;
    const int units = a.rot / 2 / P, slots = units + (a.d - a.rot) / V;
    const int mine = threadIdx.x / slots, slot = threadIdx.x - mine * slots, rows = kRopeThreads / slots;
    const long long r = (long long)blockIdx.x * rows + mine;
    if (mine >= rows || r >= (long long)a.B * a.T) return;
    const int b = (int)(r / a.T), t = (int)(r - (long long)b * a.T);
    const bool turn = slot < units;
    // channels of the unit's accesses
    const int c0 = !turn ? a.rot + (slot - units) * V : IL ? slot * 2 * P : slot * V;
    const int c1 = IL ? c0 + 1 : c0 + a.rot / 2;
    struct Heads {
        E x[kHeads][N];
    };
    Heads v[2];
    float cs[P], sn[P];
    bool known = false;
    // heads of Q, then of K (numbered from H on)
    const int h0 = blockIdx.y * a.heads, h1 = min(a.H + a.Hkv, h0 + a.heads);
#pragma unroll 1
    for (int w = h0 >= a.H; w < 2; ++w) {
        const int lo = w ? max(h0 - a.H, 0) : h0, n = (w ? h1 - a.H : min(h1, a.H)) - lo;
        if (n <= 0 || (!turn && a.same[w])) continue;
        const long long is = a.is[w][1], os = a.os[w][1];
        const T* in = (const T*)a.in[w] + b * a.is[w][0] + t * a.is[w][2] + lo * is + c0;
        T* out = (T*)a.out[w] + b * a.os[w][0] + t * a.os[w][2] + lo * os + c0;
        auto fetch = [&](Heads& v, int h) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if (h + i >= n) continue;
                const T* p = in + (h + i) * is;
                v.x[i][0].load(p);
                if (!kOne && turn) v.x[i][N - 1].load(p + (c1 - c0));
            }
        };
        auto finish = [&](Heads& v, int h) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if (h + i >= n) continue;
                T* p = out + (h + i) * os;
                if (turn) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        T& e0 = kOne ? v.x[i][0].x[(2 * j) % V] : v.x[i][0].x[j % V];
                        T& e1 = kOne ? v.x[i][0].x[(2 * j + 1) % V] : v.x[i][N - 1].x[j % V];
                        const float x0 = to_f(e0), x1 = to_f(e1);
                        e0 = from_f<T>(x0 * cs[j] - x1 * sn[j]);
                        e1 = from_f<T>(x0 * sn[j] + x1 * cs[j]);
                    }
                    if (!kOne) v.x[i][N - 1].store(p + (c1 - c0));
                }
                v.x[i][0].store(p);
            }
        };
        fetch(v[0], 0);
        if (turn && !known) {
            const long long at = a.pos ? a.pos[b * a.pos_stride + t] : t;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const long long phase = (long long)((unsigned long long)at * a.turns[slot * P + i]);  // in 2^-64 turns
                sincospif((float)phase * 1.0842021724855044e-19f, &sn[i], &cs[i]);                    // 2^-63: half turns
                cs[i] *= a.gain;
                sn[i] *= a.back ? -a.gain : a.gain;
            }
            known = true;
        }
        // the next heads are on their way while these are turned
        for (int h = 0; h < n; h += 2 * kHeads) {
            fetch(v[1], h + kHeads);
            finish(v[0], h);
            fetch(v[0], h + 2 * kHeads);
            finish(v[1], h + kHeads);
        }
    }
}

// Whether every row can be accessed V elements at a time.
static bool rope_fits(const RopeArgs& a, bool il, int elem, int V) {
    const uintptr_t bytes = (uintptr_t)elem * V;
    if ((a.d - a.rot) % V || (il ? a.rot % V : a.rot / 2 % V)) return false;
    for (int w = 0; w < (a.Hkv ? 2 : 1); ++w) {
        if (((uintptr_t)a.in[w] | (uintptr_t)a.out[w]) % bytes) return false;
        for (int i = 0; i < 3; ++i)
            if ((a.is[w][i] | a.os[w][i]) % V) return false;
    }
    return true;
}

template <typename T, bool IL, int V> static cudaError_t rope_v(RopeArgs& a, cudaStream_t st) {
    const int P = IL && V > 1 ? V / 2 : V, slots = a.rot / 2 / P + (a.d - a.rot) / V, rows = kRopeThreads / slots;
    const long long blocks = ((long long)a.B * a.T + rows - 1) / rows;
    // A block goes over as many heads as leave eight blocks for each SM: all of them for a prompt, so
    // that cos and sin are computed once, and one for a few tokens, whose time is one head's.
    const long long all = (long long)(a.H + a.Hkv);
    a.heads = (int)std::min(all, std::max(1LL, all * blocks / (8LL * num_sms())));
    k_rope<T, IL, V><<<dim3((unsigned)blocks, (unsigned)((all + a.heads - 1) / a.heads)), kRopeThreads, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <typename T, bool IL> static cudaError_t rope_t(RopeArgs& a, cudaStream_t st) {
    constexpr int kWide = 32 / sizeof(T);
    // Units of 16 pairs leave a small call's threads with 16 angles each (64 tokens, 40 heads, d = 128: 4.2 us,
    // with 8 pairs 3.3; 200 tokens 5.5 and 4.0; 256 tokens 5.5 both; 65536 tokens 167 and 235).
    const bool few = !IL && sizeof(T) == 2 && (long long)a.B * a.T * (a.H + a.Hkv) * a.d < (1 << 20);
    if (!few && rope_fits(a, IL, sizeof(T), kWide)) return rope_v<T, IL, kWide>(a, st);
    if (rope_fits(a, IL, sizeof(T), kWide / 2)) return rope_v<T, IL, kWide / 2>(a, st);
    if (rope_fits(a, IL, sizeof(T), 2)) return rope_v<T, IL, 2>(a, st);
    return rope_v<T, IL, 1>(a, st);
}

cudaError_t launch_rope(RopeArgs& a, int dtype, bool interleaved, cudaStream_t st) {
    prof_mark(st, "rope");
    if (dtype == 0) return interleaved ? rope_t<float, true>(a, st) : rope_t<float, false>(a, st);
    return interleaved ? rope_t<__nv_bfloat16, true>(a, st) : rope_t<__nv_bfloat16, false>(a, st);
}

}  // namespace mita
