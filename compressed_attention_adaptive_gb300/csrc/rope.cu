// Rotary positions: y0 = gain (x0 cos a - x1 sin a), y1 = gain (x0 sin a + x1 cos a) for the pairs of a
// row's first `rot` channels, a = position * frequency; the other channels are copied.
//
// Each row is read and written once, 6 operations per pair, so long calls are bound by HBM
// and calls of a few tokens by the launch. The angle depends on token and pair alone: a thread
// has one place of a row and goes over the heads of Q and K with its cos and sin in registers, so
// that these cost it once per token what a head's row costs.
//
// Angles. A frequency is held in turns per position as a 64-bit fraction (host: double, 2^-53
// of it); position * fraction in integers wraps at whole turns, which is the reduction, exactly. The
// signed fraction goes to sincospi as a float: 2^-24 of the angle in (-pi, pi].
#include <math.h>

#include "rope.cuh"

namespace mita {

constexpr int kRopeThreads = 256;

// V elements of a row, one access.
template <typename T, int V> struct alignas(sizeof(T) * V) Elems {
    T x[V];
};

// T: element; IL: interleaved pairs; V: elements of an access. A unit of a rotated place is V pairs (two accesses),
// or one access of V / 2 interleaved pairs.
template <typename T, bool IL, int V>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeArgs a) {
    constexpr bool kOne = IL && V > 1;       // one access holds whole pairs
    constexpr int P = kOne ? V / 2 : V;      // pairs of a unit
    constexpr int kHeads = V * sizeof(T) == 16 ? 4 : 2;  // heads whose loads are in flight together
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
    float cs[P], sn[P];
    if (turn) {
        const long long at = a.pos ? a.pos[b * a.pos_stride + t] : t;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const long long phase = (long long)((unsigned long long)at * a.turns[slot * P + i]);  // in 2^-64 turns
            sincospif((float)phase * 1.0842021724855044e-19f, &sn[i], &cs[i]);                    // 2^-63: half turns
            cs[i] *= a.gain;
            sn[i] *= a.back ? -a.gain : a.gain;
        }
    }
    const int h1 = min(a.H + a.Hkv, ((int)blockIdx.y + 1) * a.heads);
    for (int h0 = blockIdx.y * a.heads; h0 < h1; h0 += kHeads) {
        E x[kHeads], y[kOne ? 1 : kHeads];
        T* out[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int w = h0 + i >= a.H, h = w ? h0 + i - a.H : h0 + i;
            out[i] = nullptr;
            if (h0 + i >= h1 || (!turn && a.same[w])) continue;
            const T* in = (const T*)a.in[w] + b * a.is[w][0] + h * a.is[w][1] + t * a.is[w][2];
            out[i] = (T*)a.out[w] + b * a.os[w][0] + h * a.os[w][1] + t * a.os[w][2];
            x[i] = *reinterpret_cast<const E*>(in + c0);
            if (!kOne && turn) y[i % (kOne ? 1 : kHeads)] = *reinterpret_cast<const E*>(in + c1);
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (!out[i]) continue;
            if (turn) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    T& e0 = kOne ? x[i].x[(2 * j) % V] : x[i].x[j % V];
                    T& e1 = kOne ? x[i].x[(2 * j + 1) % V] : y[i % (kOne ? 1 : kHeads)].x[j % V];
                    const float x0 = to_f(e0), x1 = to_f(e1);
                    e0 = from_f<T>(x0 * cs[j] - x1 * sn[j]);
                    e1 = from_f<T>(x0 * sn[j] + x1 * cs[j]);
                }
                if (!kOne) *reinterpret_cast<E*>(out[i] + c1) = y[i % (kOne ? 1 : kHeads)];
            }
            *reinterpret_cast<E*>(out[i] + c0) = x[i];
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
    constexpr int kWide = 16 / sizeof(T);
    if (rope_fits(a, IL, sizeof(T), kWide)) return rope_v<T, IL, kWide>(a, st);
    if (rope_fits(a, IL, sizeof(T), 2)) return rope_v<T, IL, 2>(a, st);
    return rope_v<T, IL, 1>(a, st);
}

cudaError_t launch_rope(RopeArgs& a, int dtype, bool interleaved, cudaStream_t st) {
    prof_mark(st, "rope");
    if (dtype == 0) return interleaved ? rope_t<float, true>(a, st) : rope_t<float, false>(a, st);
    return interleaved ? rope_t<__nv_bfloat16, true>(a, st) : rope_t<__nv_bfloat16, false>(a, st);
}

}  // namespace mita
