// qk_probs.hip -- log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "qk_launch.h"

namespace qk {
namespace probs {

constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int FEW = 32;    // rows that lie side by side (elem > 1) a tile has at most
constexpr int TILE = 256;  // tokens of such a tile
constexpr float LN2 = 0.693147180559945f;
constexpr float LOW = -1e4f;  // 2^LOW is 0: terms below say nothing, and never as inf * 0

// One token as a number whose order is that of the logits, the lower index
// first among equals (-0 and 0 are equal); 0: none.
__device__ __forceinline__ uint64_t key_of(float z, int v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);
    return (uint64_t)(b ^ (b >> 31 ? 0xffffffffu : 0x80000000u)) << 32 | (uint32_t)~v;
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t b = (uint32_t)(k >> 32);
    return __builtin_bit_cast(float, b ^ (b >> 31 ? 0x80000000u : 0xffffffffu));
}

// Statistics of a softmax under way, t = (z - m) * scale in units of log 2:
// the maximum, sum 2^t, sum t 2^t.
struct Stats { float m, s, w; };

__device__ __forceinline__ float step(float z, float m, float scale) {
    const float t = (z - (m == -INFINITY ? 0.f : m)) * scale;
    return t < LOW ? LOW : t;  // (NaN stays)
}
// The sums as they are with maximum m >= a.m.
__device__ __forceinline__ void raise(Stats &a, float m, float scale) {
    const float d = step(a.m, m, scale), f = __builtin_amdgcn_exp2f(d);
    a.w = f * fmaf(d, a.s, a.w);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void join(Stats &a, Stats b, float scale) {
    const float m = fmaxf(a.m, b.m);
    raise(a, m, scale);
    raise(b, m, scale);
    a.s += b.s;
    a.w += b.w;
}
template <int N> __device__ __forceinline__ void add(Stats &a, const float *z, float scale) {
    float m = a.m;
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, z[e]);
    raise(a, m, scale);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float t = step(z[e], m, scale), p = __builtin_amdgcn_exp2f(t);
        a.s += p;
        a.w = fmaf(p, t, a.w);
    }
}
__device__ __forceinline__ Stats over_wave(Stats a, float scale) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) join(a, Stats{__shfl_xor(a.m, d), __shfl_xor(a.s, d), __shfl_xor(a.w, d)}, scale);
    return a;
}

__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}

// The largest keys that a wave has seen, sorted: lane i has the i-th.  Keys
// come in batches of a lane each; thr, the last one of the `top` kept, rejects
// nearly all after the first few.
struct Best {
    uint64_t key, thr;
    __device__ __forceinline__ void clear() { key = 0; thr = 0; }
    __device__ __forceinline__ void insert(uint64_t c, int top, int lane) {  // c uniform, > thr
        const int at = __popcll(__ballot(key > c));
        const uint64_t up = (uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(key >> 32), 0x138, 0xf, 0xf, false) << 32 |
                            (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)key, 0x138, 0xf, 0xf, false);  // lane - 1
        key = lane < at ? key : lane == at ? c : up;
        thr = lane_key(key, top - 1);
    }
    __device__ __forceinline__ void offer(uint64_t c, int top, int lane) {
        uint64_t m;
        while ((m = __ballot(c > thr))) {
            const int l = __ffsll((unsigned long long)m) - 1;
            insert(lane_key(c, l), top, lane);
            if (lane == l) c = 0;
        }
    }
};

struct Args {
    Probs p;
    float scale;       // in units of log 2
    int splits, span;  // parts of a row, tokens of one
    float *stats;      // [rows][splits][3]
    uint64_t *keys;    // [rows][splits][top]
};

// A row's results, from its statistics (every lane) and its sorted keys.
__device__ __forceinline__ void finish(const Args &a, int row, const Stats &st, uint64_t key, int lane) {
    const Probs &p = a.p;
    const bool none = st.m == -INFINITY && st.s == 0.f;  // every token masked
    const float l2 = __builtin_amdgcn_logf(st.s), ln = l2 * LN2;  // (base 2)
    auto lp = [&](float z) { return z == -INFINITY ? (st.s == st.s ? -INFINITY : NAN) : fmaf(z - st.m, p.scale, -ln); };
    if (lane == 0) {
        if (p.lse) p.lse[row] = none ? -INFINITY : fmaf(st.m, p.scale, ln);
        if (p.entropy) p.entropy[row] = none ? 0.f : (l2 - st.w / st.s) * LN2;
    }
    for (int i = lane; i < p.ntok; i += 64) {
        const int v = p.tokens[(int64_t)row * p.ntok + i];
        float out = 0.f;  // no token
        if (v >= 0 && v < p.vocab) {
            const int64_t o = (int64_t)row * p.z.row + (int64_t)v * p.z.elem;
            out = lp(p.z.f16 ? (float)reinterpret_cast<const _Float16 *>(p.z.p)[o] : reinterpret_cast<const float *>(p.z.p)[o]);
        }
        p.token_lp[(int64_t)row * p.ntok + i] = out;
    }
    if (lane < p.top) {
        const int64_t o = (int64_t)row * p.top + lane;
        p.top_ids[o] = key ? key_token(key) : -1;
        p.top_lp[o] = key ? lp(key_value(key)) : -INFINITY;
    }
}

template <int N> __device__ __forceinline__ void take(const float *z, int v0, int stride, bool on, Stats &st, Best &best, float scale,
                                                      int top, int lane) {
    add<N>(st, z, scale);
    if (!top) return;
#pragma unroll
    for (int e = 0; e < N; ++e) best.offer(on && z[e] > -INFINITY ? key_of(z[e], v0 + e * stride) : 0, top, lane);
}

// The parts of a block's waves, joined by the first one.
__device__ __forceinline__ bool join_waves(Stats &st, Best &best, const Args &a, int lane, int wave) {
    __shared__ Stats part[WAVES];
    __shared__ uint64_t keys[WAVES][64];
    st = over_wave(st, a.scale);
    if (lane == 0) part[wave] = st;
    keys[wave][lane] = best.key;
    __syncthreads();
    if (wave) return false;
    for (int w = 1; w < WAVES; ++w) {
        join(st, part[w], a.scale);
        if (a.p.top) best.offer(lane < a.p.top ? keys[w][lane] : 0, a.p.top, lane);
    }
    return true;
}

// Rows whose tokens lie side by side: a block for a part of a row.
template <bool F16> __global__ void __launch_bounds__(THREADS) probs_row_kernel(Args a) {
    using T = std::conditional_t<F16, _Float16, float>;
    constexpr int N = 16 / sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(N)));
    const Probs &p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t u = blockIdx.x; u < (int64_t)p.rows * a.splits; u += gridDim.x) {
        const int row = (int)(u / a.splits), part = (int)(u % a.splits);
        const int v0 = part * a.span, v1 = min(v0 + a.span, p.vocab);
        const T *z = reinterpret_cast<const T *>(p.z.p) + (int64_t)row * p.z.row;
        Stats st{-INFINITY, 0, 0};
        Best best;
        best.clear();
        // up to the first whole piece of 16 bytes, then pieces, then the rest
        const int head = min(v1, v0 + (int)((16 - ((uintptr_t)(z + v0) & 15)) % 16 / sizeof(T)));
        const int pieces = max(0, (v1 - head) / N);
        if (wave == 0 && head > v0) {
            const bool on = v0 + lane < head;
            const float x = on ? (float)z[v0 + lane] : -INFINITY;
            take<1>(&x, v0 + lane, 0, on, st, best, a.scale, p.top, lane);
        }
        for (int i = wave * 64; i < pieces; i += THREADS) {
            const bool on = i + lane < pieces;
            const int v = head + (i + lane) * N;
            float x[N];
            Vec q;
            if (on) q = *reinterpret_cast<const Vec *>(z + v);
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = on ? (float)q[e] : -INFINITY;
            take<N>(x, v, 1, on, st, best, a.scale, p.top, lane);
        }
        const int tail = head + pieces * N;
        if (wave == WAVES - 1 && tail < v1) {
            const bool on = tail + lane < v1;
            const float x = on ? (float)z[tail + lane] : -INFINITY;
            take<1>(&x, tail + lane, 0, on, st, best, a.scale, p.top, lane);
        }
        if (join_waves(st, best, a, lane, wave)) {
            if (a.splits == 1) {
                finish(a, row, st, best.key, lane);
            } else {
                if (lane == 0) {
                    float *o = a.stats + u * 3;
                    o[0] = st.m; o[1] = st.s; o[2] = st.w;
                }
                if (lane < p.top) a.keys[u * p.top + lane] = best.key;
            }
        }
        __syncthreads();
    }
}

// Rows side by side (any strides): a block for a part of up to FEW rows, TILE
// tokens at a time through LDS, from where a wave has a row's.
__global__ void __launch_bounds__(THREADS) probs_few_kernel(Args a) {
    __shared__ float z[FEW][TILE + 1];
    const Probs &p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (p.rows + FEW - 1) / FEW;
    for (int64_t u = blockIdx.x; u < (int64_t)groups * a.splits; u += gridDim.x) {
        const int r0 = (int)(u / a.splits) * FEW, nr = min(FEW, p.rows - r0), part = (int)(u % a.splits);
        const int v0 = part * a.span, v1 = min(v0 + a.span, p.vocab);
        Stats st[FEW / WAVES];
        Best best[FEW / WAVES];
#pragma unroll
        for (int k = 0; k < FEW / WAVES; ++k) {
            st[k] = Stats{-INFINITY, 0, 0};
            best[k].clear();
        }
        const int per = THREADS / nr, r = threadIdx.x % nr, first = threadIdx.x / nr;
        for (int v = v0; v < v1; v += TILE) {
            const int n = min(TILE, v1 - v);
            if (first < per)
                for (int i = first; i < n; i += per) {
                    const int64_t o = (int64_t)(r0 + r) * p.z.row + (int64_t)(v + i) * p.z.elem;
                    z[r][i] = p.z.f16 ? (float)reinterpret_cast<const _Float16 *>(p.z.p)[o] : reinterpret_cast<const float *>(p.z.p)[o];
                }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < FEW / WAVES; ++k) {
                const int rr = k * WAVES + wave;
                if (rr >= nr) continue;
                for (int i = 0; i < n; i += 64) {
                    const bool on = i + lane < n;
                    const float x = on ? z[rr][i + lane] : -INFINITY;
                    take<1>(&x, v + i + lane, 0, on, st[k], best[k], a.scale, p.top, lane);
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < FEW / WAVES; ++k) {
            const int rr = k * WAVES + wave;
            if (rr >= nr) continue;
            const Stats s = over_wave(st[k], a.scale);
            const int64_t cell = (int64_t)(r0 + rr) * a.splits + part;
            if (a.splits == 1) {
                finish(a, r0 + rr, s, best[k].key, lane);
            } else {
                if (lane == 0) {
                    float *o = a.stats + cell * 3;
                    o[0] = s.m; o[1] = s.s; o[2] = s.w;
                }
                if (lane < p.top) a.keys[cell * p.top + lane] = best[k].key;
            }
        }
    }
}

// The parts of a row, joined in a fixed order: a block a row.
__global__ void __launch_bounds__(THREADS) probs_join_kernel(Args a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = blockIdx.x, top = a.p.top;
    Stats st{-INFINITY, 0, 0};
    Best best;
    best.clear();
    for (int i = threadIdx.x; i < a.splits; i += THREADS) {
        const float *s = a.stats + ((int64_t)row * a.splits + i) * 3;
        join(st, Stats{s[0], s[1], s[2]}, a.scale);
    }
    if (top)
        for (int i = wave; i < a.splits; i += WAVES)
            best.offer(lane < top ? a.keys[((int64_t)row * a.splits + i) * top + lane] : 0, top, lane);
    if (join_waves(st, best, a, lane, wave)) finish(a, row, st, best.key, lane);
}

// How a call is cut into parts.
struct Plan { bool few; int splits, span; };
Plan plan_of(const Probs &p) {
    Plan pl;
    pl.few = p.z.elem != 1;
    const int64_t units = pl.few ? (p.rows + FEW - 1) / FEW : p.rows;
    const int64_t want = std::max<int64_t>(1, 2 * device_cus() / units);
    const int unit = pl.few ? TILE : 1024;
    int64_t splits = std::min<int64_t>(want, (p.vocab + unit - 1) / unit);
    pl.span = (int)((p.vocab + splits - 1) / splits);
    pl.span = (pl.span + unit - 1) / unit * unit;
    pl.splits = (p.vocab + pl.span - 1) / pl.span;
    return pl;
}

}  // namespace probs

int64_t probs_workspace(const Probs &p) {
    const probs::Plan pl = probs::plan_of(p);
    if (pl.splits == 1) return 0;
    const int64_t cells = (int64_t)p.rows * pl.splits;
    return cells * p.top * 8 + (cells * 12 + 15) / 16 * 16;
}

hipError_t launch_probs(const Probs &p, void *workspace, hipStream_t st) {
    using namespace probs;
    const Plan pl = plan_of(p);
    uint64_t *keys = (uint64_t *)workspace;
    const Args a{p, p.scale * 1.44269504088896f, pl.splits, pl.span,
                 reinterpret_cast<float *>(keys + (int64_t)p.rows * pl.splits * p.top), keys};
    const int64_t units = pl.few ? (p.rows + FEW - 1) / FEW : p.rows;
    const unsigned blocks = (unsigned)std::min<int64_t>(units * pl.splits, 1 << 22);  // (a grid stays below 2^32 threads)
    if (pl.few) hipLaunchKernelGGL(probs_few_kernel, dim3(blocks), dim3(THREADS), 0, st, a);
    else if (p.z.f16) hipLaunchKernelGGL(probs_row_kernel<true>, dim3(blocks), dim3(THREADS), 0, st, a);
    else hipLaunchKernelGGL(probs_row_kernel<false>, dim3(blocks), dim3(THREADS), 0, st, a);
    if (pl.splits > 1) hipLaunchKernelGGL(probs_join_kernel, dim3((unsigned)p.rows), dim3(THREADS), 0, st, a);
    return hipGetLastError();
}

}  // namespace qk
