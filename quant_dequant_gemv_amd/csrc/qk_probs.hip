// qk_probs.hip -- log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits.
//
// One pass: with a running maximum m, s = sum 2^t and w = sum t 2^t of t =
// (z - m) scale log2 e; lse = m scale + ln s, entropy = ln 2 (log2 s - w / s).
// 1021 fp16 rows of 131071 (268 MB): 63-66 us, 4.1-4.2 TB/s, vector
// instructions (about 6 a logit, 70% of the issue slots) beside the loads; one
// row of 160000: 6.0 + 5.8 us, two launches whose waves sort once each.
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "qk_launch.h"

namespace qk {
namespace probs {

// waves of a block where a row's tokens lie side by side (2048 fp32 rows of 131071 190 us, 8 waves 212; one row 10.4, 10.8)
constexpr int ROW_WAVES = 4;
constexpr int WAVES = 8;           // where rows do: two blocks a CU (17 rows of 160000: 11.6 us, one of 16 waves 15.0)
constexpr int JOIN_WAVES = 8;      // where parts are joined (160 parts of 20: 5.8 us; 4 waves 6.8, 16 waves 6.0)
constexpr int LANE = 16;           // tokens a lane has at a time
constexpr int STEP = 64 * LANE;    // and a wave
constexpr int FEW = WAVES;         // rows that lie side by side (elem > 1) a block has at most, a wave a row or more
constexpr float LN2 = 0.693147180559945f, LN2_HI = 0x1.62e4p-1f, LN2_LO = 0x1.7f7d1cp-20f;  // (HI: 15 bits)
constexpr float SLACK = 4.f;  // in units of log 2
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

// A value's place in the order of values (-0 below 0), and back.
__device__ __forceinline__ int order_of(float z) {
    const int b = __builtin_bit_cast(int, z);
    return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float of_order(int o) { return __builtin_bit_cast(float, o ^ (o >> 31 & 0x7fffffff)); }

// Statistics of a softmax under way, t = (z - m) * scale in units of log 2:
// the maximum, sum 2^t, sum t 2^t.
struct Stats {
    float m;
    double s, w;
};

// LDS between the lanes of one wave: its accesses stay in program order, the
// compiler is told not to move them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// (a term below LOW is 0, and 0 * LOW is too; NaN stays in 2^t)
__device__ __forceinline__ float step(float z, float m, float scale) { return (z - (m == -INFINITY ? 0.f : m)) * scale; }
// The sums as they are with maximum m >= a.m.
__device__ __forceinline__ void raise(Stats &a, float m, float scale) {
    const float d = step(a.m, m, scale);
    const double f = __builtin_amdgcn_exp2f(d);
    a.w = f * fma((double)fmaxf(d, LOW), a.s, a.w);
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

// The same of one lane's terms.  Many equal terms round the same way each time,
// and a lane has up to vocab / 64 of them, so its sums are s - ds and w - dw, what
// an addition loses being taken from the next one (plain fp32 sums of 2^20 such
// logits were off by 6e-5; in fp64 600 fp32 rows of 131072 took 78 us for 67).
// m is up to SLACK below the largest logit: each change of it costs a rounded
// power of 2, and maxima that rise all along a row would cost one a batch.
struct Lane {
    float m, most, s, ds, w, dw;
    __device__ __forceinline__ void clear() {
        m = -FLT_MAX;  // (finite: what a row of -inf is compared with)
        most = -INFINITY;
        s = ds = w = dw = 0.f;
    }
    // N terms more, the largest of them `top`, summed by themselves first.
    template <int N> __device__ __forceinline__ void add(const float *z, float top, float scale) {
        most = fmaxf(most, top);
        const float rise = (most - m) * scale;  // (NaN: of two infinities)
        const bool up = rise > SLACK;           // (no branch: 1021 fp16 rows of 131071 70 us with one, 66 without)
        const float d = up ? fmaxf(-rise, LOW) : 0.f, f = __builtin_amdgcn_exp2f(d);
        m = up ? most : m;
        constexpr int C = N < 2 ? N : 2;
        float p[C], q[C];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float t = (z[e] - m) * scale, x = __builtin_amdgcn_exp2f(t), y = fmaxf(t, LOW);
            p[e % C] = e < C ? x : p[e % C] + x;
            q[e % C] = e < C ? x * y : fmaf(x, y, q[e % C]);
        }
        w = fmaf(d, s, w);
        plus(s, ds, f, C == 2 ? p[0] + p[1] : p[0]);
        plus(w, dw, f, C == 2 ? q[0] + q[1] : q[0]);
    }
    // sum <- f sum + x
    static __device__ __forceinline__ void plus(float &sum, float &over, float f, float x) {
        const float y = fmaf(-f, over, x), t = fmaf(f, sum, y);
        over = fmaf(-f, sum, t) - y;
        sum = t;
    }
};

// Over the 64 lanes, by DPP inside rows of 16 (no LDS): every lane gets it.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
template <typename F> __device__ __forceinline__ float over_lanes(float v, F f) {
    v = f(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
    v = f(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
    v = f(v, dpp<0x141>(v));  // half row mirrored
    v = f(v, dpp<0x140>(v));  // row mirrored
    return f(f(lane_of(v, 0), lane_of(v, 16)), f(lane_of(v, 32), lane_of(v, 48)));
}
__device__ __forceinline__ int over_lanes_max(int v) {
    auto f = [](int a, int b) { return max(a, b); };
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, true));
    return f(f(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             f(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
__device__ __forceinline__ float wave_max(float v) {
    return over_lanes(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int CTRL> __device__ __forceinline__ double dpp(double v) {
    const uint2 w = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, make_uint2(__builtin_amdgcn_update_dpp(0, (int)w.x, CTRL, 0xf, 0xf, true),
                                                 __builtin_amdgcn_update_dpp(0, (int)w.y, CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint2 w = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, make_uint2(__builtin_amdgcn_readlane((int)w.x, lane), __builtin_amdgcn_readlane((int)w.y, lane)));
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
__device__ __forceinline__ Stats over_wave(Stats a, float scale) {
    raise(a, wave_max(a.m), scale);
    return Stats{a.m, wave_sum(a.s), wave_sum(a.w)};
}
__device__ __forceinline__ Stats over_wave(const Lane &l, float scale) {
    Stats a{l.m, (double)l.s - l.ds, (double)l.w - l.dw};
    raise(a, wave_max(l.most), scale);
    return Stats{a.m, wave_sum(a.s), wave_sum(a.w)};
}

__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}

// The largest keys that a wave has seen, sorted: lane i has the i-th.  What
// does not pass the last one of the `top` kept is rejected 64 at a time, so
// after the first batch few are looked at one by one.
struct Best {
    uint64_t key, thr;
    float low;  // value of thr before the batch under way: a token of it has to be above
    __device__ __forceinline__ void clear() { key = thr = 0; low = -INFINITY; }
    __device__ __forceinline__ void limit(int top) {
        thr = lane_key(key, top - 1);
        low = thr ? key_value(thr) : -INFINITY;
    }
    __device__ __forceinline__ void offer(uint64_t c, int top, int lane) {
        uint64_t m;
        while ((m = __ballot(c > thr))) {
            const int l = __ffsll((unsigned long long)m) - 1;
            const uint64_t k = lane_key(c, l);
            const int at = __popcll(__ballot(key > k));
            const uint64_t up = (uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(key >> 32), 0x138, 0xf, 0xf, false) << 32 |
                                (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)key, 0x138, 0xf, 0xf, false);  // lane - 1
            key = lane < at ? key : lane == at ? k : up;
            thr = lane_key(key, top - 1);
            if (lane == l) c = 0;
        }
    }
    // The first batch: N tokens a lane, value(e) and token(e) of the e-th one
    // (-inf: none), `most` the lane's largest value.  At least `top` tokens are
    // at or above a value that `top` lanes reach with their largest, and few
    // more: those go to LDS and are sorted by counting.  That value is found by
    // halving, and where it leaves up to EASY lanes (about 30 tokens) it will
    // do (comparing every lane's with every other's: 3 times the instructions).
    template <int N, typename V, typename T>
    __device__ __forceinline__ void first(V value, T token, float most, int top, int lane, uint64_t *lds) {
        constexpr int EASY = 24;
        const int o = order_of(most > -INFINITY ? most : -INFINITY), all = over_lanes_max(o);
        int lo = ~over_lanes_max(~o), hi = all + 1;  // `top` lanes reach lo, fewer hi
        int count = 64;
        while (count > max(top, EASY) && (uint32_t)hi - (uint32_t)lo > 1) {
            const int mid = (int)((uint32_t)lo + ((uint32_t)hi - (uint32_t)lo) / 2), c = __popcll(__ballot(o >= mid));
            if (c >= top) { lo = mid; count = c; }
            else hi = mid;
        }
        const float floor = fmaxf(of_order(lo), -FLT_MAX);
        int n = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float z = value(e);
            const uint64_t m = __ballot(z >= floor);
            const int at = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, n));
            if (z >= floor) lds[at & 63] = (uint64_t)(uint32_t)token(e) << 32 | __builtin_bit_cast(uint32_t, z);
            n += __popcll(m);
        }
        wave_sync();
        if (n <= 64) {
            const uint64_t c = lds[lane], mine = lane < n ? key_of(__builtin_bit_cast(float, (uint32_t)c), (int)(c >> 32)) : 0;
            wave_sync();
            lds[lane] = mine;
            wave_sync();
            int rank = 0;
            for (int j = 0; j < n; j += 4) {  // (lanes from n on hold 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) rank += lds[j + i] > mine;
            }
            wave_sync();
            if (lane < n) lds[rank] = mine;
            wave_sync();
            key = lane < n ? lds[lane] : 0;
        } else {  // (many equals, or many asked for)
            clear();
#pragma unroll
            for (int e = 0; e < N; ++e) offer(value(e) >= floor ? key_of(value(e), token(e)) : 0, top, lane);
        }
        limit(top);
        wave_sync();
    }
};

struct Args {
    Probs p;
    float scale;       // in units of log 2
    int splits, span, subs;  // parts of a row, tokens of a block, parts of a row that a block leaves
    float *stats;      // [rows][splits][3]
    uint64_t *keys;    // [rows][splits][top]
};

// A row's i-th asked token and its logit, two loads after one another: begun
// before the row's statistics are there.
struct Asked { int v; float z; };
__device__ __forceinline__ Asked asked(const Probs &p, int row, int i) {
    Asked q{-1, 0.f};
    if (i >= p.ntok) return q;
    q.v = p.tokens[(int64_t)row * p.ntok + i];
    if (q.v < 0 || q.v >= p.vocab) return Asked{-1, 0.f};
    const int64_t o = (int64_t)row * p.z.row + (int64_t)q.v * p.z.elem;
    q.z = p.z.f16 ? (float)reinterpret_cast<const _Float16 *>(p.z.p)[o] : reinterpret_cast<const float *>(p.z.p)[o];
    return q;
}

// log s: the exponent's part exactly (a sum of one term is 0), the rest within 2^-23.
__device__ __forceinline__ float log_of(double s) {
    float f = (float)__builtin_amdgcn_frexp_mant(s);
    int e = __builtin_amdgcn_frexp_exp(s);
    if (f < 0.70710678f) {
        f *= 2.f;
        --e;
    }
    return fmaf((float)e, LN2_HI, fmaf((float)e, LN2_LO, __builtin_amdgcn_logf(f) * LN2));  // (base 2)
}

// A row's results, from its statistics (every lane), its sorted keys and the
// first 64 asked tokens, one a lane.
__device__ __forceinline__ void finish(const Args &a, int row, const Stats &st, uint64_t key, Asked q, int lane) {
    const Probs &p = a.p;
    const bool none = st.m == -INFINITY && st.s == 0;  // every token masked
    const float ln = log_of(st.s < 1 ? 1 : st.s);  // (the largest logit's own term is 1: no log probability is above 0)
    auto lp = [&](float z) { return z == -INFINITY ? (st.s == st.s ? -INFINITY : NAN) : fmaf(z - st.m, p.scale, -ln); };
    if (lane == 0) {
        if (p.lse) p.lse[row] = none ? -INFINITY : fmaf(st.m, p.scale, ln);
        const float h = fmaf(-(float)st.w / (float)st.s, LN2, ln);
        if (p.entropy) p.entropy[row] = none || h < 0.f ? 0.f : h;
    }
    for (int i = lane; i < p.ntok; i += 64) {
        if (i != lane) q = asked(p, row, i);
        p.token_lp[(int64_t)row * p.ntok + i] = q.v < 0 ? 0.f : lp(q.z);
    }
    if (lane < p.top) {
        const int64_t o = (int64_t)row * p.top + lane;
        p.top_ids[o] = key ? key_token(key) : -1;
        p.top_lp[o] = key ? lp(key_value(key)) : -INFINITY;
    }
}

// N tokens a lane more (-inf: none), at(e) the e-th one's number.  Those of a
// wave come in rising batches, so an equal of the last one kept is no better in
// a later batch and `low` rejects it by value; inside a batch tokens rise with
// neither e nor the lane, and their keys decide.  fresh: the first batch.
template <int N, typename F>
__device__ __forceinline__ void take(const float *z, F at, bool fresh, Lane &st, Best &best, float scale, int top, int lane, uint64_t *lds) {
    float most = z[0];
#pragma unroll
    for (int e = 1; e < N; ++e) most = fmaxf(most, z[e]);
    st.add<N>(z, most, scale);
    if (!top) return;
    if (fresh) {
        best.first<N>([&](int e) { return z[e]; }, at, most, top, lane, lds);
    } else if (__ballot(most > best.low)) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (__ballot(z[e] > best.low)) best.offer(z[e] > best.low ? key_of(z[e], at(e)) : 0, top, lane);
        best.limit(top);
    }
}

// The largest of `count` keys from p on, for one wave.
template <typename P> __device__ __forceinline__ void gather(P p, int count, Best &best, int top, int lane, uint64_t *lds) {
    constexpr int N = 8;
    for (int i = 0; i < count; i += 64 * N) {
        uint64_t k[N];
#pragma unroll
        for (int e = 0; e < N; ++e) k[e] = i + 64 * e + lane < count ? p[i + 64 * e + lane] : 0;
        if (i == 0) {
            auto value = [&](int e) { return k[e] ? key_value(k[e]) : -INFINITY; };
            float most = value(0);
#pragma unroll
            for (int e = 1; e < N; ++e) most = fmaxf(most, value(e));
            best.first<N>(value, [&](int e) { return key_token(k[e]); }, most, top, lane, lds);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) best.offer(k[e], top, lane);
        }
    }
}

// What the waves of a block share.
template <int W> struct Shared {
    Stats part[W];
    uint64_t keys[W * 64], sort[W][64];
};

// The parts of a block's waves, joined by the first one (true).
template <int W>
__device__ __forceinline__ bool join_waves(Stats &st, Best &best, const Args &a, Shared<W> &sh, int lane, int wave) {
    const int top = a.p.top;
    if (lane == 0) sh.part[wave] = st;
    if (lane < top) sh.keys[wave * top + lane] = best.key;
    __syncthreads();
    if (wave) return false;
    st = over_wave(lane < W ? sh.part[lane] : Stats{-INFINITY, 0, 0}, a.scale);
    if (top) gather(sh.keys, W * top, best, top, lane, sh.sort[0]);
    return true;
}

__device__ __forceinline__ void leave(const Args &a, int row, int part, const Stats &st, uint64_t key, int lane) {
    const int64_t cell = (int64_t)row * a.splits + part;
    if (lane == 0) {
        float *o = a.stats + cell * 3;
        o[0] = st.m; o[1] = (float)st.s; o[2] = (float)st.w;
    }
    if (lane < a.p.top) a.keys[cell * a.p.top + lane] = key;
}

// Rows whose tokens lie side by side: a block for a part of a row, STEP tokens
// of it to a wave at a time.  A row of one block is joined in it; of more, each
// wave leaves a part of its own, since the join to come sorts once more anyway
// (one row of 160000, top 20: the kernel 8.5 us with a join of the block's waves).
template <bool F16> __global__ void __launch_bounds__(64 * ROW_WAVES) probs_row_kernel(Args a) {
    using T = std::conditional_t<F16, _Float16, float>;
    constexpr int THREADS = 64 * ROW_WAVES, N = 16 / sizeof(T), J = LANE / N;  // tokens of a piece, pieces of a lane
    typedef T Vec __attribute__((ext_vector_type(N)));
    __shared__ Shared<ROW_WAVES> sh;
    const Probs &p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks_row = a.splits == 1 ? 1 : a.splits / ROW_WAVES;
    for (int64_t u = blockIdx.x; u < (int64_t)p.rows * blocks_row; u += gridDim.x) {
        const int row = (int)(u / blocks_row), part = (int)(u % blocks_row);
        const int v0 = part * a.span, v1 = min(v0 + a.span, p.vocab);
        const T *z = reinterpret_cast<const T *>(p.z.p) + (int64_t)row * p.z.row;
        Asked q{-1, 0.f};
        if (a.splits == 1 && wave == 0) q = asked(p, row, lane);
        Lane sums;
        sums.clear();
        Best best;
        best.clear();
        // whole pieces of 16 bytes, and what is left before and behind them (wave 0 and the last one, at the end)
        const int head = min(v1, v0 + (int)((16 - ((uintptr_t)(z + v0) & 15)) % 16 / sizeof(T)));
        const int pieces = max(0, (v1 - head) / N), tail = head + pieces * N;
        bool fresh = true;
        // (scalars beside the lane: 124 registers for 133, 4 waves a SIMD; 2048 fp32 rows of 131071 190 us for 196)
        auto load = [&](int i, Vec *q) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (lane < pieces - i - 64 * j) q[j] = *reinterpret_cast<const Vec *>(z + head + (i + 64 * j + lane) * N);
        };
        Vec cur[J], nx[J];
        load(wave * 64 * J, cur);
        for (int i = wave * 64 * J; i < pieces; i += THREADS * J) {
            load(i + THREADS * J, nx);
            float x[LANE];
#pragma unroll
            for (int e = 0; e < LANE; ++e) x[e] = (float)cur[e / N][e % N];
            if (i + 64 * J > pieces) {
#pragma unroll
                for (int e = 0; e < LANE; ++e) x[e] = lane < pieces - i - 64 * (e / N) ? x[e] : -INFINITY;
            }
            take<LANE>(x, [&](int e) { return head + (i + 64 * (e / N) + lane) * N + e % N; }, fresh, sums, best, a.scale, p.top, lane,
                       sh.sort[wave]);
            fresh = false;
#pragma unroll
            for (int j = 0; j < J; ++j) cur[j] = nx[j];
        }
        auto rest = [&](int from, int to) {
            if (from >= to) return;
            const float x = from + lane < to ? (float)z[from + lane] : -INFINITY;
            sums.add<1>(&x, x, a.scale);
            if (p.top) best.offer(x > -INFINITY ? key_of(x, from + lane) : 0, p.top, lane);
        };
        if (wave == 0) rest(v0, head);
        if (wave == ROW_WAVES - 1) rest(tail, v1);
        Stats st = over_wave(sums, a.scale);
        if (a.splits > 1) {
            leave(a, row, part * ROW_WAVES + wave, st, best.key, lane);
            continue;
        }
        if (join_waves(st, best, a, sh, lane, wave)) finish(a, row, st, best.key, q, lane);
        __syncthreads();
    }
}

// Rows side by side (any strides): a block for a part of up to FEW rows, a tile
// of tokens at a time through LDS.  Where there are fewer rows than waves, a
// row's tile is shared by `subs` of them, and each leaves a part of its own.
__global__ void __launch_bounds__(64 * WAVES) probs_few_kernel(Args a) {
    constexpr int THREADS = 64 * WAVES, AHEAD = 8;
    extern __shared__ float z[];  // [rows][tile + 1]
    __shared__ uint64_t sort[WAVES][64];
    const Probs &p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (p.rows + FEW - 1) / FEW, per = (p.rows + groups - 1) / groups;
    const int blocks_row = a.splits / a.subs, tile = STEP * a.subs, pitch = tile + 1;
    for (int64_t u = blockIdx.x; u < (int64_t)groups * blocks_row; u += gridDim.x) {
        const int r0 = (int)(u / blocks_row) * per, nr = min(per, p.rows - r0), part = (int)(u % blocks_row);
        const int v0 = part * a.span, v1 = min(v0 + a.span, p.vocab);
        const bool mine = wave < nr * a.subs;
        const int row = wave % nr, t0 = wave / nr * STEP;
        Lane sums;
        sums.clear();
        Best best;
        best.clear();
        for (int v = v0; v < v1; v += tile) {
            const int n = min(tile, v1 - v), total = n * nr;
            // element e of the tile: token e / nr, row e % nr
            const int i = threadIdx.x / nr, di = THREADS / nr, dr = THREADS % nr;
            int r = threadIdx.x % nr, to = r * pitch + i;
            int64_t from = (int64_t)(r0 + r) * p.z.row + (int64_t)(v + i) * p.z.elem;
            const int64_t on = (int64_t)di * p.z.elem + (int64_t)dr * p.z.row, wrap = p.z.elem - nr * p.z.row;
            auto each = [&](auto get) {
                for (int e = threadIdx.x; e < total; e += THREADS * AHEAD) {
                    float x[AHEAD];
                    int at[AHEAD];
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        if (e + THREADS * k < total) x[k] = get(from);
                        at[k] = to;
                        const bool next = (r += dr) >= nr;
                        r -= next ? nr : 0;
                        from += on + (next ? wrap : 0);
                        to += dr * pitch + di + (next ? 1 - nr * pitch : 0);
                    }
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k)
                        if (e + THREADS * k < total) z[at[k]] = x[k];
                }
            };
            if (p.z.f16) each([&](int64_t o) { return (float)reinterpret_cast<const _Float16 *>(p.z.p)[o]; });
            else each([&](int64_t o) { return reinterpret_cast<const float *>(p.z.p)[o]; });
            __syncthreads();
            if (mine) {
                const float *tokens = z + row * pitch + t0;
                const int left = n - t0;  // (scalars beside the lane: 12 registers less, two blocks a CU)
                float x[LANE];
#pragma unroll
                for (int e = 0; e < LANE; ++e) x[e] = lane < left - 64 * e ? tokens[64 * e + lane] : -INFINITY;
                take<LANE>(x, [&](int e) { return v + t0 + 64 * e + lane; }, v == v0, sums, best, a.scale, p.top, lane, sort[wave]);
            }
            __syncthreads();
        }
        if (!mine) continue;
        const Stats st = over_wave(sums, a.scale);
        if (a.splits == 1) finish(a, r0 + row, st, best.key, asked(p, r0 + row, lane), lane);
        else leave(a, r0 + row, part * a.subs + wave / nr, st, best.key, lane);
    }
}

// The parts of a row, joined in a fixed order: a block a row.
__global__ void __launch_bounds__(64 * JOIN_WAVES) probs_join_kernel(Args a) {
    __shared__ Shared<JOIN_WAVES> sh;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = blockIdx.x, top = a.p.top;
    Stats st{-INFINITY, 0, 0};
    Best best;
    best.clear();
    const int per = (a.splits + JOIN_WAVES - 1) / JOIN_WAVES, first = min(wave * per, a.splits), count = min(per, a.splits - first);
    Asked q{-1, 0.f};
    if (wave == 0) q = asked(a.p, row, lane);
    for (int i = threadIdx.x; i < a.splits; i += 64 * JOIN_WAVES) {
        const float *s = a.stats + ((int64_t)row * a.splits + i) * 3;
        join(st, Stats{s[0], s[1], s[2]}, a.scale);
    }
    if (top) gather(a.keys + ((int64_t)row * a.splits + first) * top, count * top, best, top, lane, sh.sort[wave]);
    st = over_wave(st, a.scale);
    if (join_waves(st, best, a, sh, lane, wave)) finish(a, row, st, best.key, q, lane);
}

// How a call is cut: `splits` parts a row, `span` tokens to a block.  Two blocks
// a CU where the rows alone are fewer; else a row is one block's, and no join
// follows.
struct Plan { bool few; int splits, span, subs; };
Plan plan_of(const Probs &p) {
    Plan pl{p.z.elem != 1, 1, 0, 1};
    if (pl.few) pl.subs = std::max(1, std::min(WAVES / std::min(p.rows, FEW), (p.vocab + STEP - 1) / STEP));
    const int64_t units = pl.few ? (p.rows + FEW - 1) / FEW : p.rows;
    const int64_t grain = pl.few ? STEP * pl.subs : STEP * ROW_WAVES;
    const int64_t want = std::max<int64_t>(1, 2 * device_cus() / units), grains = (p.vocab + grain - 1) / grain;
    const int64_t span = (grains + std::min(want, grains) - 1) / std::min(want, grains) * grain;
    pl.span = (int)std::min<int64_t>(span, INT32_MAX);
    pl.splits = (int)((p.vocab + span - 1) / span);
    if (!pl.few && pl.splits > 1) pl.subs = ROW_WAVES;
    pl.splits *= pl.subs;
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
    const Args a{p, p.scale * 1.44269504088896f, pl.splits, pl.span, pl.subs,
                 reinterpret_cast<float *>(keys + (int64_t)p.rows * pl.splits * p.top), keys};
    const int64_t units = pl.few ? (p.rows + FEW - 1) / FEW : p.rows;
    const unsigned blocks = (unsigned)std::min<int64_t>(units * pl.splits / pl.subs, 1 << 22);  // (a grid stays below 2^32 threads)
    if (pl.few) {
        const hipError_t e = lds_opt_in<probs_few_kernel>(FEW * (STEP + 1) * 4);
        if (e != hipSuccess) return e;
        const int lds = std::min(p.rows, FEW) * (STEP * pl.subs + 1) * 4;
        hipLaunchKernelGGL(probs_few_kernel, dim3(blocks), dim3(64 * WAVES), lds, st, a);
    } else if (p.z.f16) {
        hipLaunchKernelGGL(probs_row_kernel<true>, dim3(blocks), dim3(64 * ROW_WAVES), 0, st, a);
    } else {
        hipLaunchKernelGGL(probs_row_kernel<false>, dim3(blocks), dim3(64 * ROW_WAVES), 0, st, a);
    }
    if (pl.splits > 1) hipLaunchKernelGGL(probs_join_kernel, dim3((unsigned)p.rows), dim3(64 * JOIN_WAVES), 0, st, a);
    return hipGetLastError();
}

}  // namespace qk
