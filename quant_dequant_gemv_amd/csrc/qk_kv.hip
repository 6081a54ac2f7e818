// qk_kv.hip -- rows of heads: norm + rotation, appending to the paged 4-bit
// cache, and reading it back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "qk_kv.h"

namespace qk {
namespace rows {

constexpr int WAVES = 4;

// LDS between the lanes of one wave: its accesses stay in program order, the
// compiler is told not to move them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float load_head(const Heads &x, int64_t i) {
    return x.f16 ? (float)reinterpret_cast<const _Float16 *>(x.p)[i] : reinterpret_cast<const float *>(x.p)[i];
}

// A lane has 4 consecutive dimensions of a head, so a wave has HPW = 256 / D
// heads of one kind side by side, and a group of 32 dimensions is 8 lanes.
constexpr int lanes_of(int D) { return D / 4; }

// v of the lane `CTRL` away inside a row of 16 lanes (a DPP pattern: no LDS)
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ double dpp(double v) {
    const uint2 w = __builtin_bit_cast(uint2, v);
    const uint2 r = make_uint2(__builtin_amdgcn_update_dpp(0, (int)w.x, CTRL, 0xf, 0xf, true),
                               __builtin_amdgcn_update_dpp(0, (int)w.y, CTRL, 0xf, 0xf, true));
    return __builtin_bit_cast(double, r);
}
constexpr int SWAP1 = 0xB1, SWAP2 = 0x4E, MIRROR8 = 0x141, MIRROR16 = 0x140;  // quad_perm [1,0,3,2], [2,3,0,1]; half row, row

// Sum over the lanes of a head: every lane gets it.
template <int LPH> __device__ __forceinline__ double head_sum(double v) {
    v += dpp<SWAP1>(v);
    v += dpp<SWAP2>(v);
    v += dpp<MIRROR8>(v);
    v += dpp<MIRROR16>(v);
    if (LPH > 16) v += __shfl_xor(v, 16);
    if (LPH > 32) v += __shfl_xor(v, 32);
    return v;
}

typedef _Float16 h4 __attribute__((ext_vector_type(4)));

// x[0..3] = 4 elements from p on (bytes), side by side (VEC) or `elem` apart.
template <bool VEC> __device__ __forceinline__ void load4(const uint8_t *p, int64_t elem, bool f16, float x[4]) {
    if (f16) {
        if constexpr (VEC) {
            const h4 v = *reinterpret_cast<const h4 *>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (float)v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (float)reinterpret_cast<const _Float16 *>(p)[e * elem];
        }
    } else {
        if constexpr (VEC) {
            const float4 v = *reinterpret_cast<const float4 *>(p);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = reinterpret_cast<const float *>(p)[e * elem];
        }
    }
}
template <bool VEC> __device__ __forceinline__ void store4(uint8_t *p, int64_t elem, bool f16, const float x[4]) {
    if (f16) {
        if constexpr (VEC) {
            *reinterpret_cast<h4 *>(p) = h4{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) reinterpret_cast<_Float16 *>(p)[e * elem] = (_Float16)x[e];
        }
    } else {
        if constexpr (VEC) {
            *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) reinterpret_cast<float *>(p)[e * elem] = x[e];
        }
    }
}
// Element (t, h, i) of a view.
__device__ __forceinline__ uint8_t *at(const Heads &x, int64_t t, int64_t h, int64_t i) {
    return reinterpret_cast<uint8_t *>(x.p) + ((t * x.row + h * x.head + i * x.elem) << (x.f16 ? 1 : 2));
}

// Sine and cosine in fp64: the angle less the nearest multiple of pi/2 (one
// exact fma and one with the rest of pi/2: off by 2^-53), then the Taylor
// series on [-pi/4, pi/4], whose first term left out is below 2^-58.
__device__ __forceinline__ void sin_cos(double a, double &sn, double &cs) {
    if (!(fabs(a) < 2147483648.0)) {  // beyond every position at a frequency up to 1
        sincos(a, &sn, &cs);
        return;
    }
    const double k = rint(a * 0x1.45f306dc9c883p-1);
    double r = fma(-k, 0x1.921fb54442d18p+0, a);
    r = fma(-k, 0x1.1a62633145c07p-54, r);
    const double z = r * r;
    double s = 1.0 / 355687428096000.0, c = 1.0 / 20922789888000.0;  // 1/17!, 1/16!
    s = fma(s, z, -1.0 / 1307674368000.0); c = fma(c, z, -1.0 / 87178291200.0);
    s = fma(s, z, 1.0 / 6227020800.0);     c = fma(c, z, 1.0 / 479001600.0);
    s = fma(s, z, -1.0 / 39916800.0);      c = fma(c, z, -1.0 / 3628800.0);
    s = fma(s, z, 1.0 / 362880.0);         c = fma(c, z, 1.0 / 40320.0);
    s = fma(s, z, -1.0 / 5040.0);          c = fma(c, z, -1.0 / 720.0);
    s = fma(s, z, 1.0 / 120.0);            c = fma(c, z, 1.0 / 24.0);
    s = fma(s, z, -1.0 / 6.0);             c = fma(c, z, -0.5);
    s = fma(s * z, r, r);                  c = fma(c, z, 1.0);
    const int quarter = (int)(int64_t)k & 3;
    sn = quarter & 1 ? c : s;
    cs = quarter & 1 ? s : c;
    if (quarter & 2) sn = -sn;
    if ((quarter + 1) & 2) cs = -cs;
}

struct RowsArgs {
    KvCache c;
    KvSeqs sq;
    RowPrep rp;
    int hq, hkv, cached;
    Heads q, qo, k, v, ko;
    int per, chunks;           // groups of HPW heads a wave takes, waves of a row
};

// Norm, rotation and grouping in registers, in fp64 up to the fp32 value that is
// grouped or stored; an fp16 output is rounded from that value, so it is off by
// half a step and 2^-24 at most.  (The fp64 value cut to 21 bits with a sticky
// last one would be rounded once: two instructions an element, 17.95 against
// 17.1 us at 2048 rows, D = 128, for one value in 2^14 one step nearer by less
// than 2^-24.)  The pair of a rotated dimension
// is in the same lane (interleaved) or, the normed value depending on its own
// element alone, loaded a second time from where it lies (an L1 hit): nothing
// but the row's sines and cosines passes LDS, once for all heads of the wave.
// The next heads are loaded before these are worked on.
// VEC: every view's heads are whole pieces of 4 elements, the weights whole
// 16 bytes, and so are the rotated part and the way to a pair (2048 rows of 32
// + 8 heads, D = 128: 17.4 us with it, 19.3 without).
// 2048 rows, D = 128: 17 us, 42 MB, floor 8: vector instructions, those of every
// element (a head's element and its pair are both normed, and types and form of
// rotation told apart as the kernel runs), not the angles, which are found once
// a row.  4096 rows, D = 64,
// into the cache: 20 us.  One token: 3.5 us, a launch.
template <int D, bool VEC>
__global__ void __launch_bounds__(64 * WAVES) kv_rows_kernel(RowsArgs a) {
    constexpr int LPH = lanes_of(D), HPW = 64 / LPH;
    using L = KvLayout<D>;
    __shared__ double2 trig_s[WAVES][D / 2];
    const KvCache &c = a.c;
    const KvSeqs &sq = a.sq;
    const RowPrep &rp = a.rp;
    const int lane = threadIdx.x & 63, li = lane & (LPH - 1), sub = lane / LPH, i0 = 4 * li;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    double2 *trig = trig_s[wave];
    const int64_t unit = (int64_t)blockIdx.x * WAVES + wave;
    const int64_t t64 = unit / a.chunks;
    if (t64 >= sq.rows) return;
    const int t = (int)t64, g0 = (int)(unit % a.chunks) * a.per, g1 = g0 + a.per;
    const int gq = (a.hq + HPW - 1) / HPW, gk = (a.hkv + HPW - 1) / HPW;
    const int half = rp.rot_dim / 2;
    const bool apart = half && !rp.interleaved;  // pairs in another lane
    const bool turn = i0 < rp.rot_dim;           // (of the lane's first dimension)

    int64_t pos = 0;   // the row's place in its sequence
    int page = -1;
    if (a.cached) {
        const RowSeq r = row_seq(sq, t, lane);
        if (r.s >= sq.nseq) return;
        pos = (int64_t)__builtin_amdgcn_readfirstlane(sq.kv_len[r.s]) - r.n + (t - r.first);
        page = __builtin_amdgcn_readfirstlane(kv_page(c, sq, r.s, pos));
    }
    double cs[4] = {1, 1, 1, 1}, sn[4] = {0, 0, 0, 0};  // of the lane's dimensions, the sine with the pair's sign
    if (half && g0 < gq + gk) {
        const double p = rp.positions ? (double)rp.positions[t] : (double)pos;
        for (int j = lane; j < half; j += 64) {
            double s1, c1;
            sin_cos(p * (double)rp.inv_freq[j], s1, c1);
            trig[j] = make_double2(c1, s1);
        }
        wave_sync();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e;
            if (i >= rp.rot_dim) continue;
            const bool second = rp.interleaved ? e & 1 : i >= half;
            const double2 w = trig[rp.interleaved ? i >> 1 : second ? i - half : i];
            cs[e] = w.x;
            sn[e] = second ? w.y : -w.y;
        }
    }

    // The groups of one kind -- 0: queries, 1: keys, 2: values -- among g0 .. g1 - 1.
    auto heads = [&](auto kind_c, const Heads &src, const Heads &dst, int count, int start, int groups) {
        constexpr int kind = decltype(kind_c)::value;
        const int ga = max(g0 - start, 0), gb = min(g1 - start, groups);
        if (ga >= gb) return;
        const bool into = kind == 2 || (kind == 1 && a.cached);
        if (into && page < 0) return;
        float f[4], fo[4] = {0, 0, 0, 0}, nf[4], no[4] = {0, 0, 0, 0};  // the lane's dimensions and their pairs
        int h = ga * HPW + sub;
        auto fetch = [&](int hh, float *x, float *y) {
            const uint8_t *row = at(src, t, min(hh, count - 1), 0);
            const int sh = src.f16 ? 1 : 2;
            load4<VEC>(row + ((i0 * src.elem) << sh), src.elem, src.f16, x);
            if (kind < 2 && apart) {
                if constexpr (VEC) {
                    if (turn) load4<true>(row + ((i0 < half ? i0 + half : i0 - half) << sh), 1, src.f16, y);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = i0 + e;
                        if (i < rp.rot_dim) y[e] = load_head(Heads{(void *)row, 0, 0, 0, src.f16}, (i < half ? i + half : i - half) * src.elem);
                    }
                }
            }
        };
        fetch(h, f, fo);
        const float *nw = kind == 0 ? rp.q_norm : kind == 1 ? rp.k_norm : nullptr;
        float w[4] = {1, 1, 1, 1}, wo[4] = {1, 1, 1, 1};
        if (kind < 2 && nw) {
            load4<VEC>(reinterpret_cast<const uint8_t *>(nw + i0), 1, false, w);
            if (apart) {
                if constexpr (VEC) {
                    if (turn) load4<true>(reinterpret_cast<const uint8_t *>(nw + (i0 < half ? i0 + half : i0 - half)), 1, false, wo);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i0 + e < rp.rot_dim) wo[e] = nw[i0 + e < half ? i0 + e + half : i0 + e - half];
                }
            }
        }
        double wd[4], wod[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wd[e] = w[e];
            wod[e] = wo[e];
        }
        // work on the heads in f and fo
        auto one = [&](float *f, float *fo) {
            const bool on = h < count;
            if constexpr (kind < 2) {
                double x[4], y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = f[e];
                    y[e] = fo[e];
                }
                if (nw) {
                    double ss = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) ss = fma(x[e], x[e], ss);
                    const double r = rsqrt(head_sum<LPH>(ss) * (1.0 / D) + (double)rp.eps);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] *= r * wd[e];
                        if (apart) y[e] *= r * wod[e];
                    }
                }
                if (turn) {
                    double z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = fma(apart ? y[e] : x[e ^ 1], sn[e], x[e] * cs[e]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (VEC || i0 + e < rp.rot_dim) x[e] = z[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = (float)x[e];
            }
            if (!into) {
                if (on) store4<VEC>(at(dst, t, h, i0), dst.elem, dst.f16, f);
            } else if constexpr (kind > 0) {
                // groups of 32 dimensions, in fp32 from the rounded row
                float lo, hi;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[e] = f[e] != f[e] ? 0.f : fminf(fmaxf(f[e], -65504.f), 65504.f);
                    lo = e ? fminf(lo, f[e]) : f[e];
                    hi = e ? fmaxf(hi, f[e]) : f[e];
                }
                lo = fminf(lo, dpp<SWAP1>(lo)); hi = fmaxf(hi, dpp<SWAP1>(hi));
                lo = fminf(lo, dpp<SWAP2>(lo)); hi = fmaxf(hi, dpp<SWAP2>(hi));
                lo = fminf(lo, dpp<MIRROR8>(lo)); hi = fmaxf(hi, dpp<MIRROR8>(hi));
                const _Float16 mh = (_Float16)lo;
                const _Float16 dh = (_Float16)((hi - (float)mh) / 15.f);
                const float mf = (float)mh, df = (float)dh;
                uint32_t code[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = df > 0.f ? rintf((f[e] - mf) / df) : 0.f;
                    code[e] = (uint32_t)fminf(fmaxf(z, 0.f), 15.f);
                }
                uint8_t *blk = c.pool + ((int64_t)page * a.hkv + min(h, count - 1)) * 2 * L::block(c.ps_log2) +
                               (kind == 2 ? L::block(c.ps_log2) : 0);
                const int p = (int)(pos & ((1 << c.ps_log2) - 1)), g = li >> 3;
                if (on && (li & 7) == 0) {
                    reinterpret_cast<_Float16 *>(blk + L::d_off(c.ps_log2))[L::by4(p, g)] = dh;
                    reinterpret_cast<_Float16 *>(blk + L::m_off(c.ps_log2))[kind == 1 ? p * L::G + g : L::by4(p, g)] = mh;
                }
                if constexpr (kind == 1) {
                    // half of word (a, g), a = li / 2 % 4
                    const uint32_t b = code[0] | code[1] << 4 | code[2] << 8 | code[3] << 12;
                    if (on)
                        *reinterpret_cast<uint16_t *>(blk + p * L::ROW + 4 * (((li >> 1) & 3) * L::G + g) + 2 * (li & 1)) =
                            (uint16_t)b;
                } else {
                    // nibble n = li / 4 % 8 of pieces l = 4 (li % 4) + e: four words that the lanes of equal li % 4
                    // (and equal li / 32) have a nibble of each; every exchange halves what a lane still works on
                    const int n = (li >> 2) & (L::VN - 1);
                    const bool b2 = li & 4, b3 = li & 8;
                    const uint32_t s0 = code[0] << (4 * n), s1 = code[1] << (4 * n), s2 = code[2] << (4 * n),
                                   s3 = code[3] << (4 * n);
                    const uint32_t w0 = (b2 ? s2 : s0) | __shfl_xor(b2 ? s0 : s2, 4);
                    const uint32_t w1 = (b2 ? s3 : s1) | __shfl_xor(b2 ? s1 : s3, 4);
                    uint32_t b = (b3 ? w1 : w0) | __shfl_xor(b3 ? w0 : w1, 8);
                    if (D > 64) b |= __shfl_xor(b, 16);
                    uint8_t *o = blk + L::v_piece(p, li >> 5, 4 * (li & 3) + 2 * b2 + b3);
                    if (on && (D == 64 || (li & 16) == 0)) {
                        if (D == 64) *reinterpret_cast<uint16_t *>(o) = (uint16_t)b;
                        else *reinterpret_cast<uint32_t *>(o) = b;
                    }
                }
            }
        };
        for (int gi = ga; gi < gb; gi += 2) {
            if (gi + 1 < gb) fetch(h + HPW, nf, no);
            one(f, fo);
            h += HPW;
            if (gi + 1 >= gb) break;
            if (gi + 2 < gb) fetch(h + HPW, f, fo);
            one(nf, no);
            h += HPW;
        }
    };
    heads(std::integral_constant<int, 0>{}, a.q, a.qo, a.hq, 0, gq);
    heads(std::integral_constant<int, 1>{}, a.k, a.ko, a.hkv, gq, gk);
    if (a.cached) heads(std::integral_constant<int, 2>{}, a.v, a.ko, a.hkv, gq + gk, gk);
}

// Keys and values of HPW heads of a row: a wave.
template <int D>
__global__ void __launch_bounds__(64 * WAVES) kv_read_kernel(KvCache c, KvSeqs sq, Heads ko, Heads vo, int vko, int vvo) {
    constexpr int LPH = lanes_of(D), HPW = 64 / LPH;
    using L = KvLayout<D>;
    const int lane = threadIdx.x & 63, li = lane & (LPH - 1);
    const int per_row = (c.hkv + HPW - 1) / HPW;
    const int64_t unit = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    const int64_t t64 = unit / per_row;
    if (t64 >= sq.rows) return;
    const int t = (int)t64, h = (int)(unit % per_row) * HPW + lane / LPH;
    const RowSeq r = row_seq(sq, t, lane);
    if (r.s >= sq.nseq || h >= c.hkv) return;
    const int64_t pos = (int64_t)sq.kv_len[r.s] - r.n + (t - r.first);
    const int page = kv_page(c, sq, r.s, pos);
    const uint8_t *blk = c.pool + ((int64_t)max(page, 0) * c.hkv + h) * 2 * L::block(c.ps_log2);
    const int p = (int)(pos & ((1 << c.ps_log2) - 1)), g = li >> 3;
    for (int kind = 0; kind < 2; ++kind, blk += L::block(c.ps_log2)) {
        const Heads &dst = kind ? vo : ko;
        if (!dst.p) continue;
        float y[4] = {0, 0, 0, 0};
        if (page >= 0) {
            const float dh = (float)reinterpret_cast<const _Float16 *>(blk + L::d_off(c.ps_log2))[L::by4(p, g)];
            const float mh =
                (float)reinterpret_cast<const _Float16 *>(blk + L::m_off(c.ps_log2))[kind ? L::by4(p, g) : p * L::G + g];
            uint32_t code[4];
            if (kind == 0) {
                const uint32_t w =
                    *reinterpret_cast<const uint16_t *>(blk + p * L::ROW + 4 * (((li >> 1) & 3) * L::G + g) + 2 * (li & 1));
#pragma unroll
                for (int e = 0; e < 4; ++e) code[e] = (w >> (4 * e)) & 15u;
            } else {
                const int n = (li >> 2) & (L::VN - 1);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    code[e] = (blk[L::v_piece(p, li >> 5, 4 * (li & 3) + e) + (n >> 1)] >> (4 * (n & 1))) & 15u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = fmaf((float)code[e], dh, mh);
        }
        uint8_t *o = at(dst, t, h, 4 * li);
        if (kind ? vvo : vko) store4<true>(o, 1, dst.f16, y);
        else store4<false>(o, dst.elem, dst.f16, y);
    }
}

// Heads whose dimensions are whole pieces of 4 elements, aligned as such.
bool whole4(const Heads &x) {
    return x.p && x.elem == 1 && x.row % 4 == 0 && x.head % 4 == 0 && ((uintptr_t)x.p & (x.f16 ? 7 : 15)) == 0;
}

}  // namespace rows

using namespace rows;

hipError_t launch_kv_rows(const KvCache *cache, const KvSeqs &seqs, const RowPrep &prep, int D, int hq, const Heads &q,
                          const Heads &qo, int hkv, const Heads &k, const Heads &v, const Heads &ko,
                          hipStream_t st) {
    const int hpw = 256 / D, gq = (hq + hpw - 1) / hpw, gk = (hkv + hpw - 1) / hpw;
    const int total = gq + gk * (cache ? 2 : 1);
    RowsArgs a{cache ? *cache : KvCache{nullptr, 0, 0, D, 0}, seqs, prep, hq, hkv, cache ? 1 : 0, q, qo, k, v, ko, 1, 1};
    const bool vec = (!hq || (whole4(q) && whole4(qo))) && (!hkv || (whole4(k) && whole4(cache ? v : ko))) &&
                     prep.rot_dim % (prep.interleaved ? 4 : 8) == 0 && (((uintptr_t)prep.q_norm | (uintptr_t)prep.k_norm) & 15) == 0;
    // Few rows: a wave for every group of heads.  Many: a row's groups share
    // the row's sines and cosines, as far as 16 waves a unit are left (2048
    // rows, D = 128: 17.4 us; a wave a group 30.6, 4 waves a unit left 22.2, 64
    // left 22.6.  64 rows into the cache, D = 128: 10.1, 10.0, 11.2, 10.0).
    a.per = (int)std::max<int64_t>(1, std::min<int64_t>(total, (int64_t)seqs.rows * total / (16 * device_cus())));
    a.chunks = (total + a.per - 1) / a.per;
    const int64_t blocks = ((int64_t)seqs.rows * a.chunks + WAVES - 1) / WAVES;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, a); };
    if (D == 64) vec ? go(kv_rows_kernel<64, true>) : go(kv_rows_kernel<64, false>);
    else if (D == 128) vec ? go(kv_rows_kernel<128, true>) : go(kv_rows_kernel<128, false>);
    else vec ? go(kv_rows_kernel<256, true>) : go(kv_rows_kernel<256, false>);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, const KvSeqs &seqs, const Heads &ko, const Heads &vo, hipStream_t st) {
    const int hpw = 256 / c.D;
    const int64_t blocks = ((int64_t)seqs.rows * ((c.hkv + hpw - 1) / hpw) + WAVES - 1) / WAVES;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, c, seqs, ko, vo, whole4(ko), whole4(vo));
    };
    if (c.D == 64) go(kv_read_kernel<64>);
    else if (c.D == 128) go(kv_read_kernel<128>);
    else go(kv_read_kernel<256>);
    return hipGetLastError();
}

}  // namespace qk
