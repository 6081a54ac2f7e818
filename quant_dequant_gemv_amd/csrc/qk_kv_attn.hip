// qk_kv_attn.hip -- attention over the paged 4-bit cache on matrix cores.
//
// Mathematics.  With K_ji = d_jg c_ji + m_jg (g = i / 32), the score of a
// query row is sum_g d_jg (sum_{i in g} q_i c_ji) + sum_g m_jg (sum_{i in g}
// q_i).  A group's inner sum is one 16x16x32 matrix instruction of 16
// positions by 16 query rows on exact operands: a nibble masked in place is
// an fp16 subnormal, code * 2^-24 (or 16 times that for the odd nibbles,
// whose queries carry 1/16), so unpacking is five bit operations for eight
// codes and nothing is converted or rounded.  The step d is one fp32 fma per
// result.  The minima's term is one more instruction for all groups, the
// queries' group sums as two fp16 terms.
// The values likewise: O_i = sum_j (p_j d_jg) c_ji + sum_j p_j m_jg, where
// p_j d_jg goes in as two fp16 terms (product, and its exact residual by fma
// plus the residual of p), so a probability is never rounded to 11 bits.
//
// Layout.  Scores are computed transposed (positions are the rows of the
// result, query rows its columns) and so is the output (dimensions by query
// rows): a lane holds the same query row in both, the probabilities of a
// lane are the operand of the second product as they are (slot j of quad a
// is position 16 (j / 4) + 4 a + j % 4 of a tile of 32), and the softmax
// statistics are one scalar per lane.  The page layout is made for this:
// every operand is whole 16-byte pieces of the page, nothing passes LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qk_kv.h"

namespace qk {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int AW = 4;            // waves of a workgroup
constexpr int MAX_SPLIT = 256;   // splits of a sequence
constexpr float M_NONE = -3e38f; // running maximum before any visible position
constexpr float GROW = 2.f;      // a probability may reach 2^GROW before the maximum is moved

__device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return (float)__builtin_bit_cast(h2, v).x; }
__device__ __forceinline__ float hi_f(uint32_t v) { return (float)__builtin_bit_cast(h2, v).y; }
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const h2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}
// N dwords (N even) from an address aligned to min(4N, 16)
template <int N> __device__ __forceinline__ void load(uint32_t *r, const uint8_t *p) {
    if constexpr (N == 1) {
        r[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const u2 v = *reinterpret_cast<const u2 *>(p);
        r[0] = v.x; r[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u4 v = *reinterpret_cast<const u4 *>(p + 4 * i);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    }
}

// Query rows of a sequence, its heads of one KV head side by side: row r is
// token r / grp, head r % grp of the group.  Tiles of RT rows; a sequence's
// tiles are numbered from first * grp / RT + s, so that every tile of every
// sequence has a number of its own without a sum over the sequences.
struct Tile {
    int s, j;            // sequence, tile of it
    int first, n;        // its rows in the call
    int64_t p0;          // position of its first row
    int64_t t0, t1;      // tiles of 32 positions that some row sees
    int ns;              // splits that have work (at least 1)
};
struct AttnArgs {
    KvCache c;
    KvSeqs sq;
    Heads q, out;
    int hq, grp, window, nsplit, ntiles, per_split;
    float scale;
    float *o;            // partial outputs [unit][RT][D], unit = (tile * hkv + head) * nsplit + split
    float2 *ml;          // running maximum and sum [unit][RT]
};

template <int RT> __device__ __forceinline__ int tile_base(const AttnArgs &a, int first, int s) {
    return (int)((int64_t)first * a.grp / RT) + s;
}

// Visible range and splits of a tile whose s, j, first, n are set.
template <int RT> __device__ __forceinline__ void tile_range(const AttnArgs &a, Tile &t) {
    const int64_t len = a.sq.kv_len[t.s];
    t.p0 = len - t.n;
    const int r0 = t.j * RT, r1 = min(r0 + RT, t.n * a.grp) - 1;
    const int64_t pmin = t.p0 + r0 / a.grp, pmax = t.p0 + r1 / a.grp;
    const int64_t end = min(pmax + 1, (int64_t)a.sq.max_pages << a.c.ps_log2);
    const int64_t begin = a.window ? max((int64_t)0, pmin - a.window + 1) : 0;
    t.t0 = begin >> 5;
    t.t1 = end > begin ? (end + 31) >> 5 : t.t0;
    const int64_t nt = t.t1 - t.t0;
    t.ns = (int)max((int64_t)1, min((int64_t)a.nsplit, (nt + a.per_split - 1) / a.per_split));
}

// The tile of number b, or false if it is none.  One wave, uniform.
template <int RT> __device__ __forceinline__ bool find_tile(const AttnArgs &a, int b, int lane, Tile &t) {
    if (!a.sq.q_start) {
        t.n = a.sq.rows / a.sq.nseq;
        const int per = (t.n * a.grp + RT - 1) / RT;
        t.s = b / per;
        t.j = b % per;
        t.first = t.s * t.n;
    } else {
        int cnt = 0;
        for (int i0 = 0; i0 < a.sq.nseq; i0 += 64) {
            const int i = min(i0 + lane, a.sq.nseq - 1);
            const int base = tile_base<RT>(a, clamp_row(a.sq, a.sq.q_start[i]), i);
            cnt += __popcll(__ballot(i0 + lane < a.sq.nseq && base <= b));
        }
        if (!cnt) return false;
        t.s = cnt - 1;
        t.first = clamp_row(a.sq, a.sq.q_start[t.s]);
        t.n = clamp_row(a.sq, a.sq.q_start[t.s + 1]) - t.first;
        t.j = b - tile_base<RT>(a, t.first, t.s);
        if (t.n <= 0 || t.j < 0 || (int64_t)t.j * RT >= (int64_t)t.n * a.grp) return false;
    }
    tile_range<RT>(a, t);
    return true;
}

__device__ __forceinline__ void store_out(const Heads &o, int64_t i, float v) {
    if (o.f16) reinterpret_cast<_Float16 *>(o.p)[i] = (_Float16)v;
    else reinterpret_cast<float *>(o.p)[i] = v;
}

// One workgroup: a tile of 16 MT query rows, one KV head, one split of the
// positions; its waves take tiles of 32 positions in turn and join at the end.
template <int D, int MT>
__global__ void __launch_bounds__(64 * AW, MT == 1 ? 2 : 1) kv_attn_kernel(AttnArgs a) {
    using L = KvLayout<D>;
    constexpr int G = L::G, RT = 16 * MT, NT = D / 16, OP = D + 4;
    constexpr int VD = D >= 128 ? 4 : 2;  // dwords of a lane's four value pieces
    __shared__ float4 red4[AW * 16 * OP / 4];
    __shared__ float2 st[AW][RT];
    float *red = reinterpret_cast<float *>(red4);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int hk = blockIdx.x % a.c.hkv, bs = blockIdx.x / a.c.hkv;
    const int split = bs % a.nsplit, tile = bs / a.nsplit;
    Tile t;
    if (!find_tile<RT>(a, tile, lane, t) || split >= t.ns) return;
    const int R = t.n * a.grp;

    // query rows as the second operand, scaled by a power of two per row so
    // that neither they nor their sixteenths are subnormal
    u4 qf[MT][G], qs[MT];
    float sc1[MT], sc2[MT];
    int lim[MT], low[MT];
    const int64_t cap = (int64_t)a.sq.max_pages << a.c.ps_log2;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = t.j * RT + mt * 16 + col, rr = min(r, R - 1), tok = rr / a.grp;
        const int64_t pos = t.p0 + tok;
        lim[mt] = (int)max((int64_t)-1, min(pos, cap - 1));
        low[mt] = a.window ? (int)min(max((int64_t)0, pos - a.window + 1), (int64_t)INT32_MAX) : 0;
        const _Float16 *src = reinterpret_cast<const _Float16 *>(a.q.p) + (int64_t)(t.first + tok) * a.q.row +
                              (int64_t)(hk * a.grp + rr % a.grp) * a.q.head;
        float v[G][8], mx = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                v[g][n] = (float)src[(int64_t)(32 * g + 8 * quad + n) * a.q.elem];
                mx = fmaxf(mx, fabsf(v[g][n]));
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        // mx * 2^e in [2^9, 2^10); infinite, NaN or zero rows as they are
        const int e = mx > 0.f && mx < 1e30f ? 10 - (int)((__float_as_uint(mx) >> 23) - 126) : 0;
        const float f = __uint_as_float((uint32_t)(127 + e) << 23), inv = __uint_as_float((uint32_t)(127 - e) << 23);
        sc2[mt] = a.scale * 1.44269504088896340736f * inv;
        sc1[mt] = sc2[mt] * 16777216.f;
        uint32_t sums[4] = {0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float s = 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                v[g][n] *= f;
                s += v[g][n];
            }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            // nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7: the odd ones' codes come 16 times too large
            qf[mt][g] = u4{pack(v[g][0], v[g][4]), pack(v[g][1] * 0.0625f, v[g][5] * 0.0625f), pack(v[g][2], v[g][6]),
                           pack(v[g][3] * 0.0625f, v[g][7] * 0.0625f)};
            const _Float16 hi = (_Float16)s;
            const _Float16 w = quad == 0 ? hi : quad == 1 ? (_Float16)(s - (float)hi) : (_Float16)0.f;
            sums[g >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, w) << (16 * (g & 1));
        }
        qs[mt] = u4{sums[0], sums[1], sums[2], sums[3]};
    }
    // (wave-uniform) tiles that every row sees whole, and positions that hold something
    const int64_t all_lo = a.window ? max((int64_t)0, t.p0 + (min(t.j * RT + RT, R) - 1) / a.grp - a.window + 1) : 0;
    const int64_t all_hi = min(t.p0 + (int64_t)(t.j * RT / a.grp), cap - 1);
    const int64_t held = min(t.p0 + t.n, cap);

    f4 o[MT][NT], om[MT];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < NT; ++i) o[mt][i] = f4{0.f, 0.f, 0.f, 0.f};
        om[mt] = f4{0.f, 0.f, 0.f, 0.f};
        m[mt] = M_NONE;
        l[mt] = 0.f;
    }

    const int64_t nt = t.t1 - t.t0;
    const int64_t x0 = t.t0 + nt * split / t.ns, x1 = t.t0 + nt * (split + 1) / t.ns;
    const int32_t *table = a.sq.pages + (int64_t)t.s * a.sq.max_pages;
    const int tsh = a.c.ps_log2 - 5;
    const int64_t pstride = 2 * a.c.hkv * L::block(a.c.ps_log2);
    const uint8_t *pool = a.c.pool + (int64_t)hk * 2 * L::block(a.c.ps_log2);
    auto page_of = [&](int64_t x) { return x < x1 ? table[x >> tsh] : -1; };

    for (int64_t x = x0 + wave; x < x1; x += AW) {
        const int page = page_of(x);
        if (page < 0 || page >= a.c.num_pages) continue;
        const uint8_t *kb = pool + page * pstride, *vb = kb + L::block(a.c.ps_log2);
        const int p0 = (int)(x & ((1 << tsh) - 1)) << 5;  // of the page
        uint32_t kc[2][G], kd[2][2 * G], km[2][G / 2], vc[2][L::VW][VD], vd[2][2 * G], vm[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int pc = p0 + 16 * u + col, pq = (p0 >> 2) + 4 * u + quad;
            load<G>(kc[u], kb + pc * L::ROW + quad * 4 * G);
            load<2 * G>(kd[u], kb + L::d_off(a.c.ps_log2) + pq * 8 * G);
            load<G / 2>(km[u], kb + L::m_off(a.c.ps_log2) + pc * 2 * G);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int pq = (p0 >> 2) + 4 * u + quad;
#pragma unroll
            for (int w = 0; w < L::VW; ++w) load<VD>(vc[u][w], vb + ((pq * L::VW + w) * 16 + col) * 4 * VD);
            load<2 * G>(vd[u], vb + L::d_off(a.c.ps_log2) + pq * 8 * G);
            load<2>(vm[u], vb + L::m_off(a.c.ps_log2) + (pq * G + min(col, G - 1)) * 8);
        }
        // places that hold nothing yet: whatever their bytes say, the step and the minimum are 0
        if (x * 32 + 32 > held) {
            const int left = (int)(held - x * 32);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int p = 16 * u + 4 * quad + 2 * k;
                    const uint32_t mask = (p < left ? 0xffffu : 0u) | (p + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
                    for (int g = 0; g < G; ++g) vd[u][2 * g + k] &= mask;
                    vm[u][k] &= mask;
                }
        }

        // scores
        float z[MT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f4 s[MT];
            u4 mo = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < G / 2; ++i) mo[i] = km[u][i];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[mt] = mfma(mo, qs[mt], f4{0.f, 0.f, 0.f, 0.f});
                s[mt] *= sc2[mt];
            }
            f4 acc[MT];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t w = kc[u][g], w8 = w >> 8;
                const u4 ko = {w & 0x000f000fu, w & 0x00f000f0u, w8 & 0x000f000fu, w8 & 0x00f000f0u};
                const float d0 = lo_f(kd[u][2 * g]), d1 = hi_f(kd[u][2 * g]), d2 = lo_f(kd[u][2 * g + 1]),
                            d3 = hi_f(kd[u][2 * g + 1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const f4 r = mfma(ko, qf[mt][g], f4{0.f, 0.f, 0.f, 0.f});
                    if (g == 0) acc[mt] = f4{d0 * r.x, d1 * r.y, d2 * r.z, d3 * r.w};
                    else
                        acc[mt] = f4{fmaf(d0, r.x, acc[mt].x), fmaf(d1, r.y, acc[mt].y), fmaf(d2, r.z, acc[mt].z),
                                     fmaf(d3, r.w, acc[mt].w)};
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[mt][u][i] = fmaf(acc[mt][i], sc1[mt], s[mt][i]);
        }
        if (x * 32 < all_lo || x * 32 + 31 > all_hi) {
            const int base = (int)(x * 32) + 4 * quad;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = base + 16 * u + i;
                        z[mt][u][i] = p <= lim[mt] && p >= low[mt] ? z[mt][u][i] : -INFINITY;
                    }
        }

        // probabilities relative to the running maximum, as two fp16 terms
        uint32_t ph[MT][2][2], pl[MT][2][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float mx = z[mt][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) mx = fmaxf(mx, z[mt][i >> 2][i & 3]);
            if (__any(mx > m[mt] + GROW)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float mn = fmaxf(mx, m[mt]), al = __builtin_amdgcn_exp2f(m[mt] - mn);
                m[mt] = mn;
                l[mt] *= al;
                om[mt] *= al;
#pragma unroll
                for (int i = 0; i < NT; ++i) o[mt][i] *= al;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float p0 = __builtin_amdgcn_exp2f(z[mt][u][2 * k] - m[mt]);
                    const float p1 = __builtin_amdgcn_exp2f(z[mt][u][2 * k + 1] - m[mt]);
                    l[mt] += p0 + p1;
                    ph[mt][u][k] = pack(p0, p1);
                    pl[mt][u][k] = pack(p0 - lo_f(ph[mt][u][k]), p1 - hi_f(ph[mt][u][k]));
                }
        }

        // values
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const u4 mo = {vm[0][0], vm[0][1], vm[1][0], vm[1][1]};
            om[mt] = mfma(mo, u4{ph[mt][0][0], ph[mt][0][1], ph[mt][1][0], ph[mt][1][1]}, om[mt]);
            om[mt] = mfma(mo, u4{pl[mt][0][0], pl[mt][0][1], pl[mt][1][0], pl[mt][1][1]}, om[mt]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            u4 v0, v1;  // dimensions 32g .. 32g+15 and 32g+16 .. 32g+31 (those 16 times too large)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t w;
                    if constexpr (D == 64) {
                        w = vc[u][0][k] >> (8 * g);
                    } else {
                        const uint32_t sel = 0x0c040c00u + 0x00010001u * (uint32_t)(g & 3);
                        w = __builtin_amdgcn_perm(vc[u][g >> 2][2 * k + 1], vc[u][g >> 2][2 * k], sel);
                    }
                    v0[2 * u + k] = w & 0x000f000fu;
                    v1[2 * u + k] = w & 0x00f000f0u;
                }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                u4 hi, lo;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const h2 d = __builtin_bit_cast(h2, vd[u][2 * g + k]);
                        const h2 p = __builtin_bit_cast(h2, ph[mt][u][k]), q = __builtin_bit_cast(h2, pl[mt][u][k]);
                        const h2 x2 = p * d;
                        const h2 r = __builtin_elementwise_fma(p, d, -x2);
                        hi[2 * u + k] = __builtin_bit_cast(uint32_t, x2);
                        lo[2 * u + k] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(q, d, r));
                    }
                o[mt][2 * g] = mfma(v0, hi, o[mt][2 * g]);
                o[mt][2 * g + 1] = mfma(v1, hi, o[mt][2 * g + 1]);
                o[mt][2 * g] = mfma(v0, lo, o[mt][2 * g]);
                o[mt][2 * g + 1] = mfma(v1, lo, o[mt][2 * g + 1]);
            }
        }
    }

    // join the waves: common maximum, then sums through LDS, 16 rows at a time
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16);
        l[mt] += __shfl_xor(l[mt], 32);
        if (quad == 0) st[wave][mt * 16 + col] = make_float2(m[mt], l[mt]);
    }
    __syncthreads();
    const int64_t unit = ((int64_t)tile * a.c.hkv + hk) * a.nsplit + split;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float mx = st[0][mt * 16 + col].x;
#pragma unroll
        for (int w = 1; w < AW; ++w) mx = fmaxf(mx, st[w][mt * 16 + col].x);
        const float f = __builtin_amdgcn_exp2f(m[mt] - mx);
        float *mine = red + (wave * 16 + col) * OP;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // the group's minima term: row g of om, held by quad g / 4
            const float mg = __shfl(om[mt][g & 3], (g >> 2) * 16 + col);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f4 v = o[mt][2 * g + k];
                const float s = k ? 1048576.f : 16777216.f;  // 2^20, 2^24: the codes' units
                *reinterpret_cast<float4 *>(mine + 32 * g + 16 * k + 4 * quad) =
                    make_float4(fmaf(v.x, s, mg) * f, fmaf(v.y, s, mg) * f, fmaf(v.z, s, mg) * f, fmaf(v.w, s, mg) * f);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * D / 4; i += 64 * AW) {
            const int row = i / (D / 4), c4 = i % (D / 4), r = t.j * RT + mt * 16 + row;
            if (r >= R) continue;
            float4 s = *reinterpret_cast<const float4 *>(red + row * OP + 4 * c4);
#pragma unroll
            for (int w = 1; w < AW; ++w) {
                const float4 v = *reinterpret_cast<const float4 *>(red + (w * 16 + row) * OP + 4 * c4);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
            float mm = st[0][mt * 16 + row].x, ll = 0.f;
#pragma unroll
            for (int w = 1; w < AW; ++w) mm = fmaxf(mm, st[w][mt * 16 + row].x);
#pragma unroll
            for (int w = 0; w < AW; ++w) ll = fmaf(__builtin_amdgcn_exp2f(st[w][mt * 16 + row].x - mm), st[w][mt * 16 + row].y, ll);
            if (t.ns == 1) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int64_t at = (int64_t)(t.first + r / a.grp) * a.out.row +
                                   (int64_t)(hk * a.grp + r % a.grp) * a.out.head + (int64_t)(4 * c4) * a.out.elem;
                store_out(a.out, at, s.x * inv);
                store_out(a.out, at + a.out.elem, s.y * inv);
                store_out(a.out, at + 2 * a.out.elem, s.z * inv);
                store_out(a.out, at + 3 * a.out.elem, s.w * inv);
            } else {
                reinterpret_cast<float4 *>(a.o + (unit * RT + mt * 16 + row) * D)[c4] = s;
                if (c4 == 0) a.ml[unit * RT + mt * 16 + row] = make_float2(mm, ll);
            }
        }
        __syncthreads();
    }
}

// Joins the splits of a row: one workgroup per row and query head.
template <int D, int RT>
__global__ void __launch_bounds__(256) kv_attn_join_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    __shared__ float wt[MAX_SPLIT], part[4][D], mx_s[4], sum_s[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = blockIdx.x / a.hq, h = blockIdx.x % a.hq;
    const RowSeq rs = row_seq(a.sq, row, lane);
    if (rs.s >= a.sq.nseq) return;
    const int hk = h / a.grp, r = (row - rs.first) * a.grp + h % a.grp;
    Tile t;
    t.s = rs.s;
    t.first = rs.first;
    t.n = rs.n;
    t.j = r / RT;
    tile_range<RT>(a, t);
    const int ns = t.ns;
    if (ns == 1) return;  // written already
    const int64_t tile = a.sq.q_start ? tile_base<RT>(a, clamp_row(a.sq, rs.first), rs.s) + t.j
                                      : (int64_t)rs.s * ((rs.n * a.grp + RT - 1) / RT) + t.j;
    if (tile >= a.ntiles) return;
    const int64_t unit = (tile * a.c.hkv + hk) * a.nsplit;
    const float2 v = tid < ns ? a.ml[(unit + tid) * RT + r % RT] : make_float2(M_NONE, 0.f);
    float mx = v.x;
    for (int i = 1; i < 64; i <<= 1) mx = fmaxf(mx, __shfl_xor(mx, i));
    if (lane == 0) mx_s[wave] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(mx_s[0], mx_s[1]), fmaxf(mx_s[2], mx_s[3]));
    const float w = __builtin_amdgcn_exp2f(v.x - mx);
    float sum = tid < ns ? w * v.y : 0.f;
    wt[tid] = w;
    for (int i = 1; i < 64; i <<= 1) sum += __shfl_xor(sum, i);
    if (lane == 0) sum_s[wave] = sum;
    __syncthreads();
    sum = (sum_s[0] + sum_s[1]) + (sum_s[2] + sum_s[3]);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 8
    for (int s = wave; s < ns; s += 4) {
        const float *p = a.o + ((unit + s) * RT + r % RT) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wt[s], p[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[wave][lane * E + e] = acc[e];
    __syncthreads();
    if (tid < D) {
        const float y = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        store_out(a.out, row * a.out.row + h * a.out.head + tid * a.out.elem, sum == 0.f ? 0.f : y / sum);
    }
}

// Launch shape: from sizes alone (the lengths are on the device).
struct Shape {
    int mt, ntiles, nsplit, per_split;
};
Shape attn_shape(const KvCache &c, const KvSeqs &sq, int hq) {
    const int grp = hq / c.hkv;
    Shape s;
    s.mt = c.D < 256 && (int64_t)sq.rows * grp > (int64_t)16 * sq.nseq ? 2 : 1;
    const int RT = 16 * s.mt;
    const int64_t n = sq.rows / sq.nseq;
    s.ntiles = (int)(sq.q_start ? (int64_t)sq.rows * grp / RT + sq.nseq : sq.nseq * ((n * grp + RT - 1) / RT));
    const int64_t most = ((int64_t)sq.max_pages << c.ps_log2) / 32;  // tiles of 32 positions
    s.per_split = 2 * AW;
    int64_t ns = 2 * device_cus() / ((int64_t)s.ntiles * c.hkv);
    ns = std::min<int64_t>(ns, (most + s.per_split - 1) / s.per_split);
    s.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>(ns, MAX_SPLIT));
    return s;
}

}  // namespace

int64_t kv_attn_workspace(const KvCache &c, const KvSeqs &sq, int hq) {
    const Shape s = attn_shape(c, sq, hq);
    if (s.nsplit == 1) return 0;
    return (int64_t)s.ntiles * c.hkv * s.nsplit * 16 * s.mt * (4 * c.D + 8);
}

hipError_t launch_kv_attn(const KvCache &c, const KvSeqs &seqs, int hq, const Heads &q, const Heads &out, float scale,
                          int window, void *workspace, hipStream_t st) {
    const Shape s = attn_shape(c, seqs, hq);
    AttnArgs a{c, seqs, q, out, hq, hq / c.hkv, window, s.nsplit, s.ntiles, s.per_split, scale, nullptr, nullptr};
    if (s.nsplit > 1) {
        a.o = (float *)workspace;
        a.ml = (float2 *)(a.o + (int64_t)s.ntiles * c.hkv * s.nsplit * 16 * s.mt * c.D);
    }
    const int64_t blocks = (int64_t)s.ntiles * c.hkv * s.nsplit;
    auto go = [&](auto kern, auto join) -> hipError_t {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * AW), 0, st, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || s.nsplit == 1) return e;
        hipLaunchKernelGGL(join, dim3((unsigned)(seqs.rows * hq)), dim3(256), 0, st, a);
        return hipGetLastError();
    };
#define QK_ATTN(D)                                                                                    \
    return s.mt == 1 ? go(kv_attn_kernel<D, 1>, kv_attn_join_kernel<D, 16>)                           \
                     : go(kv_attn_kernel<D, 2>, kv_attn_join_kernel<D, 32>)
    if (c.D == 64) QK_ATTN(64);
    if (c.D == 128) QK_ATTN(128);
    return go(kv_attn_kernel<256, 1>, kv_attn_join_kernel<256, 16>);
#undef QK_ATTN
}

}  // namespace qk
