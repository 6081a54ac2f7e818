// qk_kv.hip -- rows of heads: norm + rotation, appending to the paged 4-bit
// cache, and reading it back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_kv.h"

namespace qk {
namespace {

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
__device__ __forceinline__ void store_head(const Heads &x, int64_t i, double v) {
    if (x.f16) reinterpret_cast<_Float16 *>(x.p)[i] = (_Float16)(float)v;
    else reinterpret_cast<float *>(x.p)[i] = (float)v;
}

template <int D> struct WaveLds {
    double x[D];           // a normed row, for the pairs of the rotation
    double2 trig[D / 2];   // (cos, sin) of the row's angles
    uint8_t code[D];
};

// One wave: E = D/64 consecutive dimensions a lane, groups of 32/E lanes.  A
// row's angles are the same for all its heads, so a wave takes `per` heads of
// one row and computes them once.
template <int D>
__global__ void __launch_bounds__(64 * WAVES)
kv_rows_kernel(KvCache c, KvSeqs sq, RowPrep rp, int hq, Heads q, Heads qo, int hkv, Heads k, Heads v, Heads ko,
               int cached, int per, int chunks) {
    constexpr int E = D / 64;
    using L = KvLayout<D>;
    __shared__ WaveLds<D> lds[WAVES];
    const int lane = threadIdx.x & 63;
    WaveLds<D> &w = lds[threadIdx.x >> 6];
    const int64_t unit = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    const int64_t t64 = unit / chunks;
    if (t64 >= sq.rows) return;
    const int t = (int)t64, h0 = (int)(unit % chunks) * per;

    int64_t pos = 0;   // the row's place in its sequence
    int page = -1;
    if (cached) {
        const RowSeq r = row_seq(sq, t, lane);
        if (r.s >= sq.nseq) return;
        pos = (int64_t)sq.kv_len[r.s] - r.n + (t - r.first);
        page = kv_page(c, sq, r.s, pos);
    }
    const int half = rp.rot_dim / 2;
    if (half) {
        const double p = rp.positions ? (double)rp.positions[t] : (double)pos;
        for (int j = lane; j < half; j += 64) {
            double sn, cs;
            sincos(p * (double)rp.inv_freq[j], &sn, &cs);
            w.trig[j] = make_double2(cs, sn);
        }
        wave_sync();
    }

    const int total = hq + hkv * (cached ? 2 : 1), h1 = min(h0 + per, total);
    for (int h = h0; h < h1; ++h) {
        const int kind = h < hq ? 0 : h < hq + hkv ? 1 : 2;  // query, key, value head
        const Heads &src = kind == 0 ? q : kind == 1 ? k : v;
        const int hh = kind == 0 ? h : kind == 1 ? h - hq : h - hq - hkv;
        if (kind && cached && page < 0) continue;
        const int64_t base = t * src.row + hh * src.head + (int64_t)(lane * E) * src.elem;
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = load_head(src, base + e * src.elem);
        double x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = f[e];
        if (kind < 2) {
            const float *nw = kind == 0 ? rp.q_norm : rp.k_norm;
            if (nw) {
                double ss = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) ss = fma(x[e], x[e], ss);
#pragma unroll
                for (int m = 1; m < 64; m <<= 1) ss += __shfl_xor(ss, m);
                const double r = 1.0 / sqrt(ss * (1.0 / D) + (double)rp.eps);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = x[e] * r * (double)nw[lane * E + e];
            }
            if (half) {
#pragma unroll
                for (int e = 0; e < E; ++e) w.x[lane * E + e] = x[e];
                wave_sync();
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = lane * E + e;
                    if (i < rp.rot_dim) {
                        const int j = rp.interleaved ? i >> 1 : i < half ? i : i - half;
                        const bool second = rp.interleaved ? i & 1 : i >= half;
                        const int o = rp.interleaved ? i ^ 1 : second ? i - half : i + half;
                        const double2 cs = w.trig[j];
                        x[e] = second ? w.x[o] * cs.y + x[e] * cs.x : x[e] * cs.x - w.x[o] * cs.y;
                    }
                }
                wave_sync();
            }
            if (kind == 0 || !cached) {
                const Heads &dst = kind == 0 ? qo : ko;
                const int64_t ob = t * dst.row + hh * dst.head + (int64_t)(lane * E) * dst.elem;
#pragma unroll
                for (int e = 0; e < E; ++e) store_head(dst, ob + e * dst.elem, x[e]);
                continue;
            }
        }
        // groups of 32 dimensions, in fp32 from the rounded row
        float lo = 65504.f, hi = -65504.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float y = (float)x[e];
            f[e] = y != y ? 0.f : fminf(fmaxf(y, -65504.f), 65504.f);
            lo = fminf(lo, f[e]);
            hi = fmaxf(hi, f[e]);
        }
#pragma unroll
        for (int m = 1; m < 32 / E; m <<= 1) {
            lo = fminf(lo, __shfl_xor(lo, m));
            hi = fmaxf(hi, __shfl_xor(hi, m));
        }
        const _Float16 mh = (_Float16)lo;
        const _Float16 dh = (_Float16)((hi - (float)mh) / 15.f);
        const float mf = (float)mh, df = (float)dh;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float z = df > 0.f ? rintf((f[e] - mf) / df) : 0.f;
            w.code[lane * E + e] = (uint8_t)fminf(fmaxf(z, 0.f), 15.f);
        }
        wave_sync();
        uint8_t *blk = c.pool + ((int64_t)page * hkv + hh) * 2 * L::block(c.ps_log2) +
                       (kind == 2 ? L::block(c.ps_log2) : 0);
        const int p = (int)(pos & ((1 << c.ps_log2) - 1)), g = lane * E / 32;
        if (lane % (32 / E) == 0) {
            reinterpret_cast<_Float16 *>(blk + L::d_off(c.ps_log2))[L::by4(p, g)] = dh;
            reinterpret_cast<_Float16 *>(blk + L::m_off(c.ps_log2))[kind == 1 ? p * L::G + g : L::by4(p, g)] = mh;
        }
        if (kind == 1) {
            if (lane < D / 8) {
                const uint2 b = *reinterpret_cast<const uint2 *>(w.code + 32 * (lane % L::G) + 8 * (lane / L::G));
                uint32_t word = 0;
#pragma unroll
                for (int n = 0; n < 8; ++n) word |= (((n < 4 ? b.x : b.y) >> (8 * (n & 3))) & 15u) << (4 * n);
                reinterpret_cast<uint32_t *>(blk + p * L::ROW)[lane] = word;
            }
        } else if (lane < 16 * L::VW) {
            const uint8_t *src8 = w.code + 128 * (lane >> 4) + (lane & 15);
            uint32_t word = 0;
#pragma unroll
            for (int n = 0; n < L::VN; ++n) word |= (uint32_t)src8[16 * n] << (4 * n);
            uint8_t *o = blk + L::v_piece(p, lane >> 4, lane & 15);
            if (D == 64) *reinterpret_cast<uint16_t *>(o) = (uint16_t)word;
            else *reinterpret_cast<uint32_t *>(o) = word;
        }
        wave_sync();
    }
}

// One wave per (row, KV head), keys and values.
template <int D>
__global__ void __launch_bounds__(64 * WAVES) kv_read_kernel(KvCache c, KvSeqs sq, Heads ko, Heads vo) {
    constexpr int E = D / 64;
    using L = KvLayout<D>;
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    const int64_t t64 = unit / c.hkv;
    if (t64 >= sq.rows) return;
    const int t = (int)t64, h = (int)(unit % c.hkv);
    const RowSeq r = row_seq(sq, t, lane);
    if (r.s >= sq.nseq) return;
    const int64_t pos = (int64_t)sq.kv_len[r.s] - r.n + (t - r.first);
    const int page = kv_page(c, sq, r.s, pos);
    const uint8_t *blk = c.pool + ((int64_t)max(page, 0) * c.hkv + h) * 2 * L::block(c.ps_log2);
    const int p = (int)(pos & ((1 << c.ps_log2) - 1));
    for (int kind = 0; kind < 2; ++kind, blk += L::block(c.ps_log2)) {
        const Heads &dst = kind ? vo : ko;
        if (!dst.p) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = lane * E + e, g = i >> 5;
            float y = 0.f;
            if (page >= 0) {
                const _Float16 dh = reinterpret_cast<const _Float16 *>(blk + L::d_off(c.ps_log2))[L::by4(p, g)];
                const _Float16 mh =
                    reinterpret_cast<const _Float16 *>(blk + L::m_off(c.ps_log2))[kind ? L::by4(p, g) : p * L::G + g];
                int at, n;
                if (kind == 0) {
                    n = i & 7;
                    at = p * L::ROW + 4 * (((i >> 3) & 3) * L::G + g) + (n >> 1);
                } else {
                    n = (i >> 4) & (L::VN - 1);
                    at = L::v_piece(p, D == 64 ? 0 : i >> 7, i & 15) + (n >> 1);
                }
                const int code = (blk[at] >> (4 * (n & 1))) & 15;
                y = fmaf((float)code, (float)dh, (float)mh);
            }
            store_head(dst, t * dst.row + h * dst.head + (int64_t)i * dst.elem, y);
        }
    }
}

}  // namespace

hipError_t launch_kv_rows(const KvCache *cache, const KvSeqs &seqs, const RowPrep &prep, int D, int hq, const Heads &q,
                          const Heads &qo, int hkv, const Heads &k, const Heads &v, const Heads &ko,
                          hipStream_t st) {
    const KvCache c = cache ? *cache : KvCache{nullptr, 0, 0, D, 0};
    const int total = hq + hkv * (cache ? 2 : 1);
    const int per = 1, chunks = (total + per - 1) / per;
    const int64_t blocks = ((int64_t)seqs.rows * chunks + WAVES - 1) / WAVES;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, c, seqs, prep, hq, q, qo, hkv, k, v,
                           ko, cache ? 1 : 0, per, chunks);
    };
    if (D == 64) go(kv_rows_kernel<64>);
    else if (D == 128) go(kv_rows_kernel<128>);
    else go(kv_rows_kernel<256>);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, const KvSeqs &seqs, const Heads &ko, const Heads &vo, hipStream_t st) {
    const int64_t blocks = ((int64_t)seqs.rows * c.hkv + WAVES - 1) / WAVES;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, c, seqs, ko, vo);
    };
    if (c.D == 64) go(kv_read_kernel<64>);
    else if (c.D == 128) go(kv_read_kernel<128>);
    else go(kv_read_kernel<256>);
    return hipGetLastError();
}

}  // namespace qk
