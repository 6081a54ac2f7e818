// qk_kv_attn.hip -- attention over the paged 4-bit cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_kv.h"

namespace qk {
namespace {

// One workgroup per (row, query head): chunks of 256 positions, a score per
// thread, then a dimension per thread.
template <int D>
__global__ void __launch_bounds__(256)
kv_attn_simple_kernel(KvCache c, KvSeqs sq, int hq, Heads q, Heads out, float scale, int window) {
    using L = KvLayout<D>;
    __shared__ float qs[D], sc[256], red[256];
    const int tid = threadIdx.x, t = blockIdx.x / hq, h = blockIdx.x % hq, hk = h / (hq / c.hkv);
    const RowSeq r = row_seq(sq, t, tid & 63);
    if (r.s >= sq.nseq) return;
    const int64_t p64 = (int64_t)sq.kv_len[r.s] - r.n + (t - r.first);
    const int64_t end = min(p64 + 1, (int64_t)sq.max_pages << c.ps_log2);
    const int64_t begin = window ? max((int64_t)0, p64 - window + 1) : 0;
    for (int i = tid; i < D; i += 256)
        qs[i] = (float)reinterpret_cast<const _Float16 *>(q.p)[t * q.row + h * q.head + i * q.elem];
    float m = -INFINITY, l = 0.f, o = 0.f;
    __syncthreads();
    for (int64_t j0 = begin; j0 < end; j0 += 256) {
        const int64_t j = j0 + tid;
        const int page = j < end ? kv_page(c, sq, r.s, j) : -1;
        float s = -INFINITY;
        if (page >= 0) {
            const uint8_t *blk = c.pool + ((int64_t)page * c.hkv + hk) * 2 * L::block(c.ps_log2);
            const int p = (int)(j & ((1 << c.ps_log2) - 1));
            s = 0.f;
            for (int i = 0; i < D; ++i) {
                const int g = i >> 5, n = i & 7;
                const int code = (blk[p * L::ROW + 4 * (((i >> 3) & 3) * L::G + g) + (n >> 1)] >> (4 * (n & 1))) & 15;
                const float d = (float)reinterpret_cast<const _Float16 *>(blk + L::d_off(c.ps_log2))[L::by4(p, g)];
                const float mm = (float)reinterpret_cast<const _Float16 *>(blk + L::m_off(c.ps_log2))[p * L::G + g];
                s = fmaf(qs[i], fmaf((float)code, d, mm), s);
            }
            s *= scale;
        }
        red[tid] = s;
        __syncthreads();
        float mn = m;
        for (int i = 0; i < 256; ++i) mn = fmaxf(mn, red[i]);
        sc[tid] = page >= 0 ? expf(s - mn) : 0.f;
        __syncthreads();
        const float a = m == mn ? 1.f : expf(m - mn);
        m = mn;
        l *= a;
        o *= a;
        for (int jj = 0; jj < 256 && j0 + jj < end; ++jj) {
            const int pg = kv_page(c, sq, r.s, j0 + jj);
            if (pg < 0) continue;
            l += sc[jj];
            if (tid < D) {
                const uint8_t *blk = c.pool + (((int64_t)pg * c.hkv + hk) * 2 + 1) * L::block(c.ps_log2);
                const int p = (int)((j0 + jj) & ((1 << c.ps_log2) - 1)), i = tid, g = i >> 5;
                const int n = (i >> 4) & (L::VN - 1);
                const int code = (blk[L::v_piece(p, D == 64 ? 0 : i >> 7, i & 15) + (n >> 1)] >> (4 * (n & 1))) & 15;
                const float d = (float)reinterpret_cast<const _Float16 *>(blk + L::d_off(c.ps_log2))[L::by4(p, g)];
                const float mm = (float)reinterpret_cast<const _Float16 *>(blk + L::m_off(c.ps_log2))[L::by4(p, g)];
                o = fmaf(sc[jj], fmaf((float)code, d, mm), o);
            }
        }
        __syncthreads();
    }
    if (tid < D) {
        const float y = l > 0.f || l != l ? o / l : 0.f;
        const int64_t i = t * out.row + h * out.head + tid * out.elem;
        if (out.f16) reinterpret_cast<_Float16 *>(out.p)[i] = (_Float16)y;
        else reinterpret_cast<float *>(out.p)[i] = y;
    }
}

}  // namespace

int64_t kv_attn_workspace(const KvCache &, const KvSeqs &, int) { return 0; }

hipError_t launch_kv_attn(const KvCache &c, const KvSeqs &seqs, int hq, const Heads &q, const Heads &out, float scale,
                          int window, void *, hipStream_t st) {
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)seqs.rows * hq), dim3(256), 0, st, c, seqs, hq, q, out, scale, window);
    };
    if (c.D == 64) go(kv_attn_simple_kernel<64>);
    else if (c.D == 128) go(kv_attn_simple_kernel<128>);
    else go(kv_attn_simple_kernel<256>);
    return hipGetLastError();
}

}  // namespace qk
