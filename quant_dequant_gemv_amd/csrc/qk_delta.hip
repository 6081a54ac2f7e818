// qk_delta.hip -- the gated delta recurrence, row after row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qk_delta.h"

namespace qk {
namespace delta {

constexpr int WAVES = 4;
constexpr int COLS = 4;  // columns of the state a wave has: 16 lanes each

// v of the lane `CTRL` away inside a row of 16 lanes
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float v) {
    v += dpp<0xB1>(v);   // quad_perm [1,0,3,2]
    v += dpp<0x4E>(v);   // quad_perm [2,3,0,1]
    v += dpp<0x141>(v);  // half row mirrored
    v += dpp<0x140>(v);  // row mirrored
    return v;
}

// The state of a head is held as S[Dv][Dk]: a column j (one value dimension)
// is 16 lanes with DK / 16 values each.  With the old state S, a row is
//   d = S k, e = S q (together),  u = beta (v - a d),  o = scale (a e + u (k.q)),  S <- a S + u k
// so that only one sum over lanes lies between a state and the next one.
template <int DK> __global__ void __launch_bounds__(64 * WAVES) delta_rows_kernel(Args a) {
    constexpr int P = DK / 64;  // pieces of 4 dimensions a lane has
    const int lane = threadIdx.x & 63, l = lane & 15;
    const int per_head = a.dv / (COLS * WAVES);
    const int64_t b = blockIdx.x;
    const int s = (int)(b / ((int64_t)per_head * a.hv)), hb = (int)(b % ((int64_t)per_head * a.hv));
    const int h = hb / per_head, hk = h / a.rep;
    const int col = (hb % per_head) * (COLS * WAVES) + (threadIdx.x >> 6) * COLS + (lane >> 4);
    const SeqState sq = seq_state(a.q, s);
    const int n = a.out.p ? sq.n : sq.commit;
    if (n == 0) return;
    const int64_t cell = ((int64_t)h * a.dv + col) * DK, slot = (int64_t)a.hv * a.dv * DK;
    float S[P][4];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float4 f = make_float4(0, 0, 0, 0);
        if (sq.src >= 0) f = *reinterpret_cast<const float4 *>(a.pool + sq.src * slot + cell + 64 * p + 4 * l);
        S[p][0] = f.x; S[p][1] = f.y; S[p][2] = f.z; S[p][3] = f.w;
    }
    struct Row { float q[P][4], k[P][4], v, al, be; };
    auto fetch = [&](int t, Row &r) {
        load_row<P>(a.kv_vec, a.qh, t, hk, l, r.q);
        load_row<P>(a.kv_vec, a.kh, t, hk, l, r.k);
        r.v = load1(a.vh, t, h, col);
        r.al = load1(a.alpha, t, h, 0);
        r.be = load1(a.beta, t, h, 0);
    };
    Row cur, nxt;
    fetch(sq.first, cur);
    for (int i = 0; i < n; ++i) {
        const int t = sq.first + i;
        if (i + 1 < n) fetch(t + 1, nxt);
        float qq = 0, kk = 0, kq = 0, d = 0, e = 0;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                qq = fmaf(cur.q[p][x], cur.q[p][x], qq);
                kk = fmaf(cur.k[p][x], cur.k[p][x], kk);
                kq = fmaf(cur.k[p][x], cur.q[p][x], kq);
                d = fmaf(cur.k[p][x], S[p][x], d);
                e = fmaf(cur.q[p][x], S[p][x], e);
            }
        qq = sum16(qq); kk = sum16(kk); kq = sum16(kq); d = sum16(d); e = sum16(e);
        float rq = a.scale, rk = 1.f;
        if (a.norm) {
            rq *= rsqrtf(qq + a.eps);
            rk = rsqrtf(kk + a.eps);
        }
        const Gate g = gates(a, h, cur.al, cur.be);
        const float decay = expf(g.g);
        const float u = g.b * (cur.v - decay * (d * rk));
        const float o = rq * fmaf(u * rk, kq, decay * e);
        const float uk = u * rk;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[p][x] = fmaf(cur.k[p][x], uk, decay * S[p][x]);
        if (a.out.p && l == 0) store1(a.out, t, h, col, o);
        if (i + 1 == sq.commit) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<float4 *>(a.pool + sq.dst * slot + cell + 64 * p + 4 * l) =
                    make_float4(S[p][0], S[p][1], S[p][2], S[p][3]);
        }
        cur = nxt;
    }
}

}  // namespace delta

int64_t delta_workspace(const StateSeqs &, const DeltaState &) { return 0; }

hipError_t launch_delta(const StateSeqs &q, const DeltaState &d, const DeltaIn &in, const Heads &out, void *,
                        hipStream_t st) {
    using namespace delta;
    const Args a = make_args(q, d, in, out);
    const int64_t blocks = (int64_t)q.nseq * d.hv * (d.dv / (COLS * WAVES));
    if (d.dk == 64) hipLaunchKernelGGL(delta_rows_kernel<64>, dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, a);
    else hipLaunchKernelGGL(delta_rows_kernel<128>, dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, a);
    return hipGetLastError();
}

}  // namespace qk
