// qk_delta.hip -- the gated delta recurrence, row after row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qk_delta.h"

namespace qk {
namespace delta {

constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int R = 16;  // rows made ready at once: 16 lanes each

// A short row over 16 lanes, enlarged, and the factor that brings it to length 1
// (rows of zeros stay zeros without an eps too).
template <int P> __device__ __forceinline__ float to_length_1(float (*x)[4], float xx, float eps) {
    if (eps >= 0x1p-74f) {  // (with 2^100 below it would leave fp32)
        enlarge<P>(x, 0x1p60f);
        return rsqrtf(xx + eps) * 0x1p-60f;
    }
    const float s = sum16(enlarge<P>(x, 0x1p100f)) + eps * 0x1p100f * 0x1p100f;
    return s > 0.f ? rsqrtf(s) : 0.f;
}

// The state of a head is held as S[Dv][Dk]: a column (one value dimension) is
// 16 lanes with DK / 16 values each, a lane has CPL columns.  With the old
// state S, a row is
//   d = S k, e = S q (together),  u = beta (v - a d),  o = a e + u (k.q),  S <- a S + u k
// so that only one sum over lanes lies between a state and the next one.  What
// does not depend on the state -- normed queries and keys, k.q, gates -- is
// made ready for R rows at once, a row to 16 lanes, and waits in LDS.
// One token of 48 heads of 128 x 128 (6.4 MB of state read and written) is 5.6 us,
// latency; 64 sequences (407 MB) 85-88 us, 4.6-4.8 TB/s: memory (70 in place: the
// states stay in the Infinity Cache).  Of many rows
// each takes 0.35 us, the chain from state to state.
template <int DK, int CPL> __global__ void __launch_bounds__(THREADS) delta_rows_kernel(Args a) {
    constexpr int P = DK / 64;                 // pieces of 4 dimensions a lane has
    constexpr int COLS = 4 * WAVES * CPL;      // columns of a block
    __shared__ float4 q_s[R][P][16], k_s[R][P][16];
    __shared__ float v_s[R][COLS], o_s[R][COLS];
    __shared__ float4 g_s[R];                  // decay, step, k.q
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15;
    const int per_head = a.dv / COLS;
    const int64_t b = blockIdx.x;
    const int s = (int)(b / ((int64_t)per_head * a.hv)), hb = (int)(b % ((int64_t)per_head * a.hv));
    const int h = hb / per_head, hk = h / a.rep, c0 = (hb % per_head) * COLS;
    const int col = (tid >> 6) * 4 * CPL + (lane >> 4);  // of the block; the lane's others are 4 apart
    const SeqState sq = seq_state(a.q, s);
    const int n = a.out.p ? sq.n : sq.commit;
    if (n == 0) return;
    const int64_t cell = ((int64_t)h * a.dv + c0 + col) * DK + 4 * l, slot = (int64_t)a.hv * a.dv * DK;
    float S[CPL][P][4];
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float4 f = make_float4(0, 0, 0, 0);
            if (sq.src >= 0) f = *reinterpret_cast<const float4 *>(a.pool + sq.src * slot + cell + 4 * c * DK + 64 * p);
            S[c][p][0] = f.x; S[c][p][1] = f.y; S[c][p][2] = f.z; S[c][p][3] = f.w;
        }
    const int r = tid >> 4;  // the row that this thread's 16 lanes make ready
    for (int i0 = 0; i0 < n; i0 += R) {
        const int m = min(R, n - i0);
        if (r < m) {
            const int t = sq.first + i0 + r;
            float q[P][4], k[P][4], v[COLS / 16];
            load_pieces<P, 64>(a.q_vec, a.qh, t, hk, 4 * l, q);
            load_pieces<P, 64>(a.k_vec, a.kh, t, hk, 4 * l, k);
#pragma unroll
            for (int c = 0; c < COLS / 16; ++c) v[c] = load1(a.vh, t, h, c0 + l + 16 * c);
            const float al = load1(a.alpha, t, h, 0), be = load1(a.beta, t, h, 0);
            float qq = 0, kk = 0, kq = 0;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    qq = fmaf(q[p][x], q[p][x], qq);
                    kk = fmaf(k[p][x], k[p][x], kk);
                    kq = fmaf(k[p][x], q[p][x], kq);
                }
            qq = sum16(qq); kk = sum16(kk); kq = sum16(kq);
            float rq = a.norm ? a.scale * rsqrtf(qq + a.eps) : a.scale, rk = a.norm ? rsqrtf(kk + a.eps) : 1.f;
            float both = kq * rq * rk;
            if (a.norm && (qq < SHORT || kk < SHORT)) {  // (alike for the row's 16 lanes)
                if (qq < SHORT) rq = a.scale * to_length_1<P>(q, qq, a.eps);
                if (kk < SHORT) rk = to_length_1<P>(k, kk, a.eps);
                kq = 0;
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int x = 0; x < 4; ++x) kq = fmaf(k[p][x], q[p][x], kq);
                both = sum16(kq) * (rq * rk);
            }
            const Gate g = gates(a, h, al, be);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                q_s[r][p][l] = make_float4(q[p][0] * rq, q[p][1] * rq, q[p][2] * rq, q[p][3] * rq);
                k_s[r][p][l] = make_float4(k[p][0] * rk, k[p][1] * rk, k[p][2] * rk, k[p][3] * rk);
            }
#pragma unroll
            for (int c = 0; c < COLS / 16; ++c) v_s[r][l + 16 * c] = v[c];
            if (l == 0) g_s[r] = make_float4(expf(g.g), g.b, both, 0);
        }
        __syncthreads();
        // with one column a lane a row's numbers come from LDS while the row before is worked on
        struct Now {
            float4 q[P], k[P], g;
            float v[CPL];
        };
        auto read = [&](int i, Now &r) {
            r.g = g_s[i];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                r.q[p] = q_s[i][p][l];
                r.k[p] = k_s[i][p][l];
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c) r.v[c] = v_s[i][col + 4 * c];
        };
        auto step = [&](int i, const Now &r) {
            const float4 g = r.g, *q = r.q, *k = r.k;
            float d[CPL], e[CPL];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                float d1 = k[0].z * S[c][0][2], e1 = q[0].z * S[c][0][2];
                d[c] = k[0].x * S[c][0][0];
                e[c] = q[0].x * S[c][0][0];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (p) {
                        d[c] = fmaf(k[p].x, S[c][p][0], d[c]); e[c] = fmaf(q[p].x, S[c][p][0], e[c]);
                        d1 = fmaf(k[p].z, S[c][p][2], d1);     e1 = fmaf(q[p].z, S[c][p][2], e1);
                    }
                    d[c] = fmaf(k[p].y, S[c][p][1], d[c]); e[c] = fmaf(q[p].y, S[c][p][1], e[c]);
                    d1 = fmaf(k[p].w, S[c][p][3], d1);     e1 = fmaf(q[p].w, S[c][p][3], e1);
                }
                d[c] += d1;
                e[c] += e1;
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                d[c] = sum16(d[c]);
                e[c] = sum16(e[c]);
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float u = g.y * fmaf(-g.x, d[c], r.v[c]);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    S[c][p][0] = fmaf(k[p].x, u, g.x * S[c][p][0]);
                    S[c][p][1] = fmaf(k[p].y, u, g.x * S[c][p][1]);
                    S[c][p][2] = fmaf(k[p].z, u, g.x * S[c][p][2]);
                    S[c][p][3] = fmaf(k[p].w, u, g.x * S[c][p][3]);
                }
                if (l == 0) o_s[i][col + 4 * c] = fmaf(u, g.z, g.x * e[c]);
            }
            if (i0 + i + 1 == sq.commit) {
#pragma unroll
                for (int c = 0; c < CPL; ++c)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        *reinterpret_cast<float4 *>(a.pool + sq.dst * slot + cell + 4 * c * DK + 64 * p) =
                            make_float4(S[c][p][0], S[c][p][1], S[c][p][2], S[c][p][3]);
            }
        };
        if constexpr (CPL == 1) {
            Now even, odd;
            read(0, even);
            for (int i = 0; i < m; i += 2) {
                read(min(i + 1, m - 1), odd);
                step(i, even);
                if (i + 1 >= m) break;
                read(min(i + 2, m - 1), even);
                step(i + 1, odd);
            }
        } else {  // (registers for more waves instead: 32 sequences of 32 rows 135 us, 155 with the next row's numbers ahead)
            for (int i = 0; i < m; ++i) {
                Now now;
                read(i, now);
                step(i, now);
            }
        }
        __syncthreads();
        if (a.out.p && r < m) {
#pragma unroll
            for (int c = 0; c < COLS / 16; ++c) store1(a.out, sq.first + i0 + r, h, c0 + l + 16 * c, o_s[r][l + 16 * c]);
        }
    }
}

template <int DK, int CPL> hipError_t go(const Args &a, int nseq, hipStream_t st) {
    const int64_t blocks = (int64_t)nseq * a.hv * (a.dv / (4 * WAVES * CPL));
    hipLaunchKernelGGL((delta_rows_kernel<DK, CPL>), dim3((unsigned)blocks), dim3(THREADS), 0, st, a);
    return hipGetLastError();
}

}  // namespace delta

// Long sequences go in tiles of 64 rows on matrix cores (16 key and 48 value
// heads of 128 x 128, in a graph; rows / tiles: 1 sequence of 64 rows 25 / 34 us, of
// 128 47 / 37, of 256 91 / 44; 8 of 64 95 / 74; 32 of 64 248 / 270, of 128 479 /
// 383).  Where lengths differ they may be all in one sequence, which takes
// 0.35 us a row one by one, while tiles lose less than half at 32 rows each.  (The
// count of sequences and heads says more than rows do: 8 of 64 rows lose by this
// rule, as does one long sequence among many of few rows.)
// Rows brought to length 1 and steps in 0..1 keep what a tile's inverse holds in
// fp16's range: others go row by row.
static bool in_tiles(const StateSeqs &q, bool norm, bool raw) { return norm && raw && q.rows / q.nseq >= (q.q_start ? 32 : 80); }

int64_t delta_workspace(const StateSeqs &q, const DeltaState &d, bool norm, bool raw) {
    return in_tiles(q, norm, raw) ? delta_chunk_workspace(q, d) : 0;
}

hipError_t launch_delta(const StateSeqs &q, const DeltaState &d, const DeltaIn &in, const Heads &out, void *workspace,
                        hipStream_t st) {
    using namespace delta;
    const Args a = make_args(q, d, in, out);
    if (in_tiles(q, in.norm, in.A)) return launch_delta_chunk(a, d.hk, d.dk, workspace, st);
    // A lane's columns: more as soon as that leaves 2 blocks a CU, since what is made ready a row then
    // serves more of them; 4 of many rows, whose chain more waves hide, from 4 blocks on.  1 / 2 / 4
    // columns, 48 heads of 128 x 128, in place: 2 sequences of 1 token 6.1 / 6.0 / 6.2 us, 3 8.5 / 6.8 / 7.1,
    // 8 14.6 / 11.0 / 9.3, 64 84 / 70 / 70 (from other slots 105 / 84 / 85); 2 of 17 rows 12.6 / 13.6 / 15.9,
    // 3 18.2 / 16.5 / 19.8, 12 46.7 / 39.1 / 41.9, 16 64.7 / 51.4 / 50.6.
    const int64_t columns = (int64_t)q.nseq * d.hv * d.dv, many = q.rows > 8 * (int64_t)q.nseq ? 4 : 2;
    const int cpl = d.dv % 64 == 0 && columns >= 64 * many * device_cus() ? 4 : columns >= 32 * 2 * device_cus() ? 2 : 1;
    if (d.dk == 64) return cpl == 4 ? go<64, 4>(a, q.nseq, st) : cpl == 2 ? go<64, 2>(a, q.nseq, st) : go<64, 1>(a, q.nseq, st);
    return cpl == 4 ? go<128, 4>(a, q.nseq, st) : cpl == 2 ? go<128, 2>(a, q.nseq, st) : go<128, 1>(a, q.nseq, st);
}

}  // namespace qk
