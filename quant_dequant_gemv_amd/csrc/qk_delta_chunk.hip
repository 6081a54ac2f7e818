// qk_delta_chunk.hip -- the gated delta recurrence over long sequences: tiles
// of 64 rows on matrix cores.
//
// With G_t the sum of the log decays from a tile's first row through row t, S0
// the state before it, k^ and q^ of length 1 and c, e the rows' lengths, the
// rows of a tile solve
//   (I + L) U = b (V - e^G c (K^ S0)),      L_tj = b_t c_t c_j e^(G_t - G_j) k^_t.k^_j   (j < t)
//   O = scale (e^G e (Q^ S0) + A U),         A_tj = e_t c_j e^(G_t - G_j) q^_t.k^_j       (j <= t)
//   S = e^G_last S0 + K^T (e^(G_last - G) c U)
// What does not depend on the state -- T = (I + L)^-1 b, A, the rows brought to
// length 1 -- is made for all tiles at once (delta_tile_kernel); then a block
// takes 32 columns of a head's state through its sequence's tiles, the state in
// registers all the way (delta_scan_kernel).
//
// Matrix instructions take fp16, so every factor is a sum of two fp16 values
// (22 bits) and every product three instructions; the fp32 factors that change
// from tile to tile (state, U) are scaled by a power of two a column first, and
// what is at most 1 by 2^10 (rows) or 2^14 (T, A: their small values count).
// Sums, states, decays (their differences in fp64) and the inverse are fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "qk_delta.h"

namespace qk {
namespace delta {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int C = 64;             // rows of a tile
constexpr int FRAG = 512;         // halves of a matrix operand: 64 lanes x 8
constexpr int TRI = 6;            // operands of a lower triangle of 4 x 2 (row tile, 32 columns)
constexpr int N = 32;             // columns of a scan block
constexpr float ROW_UNIT = 1024.f, TRI_UNIT = 16384.f;

// A matrix operand's lane has row (or column) lane & 15 and, with g = lane >>
// 4, the 8 places 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3 of the 32 that are
// summed over: what two results of the instruction hold, so that a result is
// the next product's operand as it stands.
constexpr int tri_index(int row, int k) { return row < 2 ? row : row == 2 ? 2 + k : 4 + k; }

struct Chunks {
    _Float16 *rows;   // [tiles][hk][3][...]: K^, Q^ by rows, K^ by dimensions
    _Float16 *tri;    // [tiles][hv][2][TRI][2][FRAG]: T, A
    float *vec;       // [tiles][hv][256]: e^G c, e^G e, e^(G_last - G) c, e^G_last
    float *carry;     // [2][hv][dv][DK]: states between two launches
    int first, count; // tiles of this launch
    int turn;         // of `carry`
};

template <int DK> struct Sizes {
    static constexpr int KB = DK / 32;
    static constexpr int PART = 4 * KB * 2 * FRAG;  // halves of K^ (Q^, K^ by dimensions) of a tile
};

// Tiles are numbered from first_tile(s) on for sequence s; one ends where the
// state is kept, so a sequence of n rows has at most n / 64 + 2.
__device__ __forceinline__ int first_tile(const StateSeqs &q, int s) {
    const int r = q.q_start ? min(max(q.q_start[s], 0), q.rows) : s * (q.rows / q.nseq);
    return r / C + 2 * s;
}
struct Span { int before, count, n; };  // tiles up to where the state is kept, all tiles, rows worked on
__device__ __forceinline__ Span span_of(const SeqState &s, bool out) {
    const int n = out ? s.n : s.commit, before = (s.commit + C - 1) / C;
    return {before, before + (n - s.commit + C - 1) / C, n};
}
__device__ __forceinline__ int tile_row(const SeqState &s, const Span &p, int j) {
    return j < p.before ? C * j : s.commit + C * (j - p.before);
}
__device__ __forceinline__ int tile_end(const SeqState &s, const Span &p, int j) {
    return j < p.before ? min(C * j + C, s.commit) : min(s.commit + C * (j - p.before) + C, p.n);
}

__device__ __forceinline__ f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
// c + (ah + al)(bh + bl) without the product of the two small parts
__device__ __forceinline__ f4 mma3(h8 ah, h8 al, h8 bh, h8 bl, f4 c) {
    c = mma(al, bh, c);
    c = mma(ah, bl, c);
    return mma(ah, bh, c);
}

// Results that are read behind a branch: the wait states that a matrix
// instruction's result needs are kept here, in the block that made it (the
// compiler has left them out where blocks meet: the last register of a result
// was then read before it was written).
template <int M> __device__ __forceinline__ void settle(f4 (&c)[M]) {
#pragma unroll
    for (int i = 0; i < M; ++i) asm volatile("" : "+v"(c[i]));
    asm volatile("s_nop 15\n\ts_nop 7" : "+v"(c[0]), "+v"(c[M - 1]));
#pragma unroll
    for (int i = 0; i < M; ++i) asm volatile("" : "+v"(c[i]));
}

// c[i] += (a_i in two parts) (b in two parts), operand a_i at a(i): the M
// results take turns, so no instruction waits for the one before it.
template <int M, typename F> __device__ __forceinline__ void mma3_all(F a, h8 bh, h8 bl, f4 *c) {
    h8 ah[M], al[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        ah[i] = a(2 * i);
        al[i] = a(2 * i + 1);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) c[i] = mma(al[i], bh, c[i]);
#pragma unroll
    for (int i = 0; i < M; ++i) c[i] = mma(ah[i], bl, c[i]);
#pragma unroll
    for (int i = 0; i < M; ++i) c[i] = mma(ah[i], bh, c[i]);
}

__device__ __forceinline__ void split(float x, _Float16 &hi, _Float16 &lo) {
    hi = (_Float16)x;
    lo = (_Float16)(x - (float)hi);
}
// Two results of 4 as an operand in two parts.
__device__ __forceinline__ void split8(f4 a, f4 b, float s, h8 &hi, h8 &lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        _Float16 h, l;
        split(a[i] * s, h, l);
        hi[i] = h;
        lo[i] = l;
        split(b[i] * s, h, l);
        hi[i + 4] = h;
        lo[i + 4] = l;
    }
}
// The power of two that brings a column's largest value (over the four lanes
// that have it) to 2^14 .. 2^15, and its inverse.
struct Unit { float up, down; };
__device__ __forceinline__ Unit unit_of(float m) {
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const int e = min(max((int)(__builtin_bit_cast(uint32_t, m) >> 23), 32), 254);  // exponent + 127
    return {__builtin_bit_cast(float, (uint32_t)(268 - e) << 23), __builtin_bit_cast(float, (uint32_t)(e - 14) << 23)};
}

// ------------------------------------------------------------------ tiles

constexpr int TILE_THREADS = 256;

// One tile of a key head, and of each of its value heads.  Wave w has the rows
// 16 w .. 16 w + 15 of everything.
template <int DK> __global__ void __launch_bounds__(TILE_THREADS) delta_tile_kernel(Args a, Chunks ck) {
    constexpr int KB = DK / 32, PITCH = DK + 8, Q4 = DK / 16;
    using Z = Sizes<DK>;
    __shared__ _Float16 rows_s[4][C][PITCH];  // K^ and Q^, each in two parts; then L and the inverse's blocks
    __shared__ double G_s[C];
    __shared__ float c_s[C], e_s[C], b_s[C];
    float(*L)[C + 4] = reinterpret_cast<float(*)[C + 4]>(&rows_s[0][0][0]);
    float(*D)[16][20] = reinterpret_cast<float(*)[16][20]>(&L[C][0]);
    static_assert(sizeof(float) * (C * (C + 4) + 4 * 16 * 20) <= sizeof(rows_s), "L and the diagonal blocks in the rows' place");
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, g = lane >> 4;
    const int hk_n = a.hv / a.rep, local = blockIdx.x / hk_n, hk = blockIdx.x % hk_n, id = ck.first + local;
    const int s = __builtin_amdgcn_readfirstlane(count_while(a.q.nseq, lane, [&](int i) { return first_tile(a.q, i) <= id; })) - 1;
    if (s < 0) return;
    const SeqState sq = seq_state(a.q, s);
    const Span sp = span_of(sq, a.out.p != nullptr);
    const int j = id - first_tile(a.q, s);
    if (j < 0 || j >= sp.count) return;
    const int r0 = tile_row(sq, sp, j), n = tile_end(sq, sp, j) - r0;

    // Rows: a quarter of a row to a thread.
    {
        const int r = tid >> 2, l = tid & 3;
        float q[Q4][4], k[Q4][4];
        float qq = 0, kk = 0;
#pragma unroll
        for (int p = 0; p < Q4; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[p][e] = k[p][e] = 0;
        if (r < n) {
            const int64_t t = sq.first + r0 + r;
            load_pieces<Q4, 16>(a.q_vec, a.qh, t, hk, 4 * l, q);
            load_pieces<Q4, 16>(a.k_vec, a.kh, t, hk, 4 * l, k);
        }
#pragma unroll
        for (int p = 0; p < Q4; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                qq = fmaf(q[p][e], q[p][e], qq);
                kk = fmaf(k[p][e], k[p][e], kk);
            }
        qq += dpp<0xB1>(qq); kk += dpp<0xB1>(kk);
        qq += dpp<0x4E>(qq); kk += dpp<0x4E>(kk);
        const float rq = qq > 0.f ? rsqrtf(qq) : 0.f, rk = kk > 0.f ? rsqrtf(kk) : 0.f;
        if (l == 0) {
            c_s[r] = kk * rk * rsqrtf(kk + a.eps);
            e_s[r] = qq * rq * rsqrtf(qq + a.eps);
            if (!(kk > 0.f)) c_s[r] = kk;  // (0, or NaN)
            if (!(qq > 0.f)) e_s[r] = qq;
        }
#pragma unroll
        for (int p = 0; p < Q4; ++p) {
            h4 hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                _Float16 h, m;
                split(k[p][e] * rk * ROW_UNIT, h, m);
                hi[0][e] = h;
                lo[0][e] = m;
                split(q[p][e] * rq * ROW_UNIT, h, m);
                hi[1][e] = h;
                lo[1][e] = m;
            }
            *reinterpret_cast<h4 *>(&rows_s[0][r][16 * p + 4 * l]) = hi[0];
            *reinterpret_cast<h4 *>(&rows_s[1][r][16 * p + 4 * l]) = lo[0];
            *reinterpret_cast<h4 *>(&rows_s[2][r][16 * p + 4 * l]) = hi[1];
            *reinterpret_cast<h4 *>(&rows_s[3][r][16 * p + 4 * l]) = lo[1];
        }
    }
    __syncthreads();

    // Operands to memory, and the products k^_j.k^_t and k^_j.q^_t: rows j =
    // 16 i + 4 g + r, columns t = 16 w + x.
    f4 kk[4], kq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[i] = kq[i] = f4{0, 0, 0, 0};
    _Float16 *out = ck.rows + ((int64_t)local * hk_n + hk) * 3 * Z::PART;
    auto part = [&](int plane, int row, int kb) {
        const h4 u = *reinterpret_cast<const h4 *>(&rows_s[plane][row][32 * kb + 4 * g]);
        const h4 v = *reinterpret_cast<const h4 *>(&rows_s[plane][row][32 * kb + 16 + 4 * g]);
        return h8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
    };
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const h8 kh = part(0, 16 * w + x, kb), kl = part(1, 16 * w + x, kb);
        const h8 qh = part(2, 16 * w + x, kb), ql = part(3, 16 * w + x, kb);
        h8 *o = reinterpret_cast<h8 *>(out + (w * KB + kb) * 2 * FRAG) + lane;
        o[0] = kh;
        o[64] = kl;
        o = reinterpret_cast<h8 *>(out + Z::PART + (w * KB + kb) * 2 * FRAG) + lane;
        o[0] = qh;
        o[64] = ql;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (those above the diagonal too: no branches around matrix instructions)
            const h8 ah = part(0, 16 * i + x, kb), al = part(1, 16 * i + x, kb);
            kk[i] = mma3(ah, al, kh, kl, kk[i]);
            kq[i] = mma3(ah, al, qh, ql, kq[i]);
        }
    }
    settle(kk);
    settle(kq);
#pragma unroll
    for (int i = 0; i < DK / 64; ++i) {  // K^ by dimensions: rows 16 d + x
        const int d = w * (DK / 64) + i;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                h8 v;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = rows_s[p][32 * kb + 16 * (e >> 2) + 4 * g + (e & 3)][16 * d + x];
                reinterpret_cast<h8 *>(out + 2 * Z::PART + ((d * 2 + kb) * 2 + p) * FRAG)[lane] = v;
            }
    }

    const int tl = 16 * w + x;  // the lane's row t
    for (int v = 0; v < a.rep; ++v) {
        const int h = hk * a.rep + v;
        __syncthreads();  // rows_s, and the last head's L and gates, are done with
        if (w == 0) {
            double G = 0;
            float b = 0;
            if (lane < n) {
                const int64_t t = sq.first + r0 + lane;
                const Gate gt = gates(a, h, load1(a.alpha, t, h, 0), load1(a.beta, t, h, 0));
                G = fmax((double)gt.g, -1e4);  // (e^-1e4 is 0 too)
                if (gt.g != gt.g) G = gt.g;
                b = gt.b;
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const double up = __shfl_up(G, d);
                if (lane >= d) G += up;
            }
            G_s[lane] = G;
            b_s[lane] = b;
            const double last = __shfl(G, 63);
            float *o = ck.vec + ((int64_t)local * a.hv + h) * 256;
            const float eg = expf((float)G);
            o[lane] = eg * c_s[lane];
            o[64 + lane] = eg * e_s[lane];
            o[128 + lane] = expf((float)(last - G)) * c_s[lane];
            if (lane == 0) o[192] = expf((float)last);
        }
        __syncthreads();
        f4 At[4];
        const double Gt = G_s[tl];
        const float bt = b_s[tl], ct = c_s[tl], et = e_s[tl];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int jl = 16 * i + 4 * g + r;
                const float d = jl <= tl ? expf((float)(Gt - G_s[jl])) * c_s[jl] : 0.f;
                At[i][r] = d * et * kq[i][r] * (TRI_UNIT / (ROW_UNIT * ROW_UNIT));
                L[tl][jl] = jl < tl ? d * (bt * ct) * kk[i][r] * (1.f / (ROW_UNIT * ROW_UNIT)) : 0.f;
            }
        }
        __syncthreads();
        // Diagonal block w: its inverse, column x to a lane (the four of equal x do the same).
        {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float sum = i == x ? 1.f : 0.f;
#pragma unroll
                for (int m = 0; m < i; ++m) sum = fmaf(-L[16 * w + i][16 * w + m], z[m], sum);
                z[i] = sum;
            }
            if (g == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) D[w][i][x] = z[i];
            }
        }
        __syncthreads();
        // Rows of the inverse, transposed (rows j, columns t): T_wi^T = -T_ii^T sum_{m = i+1..w} L_mi^T T_wm^T, from i = w down.
        // (T_wi = 0 for i > w comes of itself)
        f4 T[4];
        const f4 own = *reinterpret_cast<const f4 *>(&D[w][x][4 * g]);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            f4 sum = f4{0, 0, 0, 0};
            T[i] = f4{0, 0, 0, 0};
#pragma unroll
            for (int m = i + 1; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sum = __builtin_amdgcn_mfma_f32_16x16x4f32(L[16 * m + 4 * g + r][16 * i + x], T[m][r], sum, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) T[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(-D[i][4 * g + r][x], sum[r], T[i], 0, 0, 0);
            settle(reinterpret_cast<f4(&)[1]>(T[i]));
#pragma unroll
            for (int r = 0; r < 4; ++r) T[i][r] = i == w ? own[r] : T[i][r];
        }
        _Float16 *to = ck.tri + ((int64_t)local * a.hv + h) * (2 * TRI * 2 * FRAG);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (2 * kb > w) continue;
            f4 t0, t1;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                t0[r] = T[2 * kb][r] * b_s[32 * kb + 4 * g + r];
                t1[r] = T[2 * kb + 1][r] * b_s[32 * kb + 16 + 4 * g + r];
            }
            h8 hi, lo;
            h8 *o = reinterpret_cast<h8 *>(to + tri_index(w, kb) * 2 * FRAG) + lane;
            split8(t0, t1, TRI_UNIT, hi, lo);
            o[0] = hi;
            o[64] = lo;
            o = reinterpret_cast<h8 *>(to + (TRI + tri_index(w, kb)) * 2 * FRAG) + lane;
            split8(At[2 * kb], At[2 * kb + 1], 1.f, hi, lo);
            o[0] = hi;
            o[64] = lo;
        }
    }
}

// ------------------------------------------------------------------ scan

constexpr int SCAN_WAVES = 6, LOADERS = 2;

// 16 bytes a lane from memory to LDS, the lanes' side by side from `to` on.
__device__ __forceinline__ void to_lds(const void *from, void *to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t *)from,
                                     (__attribute__((address_space(3))) uint32_t *)to, 16, 0, 0);
}

// N columns of a head's state through the tiles of a sequence.  Waves 0 and 1
// have 16 columns each: K^ S0 -> U -> the next state; waves 2 and 3 make the
// same columns' outputs from the states and U that those leave in LDS.  A tile
// is two phases with a barrier behind each; the operands of one phase come to
// LDS during the other, brought by waves 4 and 5 (a wave that brings them waits
// for them all at its next read of LDS).
template <int DK, typename V_T> __global__ void __launch_bounds__(64 * SCAN_WAVES) delta_scan_kernel(Args a, Chunks ck) {
    constexpr int KB = DK / 32, DT = DK / 16, PART = Sizes<DK>::PART;
    constexpr int PIECES = PART * 2 / 1024, TRI_PIECES = TRI * 2;  // of 1 KB
    extern __shared__ __align__(16) uint8_t lds[];
    _Float16 *K_s = reinterpret_cast<_Float16 *>(lds), *Q_s = K_s + PART, *KT_s = Q_s + PART, *T_s = KT_s + PART,
             *A_s = T_s + TRI * 2 * FRAG, *S_s = A_s + TRI * 2 * FRAG;   // S_s: [2][KB][2][FRAG]
    float *U_s = reinterpret_cast<float *>(S_s + 2 * KB * 2 * FRAG);     // [2][4][64][4]
    float *vec_s = U_s + 2 * 4 * 64 * 4;                                 // [2][256]
    float *unit_s = vec_s + 2 * 256;                                     // [2][16]: of the state's columns
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, g = lane >> 4;
    // blocks of one key head and sequence are 8 apart: on one XCD, whose L2 they share
    const int hk_n = a.hv / a.rep, slabs = a.dv / N, per = a.rep * slabs;
    const int64_t b = blockIdx.x, group = b % 8 + 8 * (b / (8 * per));
    if (group >= (int64_t)a.q.nseq * hk_n) return;
    const int member = (int)(b / 8 % per), s = (int)(group / hk_n), hk = (int)(group % hk_n), h = hk * a.rep + member / slabs;
    const int col = member % slabs * N + 16 * (w & 1) + x;
    const SeqState sq = seq_state(a.q, s);
    const Span sp = span_of(sq, a.out.p != nullptr);
    const int t0 = first_tile(a.q, s), j0 = max(ck.first - t0, 0), j1 = min(ck.first + ck.count - t0, sp.count);
    if (j0 >= j1) return;
    const bool chain = w < 2;
    const int64_t cell = ((int64_t)h * a.dv + col) * DK + 4 * g, slot = (int64_t)a.hv * a.dv * DK;

    // 1 KB pieces of an operand to LDS, wave after wave
    auto bring = [&](const _Float16 *from, _Float16 *to, int pieces) {
#pragma unroll
        for (int i = 0; i < pieces / LOADERS; ++i) {
            const int p = i * LOADERS + w - 4;
            to_lds(from + p * FRAG + lane * 8, to + p * FRAG);
        }
    };
    auto tile_rows = [&](int j) { return ck.rows + ((int64_t)(t0 + j - ck.first) * hk_n + hk) * 3 * PART; };
    auto tile_tri = [&](int j) { return ck.tri + ((int64_t)(t0 + j - ck.first) * a.hv + h) * (2 * TRI * 2 * FRAG); };
    auto bring_first = [&](int j) {
        bring(tile_rows(j), K_s, PIECES);
        bring(tile_rows(j) + PART, Q_s, PIECES);
        bring(tile_tri(j), T_s, TRI_PIECES);
        if (w == 4) to_lds(ck.vec + ((int64_t)(t0 + j - ck.first) * a.hv + h) * 256 + lane * 4, vec_s + (j & 1) * 256);
    };
    auto meet = [&]() {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __syncthreads();
    };
    auto frag = [&](const _Float16 *p, int i) { return reinterpret_cast<const h8 *>(p + i * FRAG)[lane]; };

    // a lower triangle of 64 x 64 times 64 rows
    auto triangle = [&](const _Float16 *p, const h8 *bh, const h8 *bl, f4(&c)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = f4{0, 0, 0, 0};
        mma3_all<4>([&](int i) { return frag(p, tri_index(i >> 1, 0) * 2 + (i & 1)); }, bh[0], bl[0], c);
        mma3_all<2>([&](int i) { return frag(p, tri_index(2 + (i >> 1), 1) * 2 + (i & 1)); }, bh[1], bl[1], c + 2);
    };

    f4 S[DT];
    h8 sh[KB], sl[KB];
    V_T raw[4][4];
    float down = 1.f;  // of the state's column
    auto part_state = [&]() {  // the state in two parts, for both waves of the columns
        float m = 0;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(S[i][r]));
        const Unit u = unit_of(m);
        down = u.down;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            split8(S[2 * kb], S[2 * kb + 1], u.up, sh[kb], sl[kb]);
            h8 *o = reinterpret_cast<h8 *>(S_s + (w * KB + kb) * 2 * FRAG) + lane;
            o[0] = sh[kb];
            o[64] = sl[kb];
        }
        if (g == 0) unit_s[w * 16 + x] = down;
    };
    auto fetch = [&](int j) {  // values of tile j (those past its end: of its last row)
        const int r0 = tile_row(sq, sp, j), n = tile_end(sq, sp, j) - r0;
        const V_T *p = reinterpret_cast<const V_T *>(a.vh.p) + (int64_t)(sq.first + r0) * a.vh.row + h * a.vh.head + col * a.vh.elem;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) raw[i][r] = p[min(16 * i + 4 * g + r, n - 1) * a.vh.row];
    };
    auto leave = [&](float *p) {
#pragma unroll
        for (int i = 0; i < DT; ++i) *reinterpret_cast<f4 *>(p + 16 * i) = S[i];
    };

    if (w >= 4) {
        bring_first(j0);
        meet();
        for (int j = j0; j < j1; ++j) {
            bring(tile_rows(j) + 2 * PART, KT_s, PIECES);
            bring(tile_tri(j) + TRI * 2 * FRAG, A_s, TRI_PIECES);
            meet();
            if (j + 1 < j1) bring_first(j + 1);
            meet();
        }
        return;
    }
    if (chain) {
        const float *from = j0 > 0 ? ck.carry + (ck.turn ^ 1) * slot + cell : sq.src >= 0 ? a.pool + sq.src * slot + cell : nullptr;
#pragma unroll
        for (int i = 0; i < DT; ++i) S[i] = from ? *reinterpret_cast<const f4 *>(from + 16 * i) : f4{0, 0, 0, 0};
        fetch(j0);
        part_state();
    }
    meet();
    for (int j = j0; j < j1; ++j) {
        const float *vec = vec_s + (j & 1) * 256;
        f4 acc[4];
        if (chain || a.out.p) {  // K^ S0, or Q^ S0
            const _Float16 *X = chain ? K_s : Q_s;
            if (!chain) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    sh[kb] = frag(S_s, ((w - 2) * KB + kb) * 2);
                    sl[kb] = frag(S_s, ((w - 2) * KB + kb) * 2 + 1);
                }
                down = unit_s[(w - 2) * 16 + x];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = f4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                mma3_all<4>([&](int i) { return frag(X, ((i >> 1) * KB + kb) * 2 + (i & 1)); }, sh[kb], sl[kb], acc);
            settle(acc);
        }
        f4 U[4];
        if (chain) {
            const float f = -down * (1.f / ROW_UNIT);
            const int n = tile_end(sq, sp, j) - tile_row(sq, sp, j);
            float m = 0;
            f4 V[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f4 ge = *reinterpret_cast<const f4 *>(vec + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    V[i][r] = 16 * i + 4 * g + r < n ? fmaf(f * ge[r], acc[i][r], (float)raw[i][r]) : 0.f;
                    m = fmaxf(m, fabsf(V[i][r]));
                }
            }
            const Unit u = unit_of(m);
            h8 rh[2], rl[2];
            split8(V[0], V[1], u.up, rh[0], rl[0]);
            split8(V[2], V[3], u.up, rh[1], rl[1]);
            triangle(T_s, rh, rl, U);
            settle(U);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r) U[i][r] *= u.down * (1.f / TRI_UNIT);
                reinterpret_cast<f4 *>(U_s)[(w * 4 + i) * 64 + lane] = U[i];
            }
        }
        meet();
        if (chain) {
            if (j + 1 < j1) fetch(j + 1);
            float m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f4 de = *reinterpret_cast<const f4 *>(vec + 128 + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    U[i][r] *= de[r];
                    m = fmaxf(m, fabsf(U[i][r]));
                }
            }
            const Unit u = unit_of(m);
            h8 uh[2], ul[2];
            split8(U[0], U[1], u.up, uh[0], ul[0]);
            split8(U[2], U[3], u.up, uh[1], ul[1]);
            const float keep = vec[192], f = u.down * (1.f / ROW_UNIT);
            f4 add[DT];
#pragma unroll
            for (int i = 0; i < DT; ++i) add[i] = f4{0, 0, 0, 0};
#pragma unroll
            for (int i0 = 0; i0 < DT; i0 += 4)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    mma3_all<4>([&](int i) { return frag(KT_s, ((i0 + (i >> 1)) * 2 + kb) * 2 + (i & 1)); }, uh[kb], ul[kb], add + i0);
            settle(add);
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] = fmaf(f, add[i][r], keep * S[i][r]);
            if (j + 1 == sp.before && sq.commit) leave(a.pool + sq.dst * slot + cell);
            if (j + 1 < j1) part_state();
        } else if (a.out.p) {
            float m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                U[i] = reinterpret_cast<const f4 *>(U_s)[((w - 2) * 4 + i) * 64 + lane];
#pragma unroll
                for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(U[i][r]));
            }
            const Unit u = unit_of(m);
            h8 uh[2], ul[2];
            split8(U[0], U[1], u.up, uh[0], ul[0]);
            split8(U[2], U[3], u.up, uh[1], ul[1]);
            const int r0 = tile_row(sq, sp, j), n = tile_end(sq, sp, j) - r0;
            const float f = a.scale * down * (1.f / ROW_UNIT), fu = a.scale * u.down * (1.f / TRI_UNIT);
            f4 o[4];
            triangle(A_s, uh, ul, o);
            settle(o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f4 we = *reinterpret_cast<const f4 *>(vec + 64 + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) o[i][r] = fmaf(f * we[r], acc[i][r], fu * o[i][r]);
            }
            const int64_t at = (sq.first + r0 + 4 * g) * a.out.row + h * a.out.head + col * a.out.elem;
            auto put = [&](auto *p) {
                p += at;
#pragma unroll
                for (int i = 0; i < 4; ++i, p += 12 * a.out.row)
#pragma unroll
                    for (int r = 0; r < 4; ++r, p += a.out.row)
                        if (16 * i + 4 * g + r < n) *p = (std::remove_reference_t<decltype(*p)>)o[i][r];
            };
            if (a.out.f16) put(reinterpret_cast<_Float16 *>(a.out.p));
            else put(reinterpret_cast<float *>(a.out.p));
        }
        meet();
    }
    if (chain && j1 < sp.count) leave(ck.carry + ck.turn * slot + cell);
}

template <int DK> constexpr int scan_lds() {
    return (3 * Sizes<DK>::PART + 2 * TRI * 2 * FRAG + 2 * (DK / 32) * 2 * FRAG) * 2 + (2 * 4 * 64 * 4 + 2 * 256 + 32) * 4;
}

template <int DK> int64_t tile_bytes(int hk, int hv) {
    return (int64_t)hk * 3 * Sizes<DK>::PART * 2 + (int64_t)hv * (2 * TRI * 2 * FRAG * 2 + 256 * 4);
}

// All tiles at once, or as many as have this much (a sequence's state is
// carried from one launch to the next).
constexpr int64_t CAP = (int64_t)256 << 20;

struct Plan { int tiles, each; int64_t bytes; };
Plan plan_of(const StateSeqs &q, int hk, int hv, int dk, int dv) {
    const int64_t one = dk == 64 ? tile_bytes<64>(hk, hv) : tile_bytes<128>(hk, hv);
    const int tiles = q.rows / C + 2 * q.nseq, each = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, CAP / one));
    return {tiles, each, each * one + (each < tiles ? 2 * (int64_t)hv * dv * dk * 4 : 0)};
}

template <int DK, typename V_T> hipError_t go(const Args &a, int hk, void *workspace, hipStream_t st) {
    const Plan pl = plan_of(a.q, hk, a.hv, DK, a.dv);
    const hipError_t e = lds_opt_in<delta_scan_kernel<DK, V_T>>(scan_lds<DK>());
    if (e != hipSuccess) return e;
    uint8_t *p = (uint8_t *)workspace;
    Chunks ck;
    ck.rows = (_Float16 *)p;
    p += (int64_t)pl.each * hk * 3 * Sizes<DK>::PART * 2;
    ck.tri = (_Float16 *)p;
    p += (int64_t)pl.each * a.hv * 2 * TRI * 2 * FRAG * 2;
    ck.vec = (float *)p;
    p += (int64_t)pl.each * a.hv * 256 * 4;
    ck.carry = (float *)p;
    const int64_t groups = ((int64_t)a.q.nseq * hk + 7) / 8 * 8;
    for (int first = 0, i = 0; first < pl.tiles; first += pl.each, ++i) {
        ck.first = first;
        ck.count = std::min(pl.each, pl.tiles - first);
        ck.turn = i & 1;
        hipLaunchKernelGGL(delta_tile_kernel<DK>, dim3((unsigned)((int64_t)ck.count * hk)), dim3(TILE_THREADS), 0, st, a, ck);
        hipLaunchKernelGGL((delta_scan_kernel<DK, V_T>), dim3((unsigned)(groups * a.rep * (a.dv / N))), dim3(64 * SCAN_WAVES), scan_lds<DK>(), st,
                           a, ck);
    }
    return hipGetLastError();
}

}  // namespace delta

int64_t delta_chunk_workspace(const StateSeqs &q, const DeltaState &d) { return delta::plan_of(q, d.hk, d.hv, d.dk, d.dv).bytes; }

hipError_t launch_delta_chunk(const delta::Args &a, int hk, int dk, void *workspace, hipStream_t st) {
    if (a.vh.f16) return dk == 64 ? delta::go<64, _Float16>(a, hk, workspace, st) : delta::go<128, _Float16>(a, hk, workspace, st);
    return dk == 64 ? delta::go<64, float>(a, hk, workspace, st) : delta::go<128, float>(a, hk, workspace, st);
}

}  // namespace qk
