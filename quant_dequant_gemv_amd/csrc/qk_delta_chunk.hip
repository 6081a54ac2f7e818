// qk_delta_chunk.hip -- the gated delta recurrence over long sequences: tiles
// of 64 rows on matrix cores.
//
// With G_t the sum of the log decays from a tile's first row through row t, S0
// the state before it, k^ and q^ of length 1 and c, e the rows' lengths, the
// rows of a tile solve
//   (I + L) U = b (V - e^G c (K^ S0)),      L_tj = b_t c_t c_j e^(G_t - G_j) k^_t.k^_j   (j < t)
//   O = scale e (e^G (Q^ S0) + A U),         A_tj = c_j e^(G_t - G_j) q^_t.k^_j           (j <= t)
//   S = e^G_last S0 + K^T (e^(G_last - G) c U)
// What does not depend on the state -- T = (I + L)^-1 b, A, the rows brought to
// length 1 -- is made for all tiles at once (delta_tile_kernel); then a block
// takes 32 columns of a head's state through its sequence's tiles, the state in
// registers all the way (delta_scan_kernel).
//
// 4096 rows of one sequence, 48 heads on 16 of 128 x 128: 267 us.  The tiles are
// 70-75 of it (171 MB written, 79 read: memory, at 2 waves a SIMD); the scan
// 185-210, 64 tiles one after another at 3 us, held by the latency of the chain
// state - R - U - state (four matrix products and three hand-overs between waves
// through LDS): without its outputs it is as long, and matrix cores are busy 16%.
// A row one by one takes 0.35 us: 1430 us.
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
constexpr int VEC = 5 * C;        // fp32 numbers of a tile and head
constexpr float ROW_UNIT = 1024.f, TRI_UNIT = 16384.f;

// A matrix operand's lane has row (or column) lane & 15 and, with g = lane >>
// 4, the 8 places 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3 of the 32 that are
// summed over: what two results of the instruction hold, so that a result is
// the next product's operand as it stands.
constexpr int tri_index(int row, int k) { return row < 2 ? row : row == 2 ? 2 + k : 4 + k; }

struct Chunks {
    _Float16 *rows;   // [tiles][hk][3][...]: K^, Q^ by rows, K^ by dimensions
    _Float16 *tri;    // [tiles][hv][2][TRI][2][FRAG]: T, A
    float *vec;       // [tiles][hv][VEC]: e^G c, e^G, e^(G_last - G) c, e (64 each), e^G_last; behind it nothing is kept
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

// c[2 i + ct] += (a_i in two parts) (b_ct in two parts), without the product
// of the two small parts: M x 2 results that take turns, so no instruction
// waits for the one before it.
template <int M, typename F> __device__ __forceinline__ void mma3_grid(F a, const h8 *bh, const h8 *bl, f4 *c) {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) c[2 * i + ct] = mma(a(i, 1), bh[ct], c[2 * i + ct]);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) c[2 * i + ct] = mma(a(i, 0), bl[ct], c[2 * i + ct]);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) c[2 * i + ct] = mma(a(i, 0), bh[ct], c[2 * i + ct]);
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
__device__ __forceinline__ float most8(f4 a, f4 b) {
    float m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
    return m;
}
// The largest over the four lanes of equal lane & 15, of values >= 0 (whose
// bits are ordered as they are).
__device__ __forceinline__ float over_rows(float m) {
    const uint32_t b = __builtin_bit_cast(uint32_t, m);
    const auto p = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t c = max(p[0], p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return __builtin_bit_cast(float, max(q[0], q[1]));
}
// The power of two that brings values up to m (of its binade) below 2^15, and
// its inverse.
struct Unit { float up, down; };
__device__ __forceinline__ Unit unit_at(float m) {
    const int e = min(max((int)(__builtin_bit_cast(uint32_t, m) >> 23), 32), 248);  // exponent + 127
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
    if (j < 0 || j >= sp.count) return;  // (below 0: of starts that decrease)
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
        // a row's length over the root that it is divided by, its square as it is or 2^200 of it
        auto length = [&](float (*x)[4], float &xx) {
            if (!(xx < SHORT)) return xx * rsqrtf(xx) * rsqrtf(xx + a.eps);  // (NaN too)
            xx = enlarge<Q4>(x, 0x1p100f);
            xx += dpp<0xB1>(xx);
            xx += dpp<0x4E>(xx);
            return xx > 0.f ? (float)sqrt(xx / (xx + a.eps * 0x1p200)) : 0.f;
        };
        const float len_k = length(k, kk), len_q = length(q, qq);
        const float rq = qq > 0.f ? rsqrtf(qq) : 0.f, rk = kk > 0.f ? rsqrtf(kk) : 0.f;
        if (l == 0) {
            c_s[r] = len_k;
            e_s[r] = len_q;
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
            float *o = ck.vec + ((int64_t)local * a.hv + h) * VEC;
            const float eg = expf((float)G);
            o[lane] = eg * c_s[lane];
            o[64 + lane] = eg;
            o[128 + lane] = expf((float)(last - G)) * c_s[lane];
            o[192 + lane] = e_s[lane];
            if (lane == 0) o[256] = expf((float)last);
        }
        __syncthreads();
        f4 At[4];
        const double Gt = G_s[tl];
        const float bt = b_s[tl], ct = c_s[tl];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int jl = 16 * i + 4 * g + r;
                const float d = jl <= tl ? expf((float)(Gt - G_s[jl])) * c_s[jl] : 0.f;
                At[i][r] = d * kq[i][r] * (TRI_UNIT / (ROW_UNIT * ROW_UNIT));
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

constexpr int SCAN_WAVES = 8;

// LDS of a block is complete for every wave (loads from memory stay under way).
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// What the waves of a scan block pass on: operands in two parts (16 columns x
// twice, ct) and what they were scaled by.
template <int KB> struct Passed {
    h8 S[2][KB][2][2][64]; // [turn]
    h8 R[2][2][2][64];   // [rows 0..31, 32..63]
    h8 U[2][2][2][64];   // e^(G_last - G) c U
    f4 out[4][2][64];    // U in fp32
    float Sd[2][2][16][4]; // [turn][ct][x][kb]: a state's value is its parts times this (0 past KB)
    float Vm[2][16][4];  // [ct][x][row tile]: largest |V|
};

// N columns of a head's state through the tiles of a sequence.  Waves 0..3
// carry the state on: wave q has 32 of its dimensions (in registers, fp32; none
// with DK = 64 and q > 1) and 16 of a tile's rows, waves 4..7 make the outputs
// of 16 rows each.  So a matrix operand of the tile is read by one wave only,
// straight from memory into registers, a tile ahead.
//   phase 1  K^ S0 -> R = V - e^G c K^ S0    | Q^ S0
//   phase 2  U = T R
//   phase 3  the state, in two parts for the next tile | A U, outputs
// R and U are scaled by bounds that are known before them (rows of K^ have
// length 1, rows of T at most 64 elements up to 1), so no maximum is in the way.
template <int DK, typename V_T> __global__ void __launch_bounds__(64 * SCAN_WAVES) delta_scan_kernel(Args a, Chunks ck) {
    constexpr int KB = DK / 32, PART = Sizes<DK>::PART, F = FRAG / 8;
    __shared__ Passed<KB> sh;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, g = lane >> 4, q = w & 3;
    // blocks of one key head and sequence are 8 apart: on one XCD, whose L2 they share
    const int hk_n = a.hv / a.rep, slabs = a.dv / N, per = a.rep * slabs;
    const int64_t b = blockIdx.x, group = b % 8 + 8 * (b / (8 * per));
    if (group >= (int64_t)a.q.nseq * hk_n) return;
    const int member = (int)(b / 8 % per), s = (int)(group / hk_n), hk = (int)(group % hk_n), h = hk * a.rep + member / slabs;
    const int col = member % slabs * N + x;  // and 16 on
    const SeqState sq = seq_state(a.q, s);
    const Span sp = span_of(sq, a.out.p != nullptr);
    const int t0 = first_tile(a.q, s), j0 = max(ck.first - t0, 0), j1 = min(ck.first + ck.count - t0, sp.count);
    if (j0 >= j1) return;

    auto rows_of = [&](int j) { return reinterpret_cast<const h8 *>(ck.rows + ((int64_t)(t0 + j - ck.first) * hk_n + hk) * 3 * PART) + lane; };
    auto tri_of = [&](int j) { return reinterpret_cast<const h8 *>(ck.tri + ((int64_t)(t0 + j - ck.first) * a.hv + h) * (2 * TRI * 2 * FRAG)) + lane; };
    auto vec_of = [&](int j) { return ck.vec + ((int64_t)(t0 + j - ck.first) * a.hv + h) * VEC; };
    // (loads are waited for in the order they are issued in: none in the phase that issues it)
    h8 X[KB][2], Y[2][2];  // the wave's rows of K^ or Q^, and of T or A
    f4 ve, le;             // of e^G c or e^G; of e (outputs)
    const int which = w >> 2;
    auto bring_rows = [&](int j, int kb) {
        const h8 *p = rows_of(j) + ((which * 4 + q) * KB + kb) * 2 * F;
        X[kb][0] = p[0];
        X[kb][1] = p[F];
    };
    auto bring_vec = [&](int j) {
        ve = *reinterpret_cast<const f4 *>(vec_of(j) + 64 * which + 16 * q + 4 * g);
        if (which) le = *reinterpret_cast<const f4 *>(vec_of(j) + 192 + 16 * q + 4 * g);
    };
    auto bring_tri = [&](int j) {
        const h8 *p = tri_of(j) + which * TRI * 2 * F;
        const int first = q < 2 ? q : 2 * q - 2, second = q < 2 ? q : 2 * q - 1;  // (tri_index)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            Y[0][i] = p[(first * 2 + i) * F];
            Y[1][i] = p[(second * 2 + i) * F];
        }
    };
    // The wave's rows times the state, all of which is read from LDS before the first product.  Operands of the next tile
    // come when this one's are used, into the same registers (the order is kept: others would be copied, and waited for).
    auto times_state = [&](f4(&c)[2], int j, int jn) {
        f4 acc[KB * 2];
        h8 bh[KB][2], bl[KB][2];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                bh[kb][ct] = sh.S[j & 1][kb][ct][0][lane];
                bl[kb][ct] = sh.S[j & 1][kb][ct][1][lane];
            }
        in_order();
#pragma unroll
        for (int i = 0; i < KB * 2; ++i) acc[i] = mma(X[i / 2][1], bh[i / 2][i % 2], f4{0, 0, 0, 0});
#pragma unroll
        for (int i = 0; i < KB * 2; ++i) acc[i] = mma(X[i / 2][0], bl[i / 2][i % 2], acc[i]);
#pragma unroll
        for (int i = 0; i < KB * 2; ++i) acc[i] = mma(X[i / 2][0], bh[i / 2][i % 2], acc[i]);
        in_order();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) bring_rows(jn, kb);
        settle(acc);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            const f4 d = *reinterpret_cast<const f4 *>(sh.Sd[j & 1][ct][x]) * (1.f / ROW_UNIT);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                c[ct][r] = d[0] * acc[ct][r];
#pragma unroll
                for (int kb = 1; kb < KB; ++kb) c[ct][r] = fmaf(d[kb], acc[2 * kb + ct][r], c[ct][r]);
            }
        }
    };
    // the wave's rows of a triangle times 64 rows, those from 32 on only where the triangle has them
    auto times_rows = [&](auto rows, f4(&c)[2]) {
        c[0] = c[1] = f4{0, 0, 0, 0};
        h8 bh[2], bl[2];
        rows(0, bh, bl);
        in_order();
        mma3_grid<1>([&](int, int i) { return Y[0][i]; }, bh, bl, c);
        if (q < 2) settle(c);
        if (q >= 2) {
            rows(1, bh, bl);
            mma3_grid<1>([&](int, int i) { return Y[1][i]; }, bh, bl, c);
            settle(c);
        }
        in_order();
    };
    // bounds of R's columns: powers of two, from the state's and the tile's values
    auto bound = [&](int ct, int j) {
        const f4 m4 = *reinterpret_cast<const f4 *>(sh.Sd[j & 1][ct][x]), v4 = *reinterpret_cast<const f4 *>(sh.Vm[ct][x]);
        const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), v = fmaxf(fmaxf(v4[0], v4[1]), fmaxf(v4[2], v4[3]));
        return unit_at(fmaf(m, 12.f * 32768.f, v));  // |K^ S0| <= the length of S0's column < 12 times its largest value
    };

    if (w >= 4) {  // ---------------------------------------------- outputs
        // A U of the tile before in phase 1, its outputs in phase 2, Q^ S0 of this one in phase 3: what takes longest where
        // the other waves have most to do.
        f4 qs[2], au[2], es;  // es: the rows' lengths and the outputs' scale
        Unit u[2];
        auto product = [&](int jn) {
            times_rows([&](int k, h8 *bh, h8 *bl) {
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
                    split8(sh.out[2 * k][ct][lane], sh.out[2 * k + 1][ct][lane], u[ct].up * (1.f / 64), bh[ct], bl[ct]);
            }, au);
            bring_tri(jn);
        };
        auto finish = [&](int j) {
            const int r0 = tile_row(sq, sp, j), n = tile_end(sq, sp, j) - r0 - 16 * q - 4 * g;
            const int64_t at = (sq.first + r0 + 16 * q + 4 * g) * a.out.row + h * a.out.head + col * a.out.elem;
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const float f = u[ct].down * (64.f / TRI_UNIT);
#pragma unroll
                for (int r = 0; r < 4; ++r) au[ct][r] = es[r] * fmaf(f, au[ct][r], qs[ct][r]);
            }
            // (rows past the tile's end go to the unused part of its decays: with branches around them the number of stores
            // under way is not known, and loads from before them are waited for with all of them)
            auto put = [&](auto *p) {
                using T = std::remove_reference_t<decltype(*p)>;
                T *none = reinterpret_cast<T *>(const_cast<float *>(vec_of(j)) + 260);
                p += at;
#pragma unroll
                for (int r = 0; r < 4; ++r, p += a.out.row) {
                    *(r < n ? p : none) = (T)au[0][r];
                    *(r < n ? p + 16 * a.out.elem : none) = (T)au[1][r];
                }
            };
            if (a.out.f16) put(reinterpret_cast<_Float16 *>(a.out.p));
            else put(reinterpret_cast<float *>(a.out.p));
        };
        if (a.out.p) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) bring_rows(j0, kb);
            bring_vec(j0);
            bring_tri(j0);
        }
        meet();
        meet();
        for (int j = j0; j < j1; ++j) {
            const int jn = min(j + 1, j1 - 1);
            if (a.out.p && j > j0) product(j);
            meet();
            if (a.out.p) {
                if (j > j0) finish(j - 1);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) u[ct] = bound(ct, j);
            }
            meet();
            if (a.out.p) {
                times_state(qs, j, jn);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int r = 0; r < 4; ++r) qs[ct][r] *= ve[r];
                es = le * a.scale;
                in_order();
                bring_vec(jn);
            }
            meet();
        }
        if (a.out.p) {
            product(j1 - 1);
            finish(j1 - 1);
        }
        return;
    }

    // ------------------------------------------------------------------ the state
    const bool holds = q < KB;
    h8 Z[2][2][2];  // K^ by the wave's dimensions, [16 of them][rows 0..31, 32..63]
    f4 de;          // of e^(G_last - G) c
    float keep;
    auto bring_dims = [&](int j) {
        const h8 *p = rows_of(j) + (2 * 4 * KB * 2 + (holds ? q : 0) * 8) * F;
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) Z[d][k][i] = p[((d * 2 + k) * 2 + i) * F];
    };
    auto bring_keep = [&](int j) { keep = vec_of(j)[256 + (lane >> 6)]; };  // (a vector load)
    auto bring_de = [&](int j) { de = *reinterpret_cast<const f4 *>(vec_of(j) + 128 + 16 * q + 4 * g); };
    V_T raw[2][4];
    auto fetch = [&](int j) {  // values of the tile's rows (those past its end: of its last one)
        const int r0 = tile_row(sq, sp, j), n = tile_end(sq, sp, j) - r0;
        const V_T *p = reinterpret_cast<const V_T *>(a.vh.p) + (int64_t)(sq.first + r0) * a.vh.row + h * a.vh.head + col * a.vh.elem;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const V_T *v = p + min(16 * q + 4 * g + r, n - 1) * a.vh.row;
            raw[0][r] = v[0];
            raw[1][r] = v[16 * a.vh.elem];
        }
    };
    auto most_v = [&]() {
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            float m = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf((float)raw[ct][r]));
            m = over_rows(m);
            if (g == 0) sh.Vm[ct][x][q] = m;
        }
    };
    f4 S[2][2];  // [16 dimensions][ct]
    auto part_state = [&](int j) {
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            const Unit u = unit_at(over_rows(most8(S[0][ct], S[1][ct])));
            h8 hi, lo;
            split8(S[0][ct], S[1][ct], u.up, hi, lo);
            sh.S[j & 1][q][ct][0][lane] = hi;
            sh.S[j & 1][q][ct][1][lane] = lo;
            if (g == 0) sh.Sd[j & 1][ct][x][q] = u.down;
        }
    };
    const int64_t cell = ((int64_t)h * a.dv + col) * DK + 32 * q + 4 * g, slot = (int64_t)a.hv * a.dv * DK;
    auto leave = [&](float *p) {
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
            for (int d = 0; d < 2; ++d) *reinterpret_cast<f4 *>(p + 16 * ct * DK + 16 * d) = S[d][ct];
    };

    const float *from = j0 > 0 ? ck.carry + (ck.turn ^ 1) * slot + cell : sq.src >= 0 ? a.pool + sq.src * slot + cell : nullptr;
    if (!holds) from = nullptr;
#pragma unroll
    for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int d = 0; d < 2; ++d) S[d][ct] = from ? *reinterpret_cast<const f4 *>(from + 16 * ct * DK + 16 * d) : f4{0, 0, 0, 0};
    if (KB < 4) (&sh.Sd[0][0][0][0])[tid] = 0;
    meet();
    fetch(j0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) bring_rows(j0, kb);
    bring_vec(j0);
    bring_tri(j0);
    bring_de(j0);
    bring_dims(j0);
    bring_keep(j0);
    most_v();
    if (holds) part_state(j0);
    meet();
    for (int j = j0; j < j1; ++j) {
        const int n = tile_end(sq, sp, j) - tile_row(sq, sp, j) - 16 * q - 4 * g, jn = min(j + 1, j1 - 1);
        // phase 1
        Unit u[2];
        {
            f4 ks[2];
            times_state(ks, j, jn);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                u[ct] = bound(ct, j);
                h4 hi, lo;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float R = r < n ? fmaf(-ve[r], ks[ct][r], (float)raw[ct][r]) : 0.f;
                    _Float16 p, m;
                    split(R * u[ct].up, p, m);
                    hi[r] = p;
                    lo[r] = m;
                }
                reinterpret_cast<h4 *>(&sh.R[q >> 1][ct][0][lane])[q & 1] = hi;
                reinterpret_cast<h4 *>(&sh.R[q >> 1][ct][1][lane])[q & 1] = lo;
            }
            in_order();
            fetch(jn);
            bring_vec(jn);
        }
        meet();
        // phase 2
        {
            f4 U[2];
            times_rows([&](int k, h8 *bh, h8 *bl) {
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
                    bh[ct] = sh.R[k][ct][0][lane];
                    bl[ct] = sh.R[k][ct][1][lane];
                }
            }, U);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const float f = u[ct].down * (1.f / TRI_UNIT), up = u[ct].up * (1.f / 64);
                h4 hi, lo;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    U[ct][r] *= f;
                    _Float16 p, m;
                    split(de[r] * U[ct][r] * up, p, m);
                    hi[r] = p;
                    lo[r] = m;
                }
                sh.out[q][ct][lane] = U[ct];
                reinterpret_cast<h4 *>(&sh.U[q >> 1][ct][0][lane])[q & 1] = hi;
                reinterpret_cast<h4 *>(&sh.U[q >> 1][ct][1][lane])[q & 1] = lo;
            }
            in_order();
            bring_tri(jn);
            bring_de(jn);
        }
        meet();
        // phase 3
        if (holds) {
            f4 add[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) add[i] = f4{0, 0, 0, 0};
            h8 bh[2][2], bl[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
                    bh[k][ct] = sh.U[k][ct][0][lane];
                    bl[k][ct] = sh.U[k][ct][1][lane];
                }
            in_order();
#pragma unroll
            for (int k = 0; k < 2; ++k) mma3_grid<2>([&](int d, int i) { return Z[d][k][i]; }, bh[k], bl[k], add);
            in_order();
            bring_dims(jn);
            settle(add);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const float f = u[ct].down * (64.f / ROW_UNIT);
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[d][ct][r] = fmaf(f, add[2 * d + ct][r], keep * S[d][ct][r]);
            }
            if (j + 1 == sp.before && sq.commit) leave(a.pool + sq.dst * slot + cell);
            in_order();
            bring_keep(jn);
            part_state(j + 1);
        }
        most_v();
        meet();
    }
    if (holds && j1 < sp.count) leave(ck.carry + ck.turn * slot + cell);
}

template <int DK> int64_t tile_bytes(int hk, int hv) {
    return (int64_t)hk * 3 * Sizes<DK>::PART * 2 + (int64_t)hv * (2 * TRI * 2 * FRAG * 2 + VEC * 4);
}

// All tiles at once, or as many as have this much (a sequence's state is
// carried from one launch to the next): 6000 rows of 48 heads on 16, so that a
// prompt of any length needs no more (12288 rows 829 us; with 64 MB a launch 939,
// 4096 rows 313 for 267).
constexpr int64_t CAP = (int64_t)256 << 20;

struct Plan { int tiles, each; int64_t bytes; };
Plan plan_of(const StateSeqs &q, int hk, int hv, int dk, int dv) {
    const int64_t one = dk == 64 ? tile_bytes<64>(hk, hv) : tile_bytes<128>(hk, hv);
    const int tiles = q.rows / C + 2 * q.nseq, each = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, CAP / one));
    return {tiles, each, each * one + (each < tiles ? 2 * (int64_t)hv * dv * dk * 4 : 0)};
}

template <int DK, typename V_T> hipError_t go(const Args &a, int hk, void *workspace, hipStream_t st) {
    const Plan pl = plan_of(a.q, hk, a.hv, DK, a.dv);
    uint8_t *p = (uint8_t *)workspace;
    Chunks ck;
    ck.rows = (_Float16 *)p;
    p += (int64_t)pl.each * hk * 3 * Sizes<DK>::PART * 2;
    ck.tri = (_Float16 *)p;
    p += (int64_t)pl.each * a.hv * 2 * TRI * 2 * FRAG * 2;
    ck.vec = (float *)p;
    p += (int64_t)pl.each * a.hv * VEC * 4;
    ck.carry = (float *)p;
    const int64_t groups = ((int64_t)a.q.nseq * hk + 7) / 8 * 8;
    for (int first = 0, i = 0; first < pl.tiles; first += pl.each, ++i) {
        ck.first = first;
        ck.count = std::min(pl.each, pl.tiles - first);
        ck.turn = i & 1;
        hipLaunchKernelGGL(delta_tile_kernel<DK>, dim3((unsigned)((int64_t)ck.count * hk)), dim3(TILE_THREADS), 0, st, a, ck);
        hipLaunchKernelGGL((delta_scan_kernel<DK, V_T>), dim3((unsigned)(groups * a.rep * (a.dv / N))), dim3(64 * SCAN_WAVES), 0, st, a, ck);
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
