// qk_conv.hip -- the short causal convolution in front of the recurrence, with
// the rows that it still needs as its state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qk_act.h"
#include "qk_state.h"

namespace qk {
namespace conv {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
constexpr int R = 16;         // rows of a tile (32: 4096 rows 69.6 us for 71.1, but 17 rows 6.3 for 5.9)
constexpr int THREADS = 64;   // a wave: few channels fill the chip too

struct Args {
    StateSeqs q;
    ConvState c;
    Heads x, y;
    int act;
    int64_t tiles;
    int chunks;               // of THREADS threads, over the channels
};

// C consecutive channels of a row: [channel] on of view v.
template <int C> __device__ __forceinline__ void load(const Heads &v, int64_t row, int c, float *x) {
    if constexpr (C == 4) {
        const int64_t o = row * v.row + c;
        if (v.f16) {
            const h4 h = *reinterpret_cast<const h4 *>(reinterpret_cast<const _Float16 *>(v.p) + o);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (float)h[e];
        } else {
            const float4 f = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(v.p) + o);
            x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
        }
    } else {
        const int64_t o = row * v.row + c * v.elem;
        x[0] = v.f16 ? (float)reinterpret_cast<const _Float16 *>(v.p)[o] : reinterpret_cast<const float *>(v.p)[o];
    }
}
template <int C> __device__ __forceinline__ void store(const Heads &v, int64_t row, int c, const float *x) {
    if constexpr (C == 4) {
        const int64_t o = row * v.row + c;
        if (v.f16) *reinterpret_cast<h4 *>(reinterpret_cast<_Float16 *>(v.p) + o) = h4{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
        else *reinterpret_cast<float4 *>(reinterpret_cast<float *>(v.p) + o) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
        const int64_t o = row * v.row + c * v.elem;
        if (v.f16) reinterpret_cast<_Float16 *>(v.p)[o] = (_Float16)x[0];
        else reinterpret_cast<float *>(v.p)[o] = x[0];
    }
}

// A thread has C channels and a tile's rows, the T - 1 rows before the current
// one in registers.  Only the first tile of a sequence reads its old state, and
// its threads write the new one: a tile is at least T - 1 rows.  Memory bounds
// it: 4096 rows of 10240 channels (335 MB) 69-75 us, 4.5-4.9 TB/s where a copy
// reaches 5.1; tiles of 16 rows read 3 rows twice, from L2 (190 MB fetched of
// 168).  17 drafts: 6 us, where lookup, weights and rows follow one another.
template <int T, int C> __global__ void __launch_bounds__(THREADS) conv_kernel(Args a) {
    static_assert(R >= T - 1, "the second tile of a sequence needs rows of the first only");
    constexpr int B = T - 1;
    const int lane = threadIdx.x & 63;
    for (int64_t u = blockIdx.x; u < a.tiles * a.chunks; u += gridDim.x) {
        const int64_t tile = u / a.chunks;
        const int c = ((int)(u % a.chunks) * THREADS + threadIdx.x) * C;
        const Tile tl = state_tile(a.q, tile, R, lane);
        if (tl.s < 0 || tl.j < 0) continue;  // (below 0: of starts that decrease)
        const SeqState sq = seq_state(a.q, tl.s);
        const int i0 = tl.j * R, i1 = min(i0 + R, sq.n);
        if (i0 >= i1 || c >= a.c.channels) continue;
        float w[C][T], bias[C], x[T][C];
#pragma unroll
        for (int e = 0; e < C; ++e) {
#pragma unroll
            for (int j = 0; j < T; ++j) w[e][j] = a.c.weight[(int64_t)(c + e) * T + j];
            bias[e] = a.c.bias ? a.c.bias[c + e] : 0.f;
        }
        const float *old = sq.src < 0 ? nullptr : a.c.pool + (sq.src * B) * a.c.channels + c;
        if (tl.j == 0) {
            float old_v[B][C];
#pragma unroll
            for (int j = 0; j < B; ++j)
#pragma unroll
                for (int e = 0; e < C; ++e) x[j][e] = old_v[j][e] = old ? old[(int64_t)j * a.c.channels + e] : 0.f;
            if (sq.commit) {
                float *out = a.c.pool + (sq.dst * B) * a.c.channels + c;
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const int i = sq.commit - B + j;  // row of the sequence, below 0: of the old state
                    float v[C];
                    if (i >= 0) {
                        load<C>(a.x, sq.first + i, c, v);
                    } else {
#pragma unroll
                        for (int e = 0; e < C; ++e) {
                            v[e] = 0;
#pragma unroll
                            for (int k = 0; k < B; ++k) v[e] = k == i + B ? old_v[k][e] : v[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < C; ++e) out[(int64_t)j * a.c.channels + e] = v[e];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < B; ++j) load<C>(a.x, sq.first + i0 - B + j, c, x[j]);
        }
        if (!a.y.p) continue;
        // H rows are loaded before the first of them is worked on (4 channels: 4 rows 75 us for 71 at 4096
        // rows, 16 139 for want of registers)
        constexpr int H = C == 4 ? 8 : R;
        for (int h0 = i0; h0 < i1; h0 += H) {
            float next[H][C];
#pragma unroll
            for (int i = 0; i < H; ++i)
                if (h0 + i < i1) load<C>(a.x, sq.first + h0 + i, c, next[i]);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if (h0 + i >= i1) break;
                float y[C];
#pragma unroll
                for (int e = 0; e < C; ++e) {
                    x[B][e] = next[i][e];
                    float s = bias[e];
#pragma unroll
                    for (int j = 0; j < T; ++j) s = fmaf(w[e][j], x[j][e], s);
                    y[e] = a.act ? silu(s) : s;
                }
                store<C>(a.y, sq.first + h0 + i, c, y);
#pragma unroll
                for (int j = 0; j < B; ++j)
#pragma unroll
                    for (int e = 0; e < C; ++e) x[j][e] = x[j + 1][e];
            }
        }
    }
}

bool whole4(const Heads &v) {
    return !v.p || (v.elem == 1 && v.row % 4 == 0 && ((uintptr_t)v.p & (v.f16 ? 7 : 15)) == 0);
}

template <int T> hipError_t go(Args a, hipStream_t st) {
    const bool vec = a.c.channels % 4 == 0 && whole4(a.x) && whole4(a.y) && ((uintptr_t)a.c.pool & 15) == 0;
    const int per = THREADS * (vec ? 4 : 1);
    a.chunks = (a.c.channels + per - 1) / per;
    a.tiles = state_tiles(a.q, R);
    const unsigned blocks = (unsigned)std::min<int64_t>(a.tiles * a.chunks, 1 << 22);  // (a grid stays below 2^32 threads)
    if (vec) hipLaunchKernelGGL((conv_kernel<T, 4>), dim3(blocks), dim3(THREADS), 0, st, a);
    else hipLaunchKernelGGL((conv_kernel<T, 1>), dim3(blocks), dim3(THREADS), 0, st, a);
    return hipGetLastError();
}

}  // namespace conv

hipError_t launch_conv(const StateSeqs &q, const ConvState &c, int act, const Heads &x, const Heads &y, hipStream_t st) {
    const conv::Args a{q, c, x, y, act, 0, 0};
    switch (c.taps) {
    case 2: return conv::go<2>(a, st);
    case 3: return conv::go<3>(a, st);
    case 4: return conv::go<4>(a, st);
    case 5: return conv::go<5>(a, st);
    case 6: return conv::go<6>(a, st);
    case 7: return conv::go<7>(a, st);
    default: return conv::go<8>(a, st);
    }
}

}  // namespace qk
