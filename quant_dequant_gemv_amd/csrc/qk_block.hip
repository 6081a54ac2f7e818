// qk_block.hip -- the norms before and after a block with its gate and
// residual, in one pass over the row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qk_act.h"
#include "qk_launch.h"

namespace qk {
namespace block {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));

struct Args {
    BlockNorm b;
    uint32_t units;  // rows x groups (at most 2^25)
    int groups, dim;
    double inv;     // 1 / dim
    Heads y, gate, res, h, x;
};

// Row t, group g of a view.
__device__ __forceinline__ char *at(const Heads &v, int64_t t, int64_t g) {
    return reinterpret_cast<char *>(v.p) + ((t * v.row + g * v.head) << (v.f16 ? 1 : 2));
}

// E elements of a group of `dim` at p, TPG threads: pieces of 4 side by side
// (VEC), or single ones `elem` apart.  Zeros past the end.  All loads of a
// thread are under way before the first is converted.
template <int TPG, int E, bool VEC>
__device__ __forceinline__ void load(const char *p, int64_t elem, bool f16, int tid, int dim, float *x) {
    if constexpr (VEC) {
        if (f16) {
            h4 h[E / 4];
#pragma unroll
            for (int j = 0; j < E / 4; ++j) {
                const int i = 4 * (tid + TPG * j);
                h[j] = i < dim ? *reinterpret_cast<const h4 *>(p + 2 * i) : h4{0, 0, 0, 0};
            }
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = (float)h[e / 4][e % 4];
        } else {
#pragma unroll
            for (int j = 0; j < E / 4; ++j) {
                const int i = 4 * (tid + TPG * j);
                const float4 f = i < dim ? *reinterpret_cast<const float4 *>(p + 4 * i) : make_float4(0, 0, 0, 0);
                x[4 * j] = f.x; x[4 * j + 1] = f.y; x[4 * j + 2] = f.z; x[4 * j + 3] = f.w;
            }
        }
    } else if (f16) {
        _Float16 h[E];
        p += tid * elem * 2;
#pragma unroll
        for (int j = 0; j < E; ++j, p += TPG * elem * 2) h[j] = tid + TPG * j < dim ? *reinterpret_cast<const _Float16 *>(p) : (_Float16)0;
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = (float)h[j];
    } else {
        p += tid * elem * 4;
#pragma unroll
        for (int j = 0; j < E; ++j, p += TPG * elem * 4) x[j] = tid + TPG * j < dim ? *reinterpret_cast<const float *>(p) : 0.f;
    }
}
template <int TPG, int E, bool VEC>
__device__ __forceinline__ void store(char *p, int64_t elem, bool f16, int tid, int dim, const float *x) {
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < E / 4; ++j) {
            const int i = 4 * (tid + TPG * j);
            if (i >= dim) continue;
            const float *f = x + 4 * j;
            if (f16) *reinterpret_cast<h4 *>(p + 2 * i) = h4{(_Float16)f[0], (_Float16)f[1], (_Float16)f[2], (_Float16)f[3]};
            else *reinterpret_cast<float4 *>(p + 4 * i) = make_float4(f[0], f[1], f[2], f[3]);
        }
    } else {
        p += (tid * elem) << (f16 ? 1 : 2);
        const int64_t step = (TPG * elem) << (f16 ? 1 : 2);
#pragma unroll
        for (int j = 0; j < E; ++j, p += step) {
            if (tid + TPG * j >= dim) continue;
            if (f16) *reinterpret_cast<_Float16 *>(p) = (_Float16)x[j];
            else *reinterpret_cast<float *>(p) = x[j];
        }
    }
}

// v of the lane `CTRL` away inside a row of 16 lanes
template <int CTRL> __device__ __forceinline__ double dpp(double v) {
    const uint2 w = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, make_uint2(__builtin_amdgcn_update_dpp(0, (int)w.x, CTRL, 0xf, 0xf, true),
                                                 __builtin_amdgcn_update_dpp(0, (int)w.y, CTRL, 0xf, 0xf, true)));
}
// Sum over the TPG threads of a group: every one gets it.  Fixed order.
template <int TPG, int THREADS> __device__ __forceinline__ double group_sum(double v, double *part, int tid) {
    v += dpp<0xB1>(v);   // quad_perm [1,0,3,2]
    v += dpp<0x4E>(v);   // quad_perm [2,3,0,1]
    v += dpp<0x141>(v);  // half row mirrored
    v += dpp<0x140>(v);  // row mirrored
    if (TPG > 16) v += __shfl_xor(v, 16);
    if (TPG > 32) v += __shfl_xor(v, 32);
    if constexpr (TPG > 64) {
        static_assert(TPG == THREADS, "one group a block above a wave");
        __syncthreads();
        if ((tid & 63) == 0) part[tid >> 6] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < TPG / 64; ++w) v += part[w];
    }
    return v;
}

__device__ __forceinline__ float gate_of(float z, int act) {
    return act == 0 ? z : act == 1 ? silu(z) : logistic(z);
}

// What brings a row of mean square m to length 1 an element: fp32 (the
// hardware's root refined once) for the sums of squares that fp32 holds, 1e-25
// to 1e37, fp64 for the others: no row overflows or vanishes (with an eps of up to
// 1e37, above which the kernel of long groups, fp64 throughout, takes all).
__device__ __forceinline__ bool ordinary(double ss) { return ss >= 1e-25 && ss <= 1e37; }
__device__ __forceinline__ float root32(double ss, double inv, float eps) {
    const float m = (float)fma(ss, inv, (double)eps), r = rsqrtf(m);
    return fmaf(r, 0.5f * fmaf(-m * r, r, 1.f), r);
}
__device__ __forceinline__ double root64(double ss, double inv, float eps) { return 1.0 / sqrt(fma(ss, inv, (double)eps)); }

// x <- x / sqrt(mean x^2 + eps) * w.  Up to 8 squares of a thread are summed in
// fp32, those sums in fp64: the root is off by 8 / 2 + 2 halves of 2^-23, an
// element by two more.
template <int TPG, int THREADS, int E, bool VEC>
__device__ __forceinline__ void norm(float *x, const float *w, float eps, int dim, double inv, int tid, double *part) {
    float wv[E];
    load<TPG, E, VEC>(reinterpret_cast<const char *>(w), 1, false, tid, dim, wv);
    double ss = 0;
#pragma unroll
    for (int j0 = 0; j0 < E; j0 += 8) {
        float s = 0;
#pragma unroll
        for (int j = j0; j < (E < j0 + 8 ? E : j0 + 8); ++j) s = fmaf(x[j], x[j], s);
        ss += s;
    }
    ss = group_sum<TPG, THREADS>(ss, part, tid);
    if (ordinary(ss)) {
        const float r = root32(ss, inv, eps);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = x[j] * r * wv[j];
        return;
    }
    ss = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) ss = fma((double)x[j], (double)x[j], ss);
    const double r = root64(group_sum<TPG, THREADS>(ss, part, tid), inv, eps);
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = (float)((double)x[j] * r) * wv[j];
}

// TPG threads a group of `dim` values, E of them each, in registers from the
// loads to the stores: every input is read once, so memory bounds it.  2048 rows
// of 48 gated heads of 128 (126 MB): 21-22 us, 5.8 TB/s, 335 instructions a wave
// and 76% of the issue slots.  One row of 5120: 3.4 us, a launch's and two
// round trips' time.  17 rows side by side (4 bytes of each line a row): 10-11 us,
// 20480 accesses a row that each take a line, one a cycle and CU.
template <int TPG, int THREADS, int E, bool VEC> __global__ void __launch_bounds__(THREADS) block_norm_kernel(Args a) {
    __shared__ double part[THREADS / 64];
    const int tid = threadIdx.x % TPG;
    constexpr int PER = THREADS / TPG;
    for (uint32_t u0 = blockIdx.x * PER; u0 < a.units; u0 += gridDim.x * PER) {
        // (units past the end work on the last one and store nothing: all threads meet at the sums)
        const uint32_t u = u0 + threadIdx.x / TPG, uc = u < a.units ? u : a.units - 1;
        const uint32_t t = uc / (uint32_t)a.groups, g = uc - t * a.groups;
        float y[E], z[E], r[E];
        load<TPG, E, VEC>(at(a.y, t, g), a.y.elem, a.y.f16, tid, a.dim, y);
        if (a.gate.p) load<TPG, E, VEC>(at(a.gate, t, g), a.gate.elem, a.gate.f16, tid, a.dim, z);
        if (a.res.p) load<TPG, E, VEC>(at(a.res, t, g), a.res.elem, a.res.f16, tid, a.dim, r);
        if (a.b.post) norm<TPG, THREADS, E, VEC>(y, a.b.post, a.b.eps, a.dim, a.inv, tid, part);
        if (a.gate.p) {
#pragma unroll
            for (int j = 0; j < E; ++j) y[j] *= gate_of(z[j], a.b.act);
        }
#pragma unroll
        for (int j = 0; j < E; ++j) y[j] = a.res.p ? fmaf(a.b.scale, y[j], r[j]) : a.b.scale * y[j];
        if (a.h.p && u < a.units) store<TPG, E, VEC>(at(a.h, t, g), a.h.elem, a.h.f16, tid, a.dim, y);
        if (a.x.p) {
            if (a.b.pre) norm<TPG, THREADS, E, VEC>(y, a.b.pre, a.b.eps, a.dim, a.inv, tid, part);
            if (u < a.units) store<TPG, E, VEC>(at(a.x, t, g), a.x.elem, a.x.f16, tid, a.dim, y);
        }
    }
}

// Groups too long for registers: the row's values wait in LDS between the
// sums, one group a block.  2048 rows of 16384 with a residual (470 MB): 118 us,
// 4.0 TB/s, its waves waiting 80% of their time; one row 9.7 us, four round trips.
template <bool VEC> __global__ void __launch_bounds__(1024) block_norm_wide_kernel(Args a) {
    constexpr int T = 1024, E = VEC ? 4 : 1;
    extern __shared__ float row[];
    __shared__ double part[T / 64];
    const int tid = threadIdx.x;
    for (uint32_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const uint32_t t = u / (uint32_t)a.groups, g = u - t * a.groups;
        double ss = 0, r = 1;
        // element i of a view, and E from it on
        auto from = [&](const Heads &v, int i) { return at(v, t, g) + ((i * v.elem) << (v.f16 ? 1 : 2)); };
        for (int i = E * tid; i < a.dim; i += E * T) {
            float y[E];
            load<T, E, VEC>(from(a.y, i), 1, a.y.f16, 0, E, y);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                row[i + e] = y[e];
                ss = fma((double)y[e], (double)y[e], ss);
            }
        }
        if (a.b.post) r = root64(group_sum<T, T>(ss, part, tid), a.inv, a.b.eps);
        ss = 0;
        for (int i = E * tid; i < a.dim; i += E * T) {
            float z[E], s[E];
            if (a.gate.p) load<T, E, VEC>(from(a.gate, i), 1, a.gate.f16, 0, E, z);
            if (a.res.p) load<T, E, VEC>(from(a.res, i), 1, a.res.f16, 0, E, s);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float y = row[i + e];
                if (a.b.post) y = (float)((double)y * r) * a.b.post[i + e];
                if (a.gate.p) y *= gate_of(z[e], a.b.act);
                row[i + e] = z[e] = a.res.p ? fmaf(a.b.scale, y, s[e]) : a.b.scale * y;
                ss = fma((double)z[e], (double)z[e], ss);
            }
            if (a.h.p) store<T, E, VEC>(from(a.h, i), 1, a.h.f16, 0, E, z);
        }
        if (!a.x.p) continue;
        if (a.b.pre) r = root64(group_sum<T, T>(ss, part, tid), a.inv, a.b.eps);
        for (int i = E * tid; i < a.dim; i += E * T) {
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = a.b.pre ? (float)((double)row[i + e] * r) * a.b.pre[i + e] : row[i + e];
            store<T, E, VEC>(from(a.x, i), 1, a.x.f16, 0, E, y);
        }
    }
}

bool whole4(const Heads &v) {
    return !v.p || (v.elem == 1 && v.row % 4 == 0 && v.head % 4 == 0 && ((uintptr_t)v.p & (v.f16 ? 7 : 15)) == 0);
}

template <int TPG, int THREADS, int E> hipError_t go(const Args &a, bool vec, hipStream_t st) {
    constexpr int PER = THREADS / TPG;
    const int64_t blocks = std::min<int64_t>(((int64_t)a.units + PER - 1) / PER, 1 << 20);  // (a grid stays below 2^32 threads)
    if (vec) hipLaunchKernelGGL((block_norm_kernel<TPG, THREADS, E, true>), dim3((unsigned)blocks), dim3(THREADS), 0, st, a);
    else hipLaunchKernelGGL((block_norm_kernel<TPG, THREADS, E, false>), dim3((unsigned)blocks), dim3(THREADS), 0, st, a);
    return hipGetLastError();
}

}  // namespace block

hipError_t launch_block_norm(const BlockNorm &b, int rows, int groups, int dim, const Heads &y, const Heads &gate,
                             const Heads &res, const Heads &h, const Heads &x, hipStream_t st) {
    using namespace block;
    const Args a{b, (uint32_t)(rows * groups), groups, dim, 1.0 / dim, y, gate, res, h, x};
    const bool vec = dim % 4 == 0 && whole4(y) && whole4(gate) && whole4(res) && whole4(h) && whole4(x) &&
                     (((uintptr_t)b.post | (uintptr_t)b.pre) & 15) == 0;
    // Threads a group: enough loads at once in each, few waves to meet at the sums (one row of 5120
    // with 8 / 16 values a thread: 4.5 / 4.2 us, 2048 rows 36.4 / 35.1; 2048 rows of 1024: 8.2 / 5.9;
    // 2048 rows of 4096: 32.4 / 21.4, but of 2048 11.5 / 13.6)
    if (b.eps <= 1e37f) {
        if (dim <= 64) return go<16, 256, 4>(a, vec, st);
        if (dim <= 128) return go<16, 256, 8>(a, vec, st);
        if (dim <= 256) return go<32, 256, 8>(a, vec, st);
        if (dim <= 512) return go<64, 256, 8>(a, vec, st);
        if (dim <= 1024) return go<64, 256, 16>(a, vec, st);
        if (dim <= 2048) return go<256, 256, 8>(a, vec, st);
        if (dim <= 4096) return go<256, 256, 16>(a, vec, st);
        if (dim <= 8192) return go<512, 512, 16>(a, vec, st);
    }
    const unsigned blocks = (unsigned)std::min<int64_t>(a.units, 1 << 20);
    auto wide = [&](auto kern, hipError_t e) {
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3(blocks), dim3(1024), 4 * dim, st, a);
        return hipGetLastError();
    };
    return vec ? wide(block_norm_wide_kernel<true>, lds_opt_in<block_norm_wide_kernel<true>>(4 * 32768))
               : wide(block_norm_wide_kernel<false>, lds_opt_in<block_norm_wide_kernel<false>>(4 * 32768));
}

}  // namespace qk
