// qk_delta.h -- device side shared by the kernels of the gated delta
// recurrence: arguments, elements of rows, gates.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_state.h"

namespace qk {
namespace delta {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));

struct Args {
    StateSeqs q;
    float *pool;              // [slots][hv][dv][DK]
    int hv, rep, dv;          // rep: value heads a key head
    int norm, q_vec, k_vec;   // _vec: rows of heads are whole pieces of 4 elements
    float eps, scale;
    Heads qh, kh, vh, alpha, beta, out;
    const float *A, *dt;
};

inline bool whole4(const Heads &v) {
    return v.elem == 1 && v.row % 4 == 0 && v.head % 4 == 0 && ((uintptr_t)v.p & (v.f16 ? 7 : 15)) == 0;
}

inline Args make_args(const StateSeqs &q, const DeltaState &d, const DeltaIn &in, const Heads &out) {
    return Args{q, d.pool, d.hv, d.hv / d.hk, d.dv, in.norm, whole4(in.q), whole4(in.k), in.eps, in.scale,
                in.q, in.k, in.v, in.alpha, in.beta, out, in.A, in.dt};
}

// v of the lane `CTRL` away inside a row of 16 lanes
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sum over 16 lanes: each gets it.
__device__ __forceinline__ float sum16(float v) {
    v += dpp<0xB1>(v);   // quad_perm [1,0,3,2]
    v += dpp<0x4E>(v);   // quad_perm [2,3,0,1]
    v += dpp<0x141>(v);  // half row mirrored
    v += dpp<0x140>(v);  // row mirrored
    return v;
}

__device__ __forceinline__ float load1(const Heads &x, int64_t t, int h, int i) {
    const int64_t o = t * x.row + h * x.head + i * x.elem;
    return x.f16 ? (float)reinterpret_cast<const _Float16 *>(x.p)[o] : reinterpret_cast<const float *>(x.p)[o];
}
__device__ __forceinline__ void store1(const Heads &x, int64_t t, int h, int i, float v) {
    const int64_t o = t * x.row + h * x.head + i * x.elem;
    if (x.f16) reinterpret_cast<_Float16 *>(x.p)[o] = (_Float16)v;
    else reinterpret_cast<float *>(x.p)[o] = v;
}
// P pieces of 4 dimensions of a row's head, from dimension i on, STEP apart.
template <int P, int STEP>
__device__ __forceinline__ void load_pieces(bool vec, const Heads &x, int64_t t, int h, int i, float (*r)[4]) {
    const int64_t o = t * x.row + h * x.head;
    if (vec && x.f16) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const h4 v = *reinterpret_cast<const h4 *>(reinterpret_cast<const _Float16 *>(x.p) + o + i + STEP * p);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[p][e] = (float)v[e];
        }
    } else if (vec) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(x.p) + o + i + STEP * p);
            r[p][0] = v.x; r[p][1] = v.y; r[p][2] = v.z; r[p][3] = v.w;
        }
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) r[p][e] = load1(x, t, h, i + STEP * p + e);
    }
}

// Rows whose sum of squares is below SHORT: fp32 has lost bits of smaller
// squares, and of products with a row of the other kind.  Their elements are
// made larger by a power of two first.
constexpr float SHORT = 0x1p-80f;
template <int P> __device__ __forceinline__ float enlarge(float (*x)[4], float up) {
    float xx = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[p][e] *= up;
            xx = fmaf(x[p][e], x[p][e], xx);
        }
    return xx;
}

// Log decay (never above 0) and step of a row's head.  Raw gates: g = A log(1 +
// e^(alpha + dt)), without overflow on either side; beta through the logistic
// function.
struct Gate { float g, b; };
__device__ __forceinline__ Gate gates(const Args &a, int h, float al, float be) {
    float g = al, b = be;
    if (a.A) {
        const float w = al + (a.dt ? a.dt[h] : 0.f);
        g = a.A[h] * (fmaxf(w, 0.f) + log1pf(expf(-fabsf(w))));
        b = 1.f / (1.f + expf(-be));
    }
    return {g > 0.f ? 0.f : g, b};  // (NaN stays)
}

}  // namespace delta

// Long sequences (qk_delta_chunk.hip); rows of length 1 and raw gates only.
int64_t delta_chunk_workspace(const StateSeqs &q, const DeltaState &d);
hipError_t launch_delta_chunk(const delta::Args &a, int hk, int dk, void *workspace, hipStream_t st);

}  // namespace qk
