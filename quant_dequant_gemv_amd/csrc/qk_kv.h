// qk_kv.h -- device side of the paged 4-bit cache, shared by the kernels that
// write it, read it back and attend over it: where a row stands, where a
// position lies, and the layout of a page (include/qkgemv.h has it in full).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_launch.h"

namespace qk {

// Byte offsets inside one head's block of a page (S = 1 << ps_log2 positions).
template <int D> struct KvLayout {
    static constexpr int G = D / 32;       // groups of a row
    static constexpr int ROW = D / 2;      // code bytes of a row
    static constexpr int VW = D >= 128 ? D / 128 : 1;   // pieces of 16 lanes in a value row
    static constexpr int VB = D >= 128 ? 4 : 2;         // bytes of a lane's piece
    static constexpr int VN = 2 * VB;                   // nibbles of it
    __host__ __device__ static constexpr int64_t block(int ps_log2) { return kv_block_bytes(D, 1 << ps_log2); }
    __device__ static int d_off(int ps_log2) { return ROW << ps_log2; }
    __device__ static int m_off(int ps_log2) { return (ROW + 2 * G) << ps_log2; }
    // fp16 element of a [S/4][G][4] plane
    __device__ static int by4(int p, int g) { return ((p >> 2) * G + g) * 4 + (p & 3); }
    // code bytes of lane l's piece w of a value row
    __device__ static int v_piece(int p, int w, int l) { return ((((p >> 2) * VW + w) * 16 + l) * 4 + (p & 3)) * VB; }
};

__device__ __forceinline__ int clamp_row(const KvSeqs &q, int v) { return min(max(v, 0), q.rows); }

// How many of the first n indices hold, `holds` being true up to one of them
// and false from there on: 64 places at a time, so one load deep up to 64 and
// three up to 2^18.  One wave, every lane gets the same answer (in 0..n
// whatever `holds` says).
template <typename F> __device__ __forceinline__ int count_while(int n, int lane, F holds) {
    int lo = 0;
    while (n > 64) {
        const int step = (n + 63) >> 6;
        const int c = __popcll(__ballot(lane * step < n && holds(lo + min(lane * step, n - 1))));
        if (!c) return lo;
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
    }
    return lo + __popcll(__ballot(lane < n && holds(lo + min(lane, n - 1))));
}

// Sequence of row t (nseq where it belongs to none) and its first row and row
// count; one wave, uniform.
struct RowSeq { int s, first, n; };
__device__ __forceinline__ RowSeq row_seq(const KvSeqs &q, int t, int lane) {
    if (!q.q_start) {
        const int n = q.rows / q.nseq;
        return {t / n, t / n * n, n};
    }
    const int s = __builtin_amdgcn_readfirstlane(count_while(q.nseq, lane, [&](int i) { return q.q_start[i] <= t; })) - 1;
    if (s < 0) return {q.nseq, 0, 0};
    const int first = clamp_row(q, q.q_start[s]), end = clamp_row(q, q.q_start[s + 1]);
    if (t < first || t >= end) return {q.nseq, 0, 0};  // behind the last sequence (or starts that decrease)
    return {s, first, end - first};
}

// Page of position p of sequence s, or -1 where none is held.
__device__ __forceinline__ int kv_page(const KvCache &c, const KvSeqs &q, int s, int64_t p) {
    if (p < 0 || p >= ((int64_t)q.max_pages << c.ps_log2)) return -1;
    const int page = q.pages[(int64_t)s * q.max_pages + (p >> c.ps_log2)];
    return page >= 0 && page < c.num_pages ? page : -1;
}

}  // namespace qk
