// qk_state.h -- device side of sequences that carry a recurrent state: which
// rows are a sequence's, where its state comes from and where it is left.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_kv.h"

namespace qk {

struct SeqState {
    int first, n;     // its rows
    int64_t src, dst; // slots, -1: zeros / not kept
    int commit;       // the state after this many rows is kept (0: none)
};

// (uniform loads; every index is bounded here)
__device__ __forceinline__ SeqState seq_state(const StateSeqs &q, int s) {
    SeqState r;
    if (q.q_start) {
        const int a = min(max(q.q_start[s], 0), q.rows);
        r.first = a;
        r.n = max(min(max(q.q_start[s + 1], 0), q.rows) - a, 0);
    } else {
        r.n = q.rows / q.nseq;
        r.first = s * r.n;
    }
    const int in = q.slots[s], out = q.slots_out ? q.slots_out[s] : in;
    const bool go_on = !q.kv_len || q.kv_len[s] > r.n;
    r.src = go_on && in >= 0 && in < q.num_slots ? in : -1;
    r.dst = out >= 0 && out < q.num_slots ? out : -1;
    r.commit = q.commit ? min(max(q.commit[s], 0), r.n) : r.n;
    if (r.dst < 0) r.commit = 0;
    return r;
}

// Tiles of R rows, each of one sequence.  Where sequences differ in length,
// sequence s has the numbers from q_start[s] / R + s on: those of the next one
// begin behind its last, whatever its length, and rows / R + nseq are enough.
inline int64_t state_tiles(const StateSeqs &q, int R) {
    if (q.q_start) return (int64_t)q.rows / R + q.nseq;
    return (int64_t)q.nseq * ((q.rows / q.nseq + R - 1) / R);
}

struct Tile { int s, j; };  // sequence (-1: none), tile of it
__device__ __forceinline__ Tile state_tile(const StateSeqs &q, int64_t b, int R, int lane) {
    if (!q.q_start) {
        const int per = (q.rows / q.nseq + R - 1) / R;
        return {(int)(b / per), (int)(b % per)};
    }
    auto first = [&](int i) { return (int64_t)(min(max(q.q_start[i], 0), q.rows) / R + i); };
    const int s = __builtin_amdgcn_readfirstlane(count_while(q.nseq, lane, [&](int i) { return first(i) <= b; })) - 1;
    return {s, s < 0 ? 0 : (int)(b - first(s))};
}

}  // namespace qk
