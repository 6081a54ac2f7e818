// qk_api.hip -- the C ABI declared in include/qkgemv.h: argument checks,
// type x ncols dispatch, launch on the caller's stream.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/qkgemv.h"
#include "qk_launch.h"

#ifndef QKGEMV_VERSION
#define QKGEMV_VERSION "0.1.0"
#endif

namespace {

thread_local char g_launch_msg[256] = "launch failed";

static_assert(QK_PLANAR == qk::PLANAR_FLAG, "layout flag of the C ABI and the kernels");

int block_bytes(int type) {
    switch (type) {
    case QK_Q4_K: return 144;
    case QK_Q5_K: return 176;
    case QK_Q6_K: return 210;
    case QK_IQ4_XS: return 136;
    default: return -1;
    }
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Bytes of one row in the layout the type flags name, or -1.
int64_t row_bytes_of(int type, int64_t K) {
    const int bb = block_bytes(type & ~QK_PLANAR);
    if (bb < 0 || (type & ~(QK_PLANAR | 0xff)) != 0 || K < 256 || (K % 256) != 0) return -1;
    if (type == (QK_IQ4_XS | QK_PLANAR)) return -1;  // the k-quants only
    const int64_t b = (K / 256) * bb;
    return (type & QK_PLANAR) ? (b + 15) / 16 * 16 : b;
}

// Shared shape check.  Rows and columns must keep every byte offset inside
// int64 and every per-launch index inside the kernels' 32-bit ranges.
int check_shape(int type, int64_t N, int64_t K, int ncols) {
    if (block_bytes(type & ~QK_PLANAR) < 0 || (type & ~(QK_PLANAR | 0xff)) != 0) return QK_EINVAL_TYPE;
    if (N < 1 || K < 256 || (K % 256) != 0) return QK_EINVAL_SHAPE;
    if (ncols < 1 || ncols > QK_MAX_NCOLS) return QK_EINVAL_SHAPE;
    if ((type & QK_PLANAR) && (ncols != 1 || (type & ~QK_PLANAR) == QK_IQ4_XS)) return QK_EINVAL_TYPE;
    if (K > (int64_t)1 << 30 || N > ((int64_t)1 << 31) - 1) return QK_EINVAL_SHAPE;
    const int64_t row_bytes = row_bytes_of(type, K);
    if (N > INT64_MAX / row_bytes) return QK_EINVAL_SHAPE;
    if (N > INT64_MAX / ((int64_t)K * 4)) return QK_EINVAL_SHAPE;
    return QK_OK;
}

int launched(hipError_t e);

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

// Pointer checks of the GEMV entry points (y fp32 or, with QK_Y_F16, fp16;
// the residual may be y itself only when y is fp32).  y is written while W
// and x are still being read by other workgroups, so y may overlap neither.
int check_io(int type, const void *W, const void *x, void *y, const void *res, int64_t N, int64_t K, int ncols,
             int flags) {
    if (!x || !y || !aligned(x, 16)) return QK_EINVAL_PTR;
    const bool f16 = (flags & QK_Y_F16) != 0;
    if (!aligned(y, f16 ? 2 : 4)) return QK_EINVAL_PTR;
    const int64_t n = N * ncols, ybytes = (f16 ? 2 : 4) * n;
    if (overlap(y, ybytes, W, N * row_bytes_of(type, K)) || overlap(y, ybytes, x, 2 * K * ncols))
        return QK_EINVAL_PTR;
    if (res) {
        if (!aligned(res, 4)) return QK_EINVAL_PTR;
        if (!(res == y && !f16) && overlap(res, 4 * n, y, ybytes)) return QK_EINVAL_PTR;
    }
    return QK_OK;
}

int gemv_launch(int type, const void *W, const void *W2, const void *x, void *y, int64_t N, int64_t K,
                int ncols, const void *residual, int flags, void *stream) {
    const qk::Epilogue ep{W2, (const float *)residual, (flags & QK_Y_F16) ? 1 : 0};
    hipStream_t st = (hipStream_t)stream;
    if (ncols == 1) return launched(qk::launch_gemv1(type, W, x, y, N, K, ep, st));
    return launched(qk::launch_gemv_multi(type, W, x, y, N, K, ncols, ep, st));
}

int launched(hipError_t e) {
    if (e == hipSuccess) return QK_OK;
    snprintf(g_launch_msg, sizeof g_launch_msg, "launch failed: %s", hipGetErrorString(e));
    return QK_ELAUNCH;
}

// ---- the attention side

bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

// A view of rows x heads x D elements: pointer, alignment, strides, and the
// range of bytes it spans.
struct Span {
    const void *p;
    int64_t n;
};
int check_heads(const qk_heads *x, int64_t rows, int64_t heads, int64_t D, bool output, Span *span) {
    if (x->f16 != 0 && x->f16 != 1) return QK_EINVAL_TYPE;
    if (!x->p || !aligned(x->p, x->f16 ? 2 : 4)) return QK_EINVAL_PTR;
    const int64_t size[3] = {rows, heads, D}, stride[3] = {x->row, x->head, x->elem};
    int64_t last = 0, ext;
    for (int i = 0; i < 3; ++i) {
        if (stride[i] < 0 || !mul_ok(size[i] - 1, stride[i], &ext) || __builtin_add_overflow(last, ext, &last))
            return QK_EINVAL_SHAPE;
    }
    if (last > (INT64_MAX >> 3)) return QK_EINVAL_SHAPE;
    if (output) {  // elements of their own: sorted by stride, each past the extent of the smaller ones
        int o[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (stride[o[j]] < stride[o[i]]) { const int t = o[i]; o[i] = o[j]; o[j] = t; }
        int64_t reach = 0;
        for (int i = 0; i < 3; ++i) {
            if (size[o[i]] == 1) continue;
            if (stride[o[i]] <= reach) return QK_EINVAL_SHAPE;
            reach += (size[o[i]] - 1) * stride[o[i]];
        }
    }
    *span = Span{x->p, (last + 1) * (x->f16 ? 2 : 4)};
    return QK_OK;
}

bool same_view(const qk_heads *a, const qk_heads *b) {
    return a->p == b->p && a->row == b->row && a->head == b->head && a->elem == b->elem && a->f16 == b->f16;
}

bool spans_meet(const Span &a, const Span &b) { return a.p && b.p && overlap(a.p, a.n, b.p, b.n); }

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

int check_rope(const qk_rope *r, int64_t rows, int D, bool need_positions, Span *in, int *nin) {
    if (r->rot_dim < 0 || r->rot_dim > D || (r->rot_dim & 1)) return QK_EINVAL_SHAPE;
    if (!(r->eps >= 0.f) || !isfinite(r->eps)) return QK_EINVAL_SHAPE;
    if (r->interleaved != 0 && r->interleaved != 1) return QK_EINVAL_FLAGS;
    if (r->rot_dim && (!r->inv_freq || (need_positions && !r->positions))) return QK_EINVAL_PTR;
    const Span s[4] = {{r->q_norm, 4 * D}, {r->k_norm, 4 * D}, {r->inv_freq, 2 * r->rot_dim}, {r->positions, 4 * rows}};
    for (const Span &x : s) {
        if (x.p && !aligned(x.p, 4)) return QK_EINVAL_PTR;
        in[(*nin)++] = x;
    }
    return QK_OK;
}

// Sizes of the cache and of the call's rows (host values only).
int check_cache(const qk_kv_cache *c, const qk_kv_seqs *q) {
    if (!c || !q) return QK_EINVAL_PTR;
    if (qk_kv_page_bytes(c->head_dim, c->n_kv_heads, c->page_size) < 0) return QK_EINVAL_SHAPE;
    if (c->num_pages < 1 || c->num_pages > INT32_MAX) return QK_EINVAL_SHAPE;
    if (q->rows < 0 || q->rows > 1 << 22 || q->nseq < 1 || q->nseq > 65536 || q->max_pages < 1) return QK_EINVAL_SHAPE;
    if ((int64_t)q->max_pages * c->page_size > (int64_t)1 << 30) return QK_EINVAL_SHAPE;
    if (!q->q_start && q->rows % q->nseq) return QK_EINVAL_SHAPE;
    return QK_OK;
}
// ... and its pointers; adds what the call reads to `in`.
int check_cache_ptrs(const qk_kv_cache *c, const qk_kv_seqs *q, Span *pool, Span *in, int *nin) {
    if (!c->pool || !aligned(c->pool, 16) || !q->kv_len || !q->pages) return QK_EINVAL_PTR;
    if (!aligned(q->kv_len, 4) || !aligned(q->pages, 4) || !aligned(q->q_start, 4)) return QK_EINVAL_PTR;
    *pool = Span{c->pool, c->num_pages * qk_kv_page_bytes(c->head_dim, c->n_kv_heads, c->page_size)};
    in[(*nin)++] = Span{q->q_start, 4 * ((int64_t)q->nseq + 1)};
    in[(*nin)++] = Span{q->kv_len, 4 * (int64_t)q->nseq};
    in[(*nin)++] = Span{q->pages, 4 * (int64_t)q->nseq * q->max_pages};
    return QK_OK;
}

int log2_of(int v) {
    int n = 0;
    while (1 << n < v) ++n;
    return n;
}

// (the stride of a dimension of size 1 says nothing: 0)
qk::Heads to_heads(const qk_heads *x, int64_t rows, int64_t heads) {
    if (!x) return qk::Heads{nullptr, 0, 0, 0, 0};
    return qk::Heads{x->p, rows == 1 ? 0 : x->row, heads == 1 ? 0 : x->head, x->elem, x->f16};
}
qk::KvCache to_cache(const qk_kv_cache *c) {
    return qk::KvCache{(uint8_t *)c->pool, c->num_pages, c->n_kv_heads, c->head_dim, log2_of(c->page_size)};
}
qk::KvSeqs to_seqs(const qk_kv_seqs *q) {
    return qk::KvSeqs{q->rows, q->nseq, q->max_pages, q->q_start, q->kv_len, q->pages};
}
qk::RowPrep to_prep(const qk_rope *r) {
    if (!r) return qk::RowPrep{nullptr, nullptr, nullptr, nullptr, 0.f, 0, 0};
    return qk::RowPrep{r->q_norm, r->k_norm, r->inv_freq, r->positions, r->eps, r->rot_dim, r->interleaved};
}

constexpr int MAX_HEADS = 4096;
// Grids stay below 2^32 threads: rows of heads take a wave each at most; an
// attention tile has 8 row-heads or more but for a sequence's last, and at most
// 512 threads.
constexpr int64_t MAX_ROW_HEADS = (int64_t)1 << 25;
constexpr int64_t MAX_SEQ_HEADS = (int64_t)1 << 21;  // sequences with rows x KV heads (attention)

// ---- the rest of a token

// An output's span against the inputs' (an input of the same view and type is
// its own: in place).
struct View {
    const qk_heads *x;
    Span s;
};
bool meets_another(const View &out, const View *in, int nin) {
    for (int i = 0; i < nin; ++i)
        if (!(in[i].x && same_view(out.x, in[i].x)) && spans_meet(out.s, in[i].s)) return true;
    return false;
}

// Sequences of a layer with a state (host values), then their pointers.
int check_state_seqs(const qk_state_seqs *q, int64_t num_slots) {
    if (q->rows < 0 || q->rows > 1 << 22 || q->nseq < 1 || q->nseq > 65536) return QK_EINVAL_SHAPE;
    if (!q->q_start && q->rows % q->nseq) return QK_EINVAL_SHAPE;
    if (num_slots < 1 || num_slots > INT32_MAX) return QK_EINVAL_SHAPE;
    return QK_OK;
}
int check_state_ptrs(const qk_state_seqs *q, Span *in, int *nin) {
    if (!q->slots) return QK_EINVAL_PTR;
    const int64_t n = 4 * (int64_t)q->nseq;
    const Span s[5] = {{q->q_start, n + 4}, {q->slots, n}, {q->slots_out, n}, {q->kv_len, n}, {q->commit, n}};
    for (const Span &x : s) {
        if (!aligned(x.p, 4)) return QK_EINVAL_PTR;
        in[(*nin)++] = x;
    }
    return QK_OK;
}
qk::StateSeqs to_state_seqs(const qk_state_seqs *q, int64_t num_slots) {
    return qk::StateSeqs{q->rows, q->nseq, q->q_start, q->slots, q->slots_out, q->kv_len, q->commit, num_slots};
}

int check_delta(const qk_delta *d, const qk_state_seqs *q) {
    if (!d || !q) return QK_EINVAL_PTR;
    if (d->k_heads < 1 || d->v_heads < 1 || d->k_heads > MAX_HEADS || d->v_heads > MAX_HEADS || d->v_heads % d->k_heads)
        return QK_EINVAL_SHAPE;
    if ((d->key_dim != 64 && d->key_dim != 128) || d->value_dim < 32 || d->value_dim > 512 || d->value_dim % 32)
        return QK_EINVAL_SHAPE;
    const int rc = check_state_seqs(q, d->num_slots);
    if (rc) return rc;
    // (16 lanes a column of a state: a grid stays below 2^32 threads)
    if ((int64_t)q->nseq * d->v_heads * d->value_dim > (int64_t)1 << 27) return QK_EINVAL_SHAPE;
    return (int64_t)q->rows * d->v_heads > MAX_ROW_HEADS ? QK_EINVAL_SHAPE : QK_OK;
}
qk::DeltaState to_delta(const qk_delta *d) {
    return qk::DeltaState{d->pool, d->k_heads, d->v_heads, d->key_dim, d->value_dim};
}

int check_probs(const qk_heads *z, int rows, int64_t vocab, int top) {
    if (!z) return QK_EINVAL_PTR;
    if (rows < 0 || rows > 1 << 22 || vocab < 1 || vocab > (int64_t)1 << 30 || top < 0 || top > 64) return QK_EINVAL_SHAPE;
    return QK_OK;
}
qk::Probs to_probs(const qk_heads *z, int rows, int64_t vocab, float scale, const qk_probs *o, int top) {
    qk::Probs p{to_heads(z, rows, 1), rows, (int)vocab, 0, top, scale, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    if (o) {
        p.ntok = o->ntok;
        p.tokens = o->tokens;
        p.token_lp = o->token_lp;
        p.lse = o->lse;
        p.entropy = o->entropy;
        p.top_lp = o->top_lp;
        p.top_ids = o->top_ids;
    }
    return p;
}

}  // namespace

extern "C" {

int qk_block_bytes(int type) { return block_bytes(type); }

int64_t qk_row_bytes(int type, int64_t K) { return row_bytes_of(type, K); }

int qk_gemv(int type, const void *W, const void *x, void *y, int64_t N, int64_t K, int ncols, void *stream) {
    return qk_gemv_ex(type, W, x, y, N, K, ncols, nullptr, 0, stream);
}

int qk_gemv_ex(int type, const void *W, const void *x, void *y, int64_t N, int64_t K, int ncols,
               const void *residual, int flags, void *stream) {
    int rc = check_shape(type, N, K, ncols);
    if (rc) return rc;
    if (flags & ~QK_Y_F16) return QK_EINVAL_FLAGS;
    if (!W || !aligned(W, 16)) return QK_EINVAL_PTR;
    if ((rc = check_io(type, W, x, y, residual, N, K, ncols, flags))) return rc;
    return gemv_launch(type, W, nullptr, x, y, N, K, ncols, residual, flags, stream);
}

int qk_gemv_swiglu(int type, const void *Wg, const void *Wu, const void *x, void *y, int64_t N, int64_t K,
                   int ncols, int flags, void *stream) {
    int rc = check_shape(type, N, K, ncols);
    if (rc) return rc;
    if (flags & ~QK_Y_F16) return QK_EINVAL_FLAGS;
    if (!Wg || !Wu || !aligned(Wg, 16) || !aligned(Wu, 16)) return QK_EINVAL_PTR;
    if ((rc = check_io(type, Wg, x, y, nullptr, N, K, ncols, flags))) return rc;
    if (overlap(y, ((flags & QK_Y_F16) ? 2 : 4) * N * ncols, Wu, N * row_bytes_of(type, K))) return QK_EINVAL_PTR;
    return gemv_launch(type, Wg, Wu, x, y, N, K, ncols, nullptr, flags, stream);
}

int qk_gemv_batch(const qk_gemv_item *items, int count, void *stream) {
    if (!items || count < 1 || count > QK_MAX_BATCH || count > qk::MAX_BATCH) return QK_EINVAL_SHAPE;
    qk::BatchEntry e[qk::MAX_BATCH];
    for (int i = 0; i < count; ++i) {
        const qk_gemv_item &it = items[i];
        const int rc = check_shape(it.type, it.N, it.K, 1);
        if (rc) return rc;
        if (!it.W || !it.x || !it.y || !aligned(it.W, 16) || !aligned(it.x, 16) || !aligned(it.y, 4))
            return QK_EINVAL_PTR;
        e[i] = qk::BatchEntry{it.type, it.W, it.x, it.y, it.N, it.K};
    }
    // the entries run concurrently: no y may overlap any entry's W, x or y
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j) {
            const qk_gemv_item &a = items[i], &b = items[j];
            if (overlap(a.y, 4 * a.N, b.W, b.N * row_bytes_of(b.type, b.K)) || overlap(a.y, 4 * a.N, b.x, 2 * b.K) ||
                (i != j && overlap(a.y, 4 * a.N, b.y, 4 * b.N)))
                return QK_EINVAL_PTR;
        }
    return launched(qk::launch_gemv_batch(e, count, (hipStream_t)stream));
}

int64_t qk_chain_plan_bytes(int nsteps, int nentries) {
    if (nsteps < 1 || nentries < nsteps) return -1;
    return qk::chain_plan_bytes(nsteps, nentries);
}

int qk_chain_plan(const qk_chain_entry *entries, int nentries, const int *step_sizes, int nsteps, void *plan,
                  int64_t plan_bytes) {
    if (!entries || !step_sizes || nsteps < 1 || nentries < nsteps) return QK_EINVAL_SHAPE;
    if (!plan || plan_bytes < qk::chain_plan_bytes(nsteps, nentries)) return QK_EINVAL_SHAPE;
    static_assert(sizeof(qk_chain_entry) == 64, "qk_chain_entry layout");
    int sum = 0;
    for (int s = 0; s < nsteps; ++s) {
        if (step_sizes[s] < 1 || step_sizes[s] > QK_MAX_BATCH) return QK_EINVAL_SHAPE;
        sum += step_sizes[s];
    }
    if (sum != nentries) return QK_EINVAL_SHAPE;
    // each entry as qk_gemv_ex / qk_gemv_swiglu with one column
    for (int i = 0; i < nentries; ++i) {
        const qk_chain_entry &e = entries[i];
        int rc = check_shape(e.type, e.N, e.K, 1);
        if (rc) return rc;
        if (e.flags & ~QK_Y_F16) return QK_EINVAL_FLAGS;
        if (e.W2 && (e.type & ~QK_PLANAR) != QK_Q4_K) return QK_EINVAL_TYPE;  // SwiGLU pairs: Q4_K
        if (e.type == QK_IQ4_XS) return QK_EINVAL_TYPE;                       // k-quants only
        if (!e.W || !aligned(e.W, 16) || (e.W2 && !aligned(e.W2, 16))) return QK_EINVAL_PTR;
        if ((rc = check_io(e.type, e.W, e.x, e.y, e.residual, e.N, e.K, 1, e.flags))) return rc;
        if (e.W2 && overlap(e.y, ((e.flags & QK_Y_F16) ? 2 : 4) * e.N, e.W2, e.N * row_bytes_of(e.type, e.K)))
            return QK_EINVAL_PTR;
    }
    // the entries of a step run concurrently: no y may overlap anything
    // another entry of the step reads or writes
    for (int s = 0, e0 = 0; s < nsteps; e0 += step_sizes[s], ++s)
        for (int i = e0; i < e0 + step_sizes[s]; ++i)
            for (int j = e0; j < e0 + step_sizes[s]; ++j) {
                if (i == j) continue;
                const qk_chain_entry &a = entries[i], &b = entries[j];
                const int64_t ya = ((a.flags & QK_Y_F16) ? 2 : 4) * a.N, yb = ((b.flags & QK_Y_F16) ? 2 : 4) * b.N;
                const int64_t wb = b.N * row_bytes_of(b.type, b.K);
                if (overlap(a.y, ya, b.W, wb) || (b.W2 && overlap(a.y, ya, b.W2, wb)) ||
                    overlap(a.y, ya, b.x, 2 * b.K) || overlap(a.y, ya, b.y, yb) ||
                    (b.residual && overlap(a.y, ya, b.residual, 4 * b.N)))
                    return QK_EINVAL_PTR;
            }
    qk::ChainEntryIn in_stack[64];
    qk::ChainEntryIn *in = nentries <= 64 ? in_stack : new (std::nothrow) qk::ChainEntryIn[nentries];
    if (!in) return QK_ELAUNCH;
    for (int i = 0; i < nentries; ++i) {
        const qk_chain_entry &e = entries[i];
        in[i] = qk::ChainEntryIn{e.type, (e.flags & QK_Y_F16) ? 1 : 0, e.W, e.W2, e.x, e.y, e.residual, e.N, e.K,
                                 row_bytes_of(e.type, e.K)};
    }
    const hipError_t err = qk::chain_plan(in, nentries, step_sizes, nsteps, plan, plan_bytes);
    if (in != in_stack) delete[] in;
    return err == hipSuccess ? QK_OK : QK_EINVAL_SHAPE;
}

int64_t qk_chain_workspace_bytes(int nsteps) {
    if (nsteps < 1) return -1;
    return ((int64_t)(nsteps + 2) * 4 + 255) / 256 * 256;
}

int qk_gemv_chain(const void *plan, const void *plan_dev, void *workspace, int64_t workspace_bytes,
                  int64_t timeout_us, void *stream) {
    if (!plan || !plan_dev || !workspace || !aligned(plan_dev, 16) || !aligned(workspace, 4)) return QK_EINVAL_PTR;
    const int nsteps = qk::chain_steps(plan);
    if (nsteps < 1) return QK_EINVAL_SHAPE;
    if (workspace_bytes < qk_chain_workspace_bytes(nsteps)) return QK_EINVAL_SHAPE;
    const hipError_t e = qk::launch_chain(plan, plan_dev, static_cast<uint32_t *>(workspace), workspace_bytes / 4,
                                          timeout_us, (hipStream_t)stream);
    if (e == hipSuccess) return QK_OK;
    snprintf(g_launch_msg, sizeof g_launch_msg, "launch failed (%s): %s", qk::chain_stage(), hipGetErrorString(e));
    return QK_ELAUNCH;
}

int qk_gemv_chain_noalloc(const void *plan, const void *plan_dev, void *status, int64_t timeout_us, void *stream) {
    static_assert(QK_CHAIN_NOALLOC_MAX_STEPS + 2 <= qk::CHAIN_SCRATCH_WORDS, "chain scratch size");
    if (!plan || !plan_dev || !aligned(plan_dev, 16) || !aligned(status, 4)) return QK_EINVAL_PTR;
    const int nsteps = qk::chain_steps(plan);
    if (nsteps < 1 || nsteps > QK_CHAIN_NOALLOC_MAX_STEPS) return QK_EINVAL_SHAPE;
    const hipError_t e = qk::launch_chain_noalloc(plan, plan_dev, status, timeout_us, (hipStream_t)stream);
    if (e == hipSuccess) return QK_OK;
    snprintf(g_launch_msg, sizeof g_launch_msg, "launch failed (%s): %s", qk::chain_stage(), hipGetErrorString(e));
    return QK_ELAUNCH;
}

int qk_dequant(int type, const void *W, void *out, int64_t N, int64_t K, void *stream) {
    const int rc = check_shape(type, N, K, 1);
    if (rc) return rc;
    if (!W || !out || !aligned(W, 16) || !aligned(out, 4)) return QK_EINVAL_PTR;
    if (overlap(out, 4 * N * K, W, N * row_bytes_of(type, K))) return QK_EINVAL_PTR;
    return launched(qk::launch_dequant(type, W, out, N, K, (hipStream_t)stream));
}

int qk_repack(int type, const void *W, void *Wp, int64_t N, int64_t K, void *stream) {
    if ((type & QK_PLANAR) || type == QK_IQ4_XS) return QK_EINVAL_TYPE;
    const int rc = check_shape(type, N, K, 1);
    if (rc) return rc;
    if (!W || !Wp || !aligned(W, 16) || !aligned(Wp, 16)) return QK_EINVAL_PTR;
    const uintptr_t a0 = (uintptr_t)W, a1 = a0 + (uintptr_t)(N * row_bytes_of(type, K));
    const uintptr_t b0 = (uintptr_t)Wp, b1 = b0 + (uintptr_t)(N * row_bytes_of(type | QK_PLANAR, K));
    if (a0 < b1 && b0 < a1) return QK_EINVAL_PTR;
    return launched(qk::launch_repack(type, W, Wp, N, K, (hipStream_t)stream));
}

int64_t qk_kv_page_bytes(int head_dim, int n_kv_heads, int page_size) {
    if (!head_dim_ok(head_dim) || n_kv_heads < 1 || n_kv_heads > MAX_HEADS) return -1;
    if (page_size < 32 || page_size > 1024 || (page_size & (page_size - 1))) return -1;
    return qk::kv_page_bytes(head_dim, n_kv_heads, page_size);
}

int qk_norm_rope(const qk_rope *rope, int rows, int head_dim, int n_heads, const qk_heads *q, const qk_heads *q_out,
                 int n_kv_heads, const qk_heads *k, const qk_heads *k_out, void *stream) {
    if (!rope || !q != !q_out || !k != !k_out || (!q && !k)) return QK_EINVAL_PTR;
    if (!head_dim_ok(head_dim) || rows < 0 || rows > 1 << 22) return QK_EINVAL_SHAPE;
    const int hq = q ? n_heads : 0, hk = k ? n_kv_heads : 0;
    if ((q && (hq < 1 || hq > MAX_HEADS)) || (k && (hk < 1 || hk > MAX_HEADS))) return QK_EINVAL_SHAPE;
    if ((int64_t)rows * (hq + hk) > MAX_ROW_HEADS) return QK_EINVAL_SHAPE;
    if (rows == 0) return QK_OK;
    Span in[8];
    int nin = 0, rc;
    if ((rc = check_rope(rope, rows, head_dim, true, in, &nin))) return rc;
    Span sq{}, sqo{}, sk{}, sko{};
    if (q && ((rc = check_heads(q, rows, hq, head_dim, false, &sq)) || (rc = check_heads(q_out, rows, hq, head_dim, true, &sqo))))
        return rc;
    if (k && ((rc = check_heads(k, rows, hk, head_dim, false, &sk)) || (rc = check_heads(k_out, rows, hk, head_dim, true, &sko))))
        return rc;
    if ((q && !same_view(q, q_out) && spans_meet(sqo, sq)) || (k && !same_view(k, k_out) && spans_meet(sko, sk)) ||
        spans_meet(sqo, sk) || spans_meet(sko, sq) || spans_meet(sqo, sko))
        return QK_EINVAL_PTR;
    for (int i = 0; i < nin; ++i)
        if (spans_meet(sqo, in[i]) || spans_meet(sko, in[i])) return QK_EINVAL_PTR;
    const qk::KvSeqs seqs{rows, 1, 0, nullptr, nullptr, nullptr};
    return launched(qk::launch_kv_rows(nullptr, seqs, to_prep(rope), head_dim, hq, to_heads(q, rows, hq),
                                       to_heads(q_out, rows, hq), hk, to_heads(k, rows, hk), to_heads(nullptr, 0, 0),
                                       to_heads(k_out, rows, hk), (hipStream_t)stream));
}

int qk_kv_append(const qk_kv_cache *cache, const qk_kv_seqs *seqs, const qk_rope *rope, const qk_heads *k,
                 const qk_heads *v, int n_heads, const qk_heads *q, const qk_heads *q_out, void *stream) {
    int rc = check_cache(cache, seqs);
    if (rc) return rc;
    if (!k || !v || !q != !q_out) return QK_EINVAL_PTR;
    const int D = cache->head_dim, hk = cache->n_kv_heads, hq = q ? n_heads : 0, rows = seqs->rows;
    if (q && (hq < 1 || hq > MAX_HEADS)) return QK_EINVAL_SHAPE;
    if ((int64_t)rows * (hq + 2 * hk) > MAX_ROW_HEADS) return QK_EINVAL_SHAPE;
    if (rows == 0) return QK_OK;
    Span in[12], pool, sk, sv, sq{}, sqo{};
    int nin = 0;
    if ((rc = check_cache_ptrs(cache, seqs, &pool, in, &nin))) return rc;
    if (rope && (rc = check_rope(rope, rows, D, false, in, &nin))) return rc;
    if ((rc = check_heads(k, rows, hk, D, false, &sk)) || (rc = check_heads(v, rows, hk, D, false, &sv))) return rc;
    if (q && ((rc = check_heads(q, rows, hq, D, false, &sq)) || (rc = check_heads(q_out, rows, hq, D, true, &sqo))))
        return rc;
    in[nin++] = sk;
    in[nin++] = sv;
    for (int i = 0; i < nin; ++i)
        if (spans_meet(pool, in[i]) || spans_meet(sqo, in[i])) return QK_EINVAL_PTR;
    if (spans_meet(pool, sq) || spans_meet(pool, sqo) || (q && !same_view(q, q_out) && spans_meet(sqo, sq)))
        return QK_EINVAL_PTR;
    const qk::KvCache c = to_cache(cache);
    return launched(qk::launch_kv_rows(&c, to_seqs(seqs), to_prep(rope), D, hq, to_heads(q, rows, hq),
                                       to_heads(q_out, rows, hq), hk, to_heads(k, rows, hk), to_heads(v, rows, hk),
                                       to_heads(nullptr, 0, 0), (hipStream_t)stream));
}

int qk_kv_read(const qk_kv_cache *cache, const qk_kv_seqs *seqs, const qk_heads *k_out, const qk_heads *v_out,
               void *stream) {
    int rc = check_cache(cache, seqs);
    if (rc) return rc;
    if (!k_out && !v_out) return QK_EINVAL_PTR;
    const int D = cache->head_dim, hk = cache->n_kv_heads, rows = seqs->rows;
    if ((int64_t)rows * hk > MAX_ROW_HEADS) return QK_EINVAL_SHAPE;
    if (rows == 0) return QK_OK;
    Span in[4], sk{}, sv{};
    int nin = 1;
    if ((rc = check_cache_ptrs(cache, seqs, &in[0], in, &nin))) return rc;
    if (k_out && (rc = check_heads(k_out, rows, hk, D, true, &sk))) return rc;
    if (v_out && (rc = check_heads(v_out, rows, hk, D, true, &sv))) return rc;
    for (int i = 0; i < nin; ++i)
        if (spans_meet(sk, in[i]) || spans_meet(sv, in[i])) return QK_EINVAL_PTR;
    if (spans_meet(sk, sv)) return QK_EINVAL_PTR;
    return launched(qk::launch_kv_read(to_cache(cache), to_seqs(seqs), to_heads(k_out, rows, hk), to_heads(v_out, rows, hk),
                                       (hipStream_t)stream));
}

static int check_attn(const qk_kv_cache *cache, const qk_kv_seqs *seqs, int n_heads) {
    const int rc = check_cache(cache, seqs);
    if (rc) return rc;
    if (n_heads < 1 || n_heads > MAX_HEADS || n_heads % cache->n_kv_heads) return QK_EINVAL_SHAPE;
    if ((int64_t)seqs->rows * n_heads > MAX_ROW_HEADS) return QK_EINVAL_SHAPE;
    if ((int64_t)(seqs->rows < seqs->nseq ? seqs->rows : seqs->nseq) * cache->n_kv_heads > MAX_SEQ_HEADS)
        return QK_EINVAL_SHAPE;
    return QK_OK;
}

int64_t qk_kv_attn_workspace_bytes(const qk_kv_cache *cache, const qk_kv_seqs *seqs, int n_heads) {
    if (check_attn(cache, seqs, n_heads)) return -1;
    return seqs->rows ? qk::kv_attn_workspace(to_cache(cache), to_seqs(seqs), n_heads) : 0;
}

int qk_kv_attn(const qk_kv_cache *cache, const qk_kv_seqs *seqs, int n_heads, const qk_heads *q, const qk_heads *out,
               float scale, int window, void *workspace, int64_t workspace_bytes, void *stream) {
    int rc = check_attn(cache, seqs, n_heads);
    if (rc) return rc;
    if (!(fabsf(scale) <= 0x1p64f) || window < 0) return QK_EINVAL_SHAPE;
    if (!q || !out) return QK_EINVAL_PTR;
    if (q->f16 != 1) return QK_EINVAL_TYPE;
    const int rows = seqs->rows, D = cache->head_dim;
    if (rows == 0) return QK_OK;
    Span in[8], so, sq;
    int nin = 1;
    if ((rc = check_cache_ptrs(cache, seqs, &in[0], in, &nin))) return rc;
    if ((rc = check_heads(q, rows, n_heads, D, false, &sq)) || (rc = check_heads(out, rows, n_heads, D, true, &so)))
        return rc;
    in[nin++] = sq;
    const qk::KvCache c = to_cache(cache);
    const qk::KvSeqs sqs = to_seqs(seqs);
    const int64_t need = qk::kv_attn_workspace(c, sqs, n_heads);
    if (workspace_bytes < need) return QK_EINVAL_SHAPE;
    if (need && (!workspace || !aligned(workspace, 16))) return QK_EINVAL_PTR;
    const Span ws{need ? workspace : nullptr, need};
    for (int i = 0; i < nin; ++i)
        if (spans_meet(so, in[i]) || spans_meet(ws, in[i])) return QK_EINVAL_PTR;
    if (spans_meet(so, ws)) return QK_EINVAL_PTR;
    return launched(qk::launch_kv_attn(c, sqs, n_heads, to_heads(q, rows, n_heads), to_heads(out, rows, n_heads), scale, window, workspace,
                                       (hipStream_t)stream));
}

int qk_block_norm(const qk_block *b, int rows, int groups, int dim, const qk_heads *y, const qk_heads *gate,
                  const qk_heads *residual, const qk_heads *h_out, const qk_heads *x_out, void *stream) {
    if (!b || !y || (!h_out && !x_out)) return QK_EINVAL_PTR;
    if (rows < 0 || rows > 1 << 22 || groups < 1 || groups > MAX_HEADS || dim < 1 || dim > 32768) return QK_EINVAL_SHAPE;
    if ((int64_t)rows * groups > MAX_ROW_HEADS) return QK_EINVAL_SHAPE;
    if (!(b->eps >= 0.f) || !isfinite(b->eps) || !isfinite(b->scale)) return QK_EINVAL_SHAPE;
    if (b->act != QK_ACT_NONE && b->act != QK_ACT_SILU && b->act != QK_ACT_SIGMOID) return QK_EINVAL_FLAGS;
    if (rows == 0) return QK_OK;
    if (!aligned(b->post_norm, 4) || !aligned(b->pre_norm, 4)) return QK_EINVAL_PTR;
    View in[5] = {{nullptr, {b->post_norm, 4 * (int64_t)dim}}, {nullptr, {b->pre_norm, 4 * (int64_t)dim}}}, h{}, x{};
    int nin = 2, rc;
    for (const qk_heads *v : {y, gate, residual}) {
        if (!v) continue;
        in[nin].x = v;
        if ((rc = check_heads(v, rows, groups, dim, false, &in[nin++].s))) return rc;
    }
    h.x = h_out;
    x.x = x_out;
    if (h_out && (rc = check_heads(h_out, rows, groups, dim, true, &h.s))) return rc;
    if (x_out && (rc = check_heads(x_out, rows, groups, dim, true, &x.s))) return rc;
    if ((h_out && meets_another(h, in, nin)) || (x_out && meets_another(x, in, nin)) || spans_meet(h.s, x.s))
        return QK_EINVAL_PTR;
    const qk::BlockNorm bn{b->post_norm, b->pre_norm, b->eps, b->scale, b->act};
    return launched(qk::launch_block_norm(bn, rows, groups, dim, to_heads(y, rows, groups), to_heads(gate, rows, groups),
                                          to_heads(residual, rows, groups), to_heads(h_out, rows, groups),
                                          to_heads(x_out, rows, groups), (hipStream_t)stream));
}

int qk_conv_silu(const qk_conv *c, const qk_state_seqs *seqs, int act, const qk_heads *x, const qk_heads *y,
                 void *stream) {
    if (!c || !seqs || !x) return QK_EINVAL_PTR;
    if (c->channels < 1 || c->channels > 65536 || c->taps < 2 || c->taps > 8) return QK_EINVAL_SHAPE;
    int rc = check_state_seqs(seqs, c->num_slots);
    if (rc) return rc;
    if (act != QK_ACT_NONE && act != QK_ACT_SILU) return QK_EINVAL_FLAGS;
    const int rows = seqs->rows;
    if (rows == 0) return QK_OK;
    Span in[8], pool, sy{};
    int nin = 0;
    if (!c->pool || !aligned(c->pool, 16) || !c->weight || !aligned(c->weight, 4) || !aligned(c->bias, 4)) return QK_EINVAL_PTR;
    pool = Span{c->pool, c->num_slots * (c->taps - 1) * c->channels * 4};
    in[nin++] = Span{c->weight, 4 * (int64_t)c->channels * c->taps};
    in[nin++] = Span{c->bias, 4 * (int64_t)c->channels};
    if ((rc = check_state_ptrs(seqs, in, &nin))) return rc;
    if ((rc = check_heads(x, rows, 1, c->channels, false, &in[nin++]))) return rc;
    if (y && (rc = check_heads(y, rows, 1, c->channels, true, &sy))) return rc;
    for (int i = 0; i < nin; ++i)
        if (spans_meet(pool, in[i]) || spans_meet(sy, in[i])) return QK_EINVAL_PTR;
    if (spans_meet(pool, sy)) return QK_EINVAL_PTR;
    const qk::ConvState cs{c->pool, c->channels, c->taps, c->weight, c->bias};
    return launched(qk::launch_conv(to_state_seqs(seqs, c->num_slots), cs, act == QK_ACT_SILU, to_heads(x, rows, 1),
                                    to_heads(y, rows, 1), (hipStream_t)stream));
}

int64_t qk_delta_workspace_bytes(const qk_delta *delta, const qk_state_seqs *seqs) {
    if (check_delta(delta, seqs)) return -1;
    return seqs->rows ? qk::delta_workspace(to_state_seqs(seqs, delta->num_slots), to_delta(delta), true, true) : 0;
}

int qk_delta_rule(const qk_delta *d, const qk_state_seqs *seqs, const qk_delta_rows *r, const qk_heads *out,
                  void *workspace, int64_t workspace_bytes, void *stream) {
    int rc = check_delta(d, seqs);
    if (rc) return rc;
    if (!r) return QK_EINVAL_PTR;
    if (!(r->eps >= 0.f && r->eps <= 0x1p126f) || !isfinite(r->scale)) return QK_EINVAL_SHAPE;  // (a row's sum and eps: below 2^127)
    if (r->norm != 0 && r->norm != 1) return QK_EINVAL_FLAGS;
    const int rows = seqs->rows, hk = d->k_heads, hv = d->v_heads;
    if (rows == 0) return QK_OK;
    if (!d->pool || !aligned(d->pool, 16) || !aligned(r->A, 4) || !aligned(r->dt_bias, 4) || (r->dt_bias && !r->A))
        return QK_EINVAL_PTR;
    const Span pool{d->pool, d->num_slots * hv * d->value_dim * d->key_dim * 4};
    Span in[12], so{};
    int nin = 0;
    in[nin++] = Span{r->A, 4 * (int64_t)hv};
    in[nin++] = Span{r->dt_bias, 4 * (int64_t)hv};
    if ((rc = check_state_ptrs(seqs, in, &nin))) return rc;
    if ((rc = check_heads(&r->q, rows, hk, d->key_dim, false, &in[nin++])) ||
        (rc = check_heads(&r->k, rows, hk, d->key_dim, false, &in[nin++])) ||
        (rc = check_heads(&r->v, rows, hv, d->value_dim, false, &in[nin++])) ||
        (rc = check_heads(&r->alpha, rows, hv, 1, false, &in[nin++])) ||
        (rc = check_heads(&r->beta, rows, hv, 1, false, &in[nin++])))
        return rc;
    if (out && (rc = check_heads(out, rows, hv, d->value_dim, true, &so))) return rc;
    const qk::StateSeqs sq = to_state_seqs(seqs, d->num_slots);
    const int64_t need = qk::delta_workspace(sq, to_delta(d), r->norm, r->A);
    if (workspace_bytes < need) return QK_EINVAL_SHAPE;
    if (need && (!workspace || !aligned(workspace, 16))) return QK_EINVAL_PTR;
    const Span ws{need ? workspace : nullptr, need};
    for (int i = 0; i < nin; ++i)
        if (spans_meet(pool, in[i]) || spans_meet(so, in[i]) || spans_meet(ws, in[i])) return QK_EINVAL_PTR;
    if (spans_meet(pool, so) || spans_meet(pool, ws) || spans_meet(so, ws)) return QK_EINVAL_PTR;
    const qk::DeltaIn di{to_heads(&r->q, rows, hk), to_heads(&r->k, rows, hk), to_heads(&r->v, rows, hv),
                         to_heads(&r->alpha, rows, hv), to_heads(&r->beta, rows, hv), r->A, r->dt_bias, r->norm, r->eps,
                         r->scale};
    return launched(qk::launch_delta(sq, to_delta(d), di, to_heads(out, rows, hv), workspace, (hipStream_t)stream));
}

int64_t qk_logprobs_workspace_bytes(const qk_heads *logits, int rows, int64_t vocab, int top) {
    if (check_probs(logits, rows, vocab, top)) return -1;
    return rows ? qk::probs_workspace(to_probs(logits, rows, vocab, 1.f, nullptr, top)) : 0;
}

int qk_logprobs(const qk_heads *logits, int rows, int64_t vocab, float scale, const qk_probs *o, void *workspace,
                int64_t workspace_bytes, void *stream) {
    if (!o) return QK_EINVAL_PTR;
    int rc = check_probs(logits, rows, vocab, o->top);
    if (rc) return rc;
    if (!(scale > 0.f && scale <= 0x1p64f) || o->ntok < 0 || o->ntok > 1024) return QK_EINVAL_SHAPE;
    if (rows == 0) return QK_OK;
    if (!o->ntok != !o->tokens || !o->ntok != !o->token_lp || !o->top != !o->top_ids || !o->top != !o->top_lp)
        return QK_EINVAL_PTR;
    if (!o->ntok && !o->top && !o->lse && !o->entropy) return QK_EINVAL_PTR;
    Span in[2] = {{o->tokens, 4 * (int64_t)rows * o->ntok}, {}};
    if ((rc = check_heads(logits, rows, 1, vocab, false, &in[1]))) return rc;
    const qk::Probs p = to_probs(logits, rows, vocab, scale, o, o->top);
    const int64_t need = qk::probs_workspace(p);
    if (workspace_bytes < need) return QK_EINVAL_SHAPE;
    if (need && (!workspace || !aligned(workspace, 16))) return QK_EINVAL_PTR;
    const Span out[6] = {{o->token_lp, 4 * (int64_t)rows * o->ntok}, {o->lse, 4 * (int64_t)rows}, {o->entropy, 4 * (int64_t)rows},
                         {o->top_ids, 4 * (int64_t)rows * o->top}, {o->top_lp, 4 * (int64_t)rows * o->top},
                         {need ? workspace : nullptr, need}};
    if (!aligned(o->tokens, 4)) return QK_EINVAL_PTR;
    for (int i = 0; i < 6; ++i) {
        if (!aligned(out[i].p, 4)) return QK_EINVAL_PTR;
        for (const Span &x : in)
            if (spans_meet(out[i], x)) return QK_EINVAL_PTR;
        for (int j = 0; j < i; ++j)
            if (spans_meet(out[i], out[j])) return QK_EINVAL_PTR;
    }
    return launched(qk::launch_probs(p, workspace, (hipStream_t)stream));
}

const char *qk_strerror(int code) {
    switch (code) {
    case QK_OK: return "ok";
    case QK_EINVAL_TYPE:
        return "invalid type: expected QK_Q4_K (12), QK_Q5_K (13), QK_Q6_K (14) or QK_IQ4_XS (23); the k-quants "
               "optionally | QK_PLANAR (0x100) with ncols = 1 (qk_repack takes the type without the flag); "
               "qk_repack and chains take the k-quants only, chain SwiGLU pairs Q4_K only; heads of f16 = 0 or 1, the "
               "queries of qk_kv_attn fp16";
    case QK_EINVAL_SHAPE:
        return "invalid shape: need N >= 1, K a positive multiple of 256, 1 <= ncols <= 32; a chain needs 1.."
               "QK_MAX_BATCH entries per step, a workspace of qk_chain_workspace_bytes, and for "
               "qk_gemv_chain_noalloc at most QK_CHAIN_NOALLOC_MAX_STEPS (4094) steps; the attention side needs "
               "head_dim 64, 128 or 256, page_size a power of two in 32..1024, rows a multiple of nseq without q_start, "
               "rot_dim even and at most head_dim, query heads a multiple of the KV heads, strides >= 0 and outputs "
               "whose elements do not coincide, at most 2^25 rows x heads and 2^21 sequences x KV heads, |scale| <= 2^64, a window >= 0, a workspace of "
               "qk_kv_attn_workspace_bytes; qk_block_norm 1..4096 groups of 1..32768 and a finite scale; recurrent layers "
               "1..65536 channels, 2..8 taps, key_dim 64 or 128, value_dim a multiple of 32 in 32..512, value heads a "
               "multiple of the key heads, an eps up to 2^126, at most 2^27 sequences x value heads x value_dim, a workspace of "
               "qk_delta_workspace_bytes; qk_logprobs a vocabulary of 1..2^30, 0..1024 tokens, the top 0..64, "
               "0 < scale <= 2^64, a workspace of qk_logprobs_workspace_bytes";
    case QK_EINVAL_PTR:
        return "invalid pointer: NULL, or W/x not 16-byte aligned, or y/out/residual not 4-byte aligned (fp16 y: 2), "
               "or an output that overlaps an input (y with W or x, out with W, a batch entry's y with any entry's "
               "W, x or y, Wp with W), or a residual that overlaps y without being y (fp32 y); heads not aligned to their type, the pool or the "
               "workspace not to 16 bytes, int32 arrays not to 4";
    case QK_EINVAL_FLAGS: return "invalid flags: the only epilogue flag is QK_Y_F16 (0x1); interleaved is 0 or 1, as is "
                                 "norm of qk_delta_rule; act is a QK_ACT_* (SILU or NONE for qk_conv_silu)";
    case QK_ELAUNCH: return g_launch_msg;
    default: return "unknown error code";
    }
}

const char *qk_version(void) { return "qkgemv " QKGEMV_VERSION " gfx950"; }

}  // extern "C"
