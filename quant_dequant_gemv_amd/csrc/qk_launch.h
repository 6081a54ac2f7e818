// qk_launch.h -- internal launch entry points (C++ linkage) behind the C ABI.
// Arguments are validated by the callers in qk_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace qk {

// Host state kept per device and safe under concurrent calls from several
// threads (the C ABI's calls are thread-safe).  Devices are numbered below
// MAX_DEVICES.
constexpr int MAX_DEVICES = 64;

inline int current_device() {
    int d = 0;
    return hipGetDevice(&d) == hipSuccess && d >= 0 && d < MAX_DEVICES ? d : 0;
}

// Compute units of the current device, read once per device.
inline int device_cus() {
    static std::atomic<int> cache[MAX_DEVICES];
    const int dev = current_device();
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

// Kernel F's opt-in to `bytes` of dynamic LDS (above the default 64 KB) on
// the current device, made once per device and kernel (a racing thread may
// repeat it: harmless).
template <auto F>
inline hipError_t lds_opt_in(int bytes) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = uint64_t(1) << current_device();
    if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(F),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Layout flag carried in the type argument (QK_PLANAR of the C ABI).
constexpr int PLANAR_FLAG = 0x100;

// What happens at the store of y (a by-value kernel argument; all-zero = the
// plain GEMV): act = W x, or silu(W x) * (W2 x) when W2 is set (the up tensor,
// same type, layout and shape as W); then y = act + res when res is set (fp32
// [N][ncols], may be y itself); y is fp16 (round to nearest even) when f16.
struct Epilogue {
    const void *W2;
    const float *res;
    int f16;
};

// ncols == 1: the streaming GEMV.
hipError_t launch_gemv1(int type, const void *W, const void *x, void *y, int64_t N, int64_t K,
                        const Epilogue &ep, hipStream_t stream);

// Independent one-column GEMVs in one launch (at most MAX_BATCH).
constexpr int MAX_BATCH = 16;
struct BatchEntry {
    int type;
    const void *W;
    const void *x;
    void *y;
    int64_t N, K;
};
hipError_t launch_gemv_batch(const BatchEntry *entries, int count, hipStream_t stream);

// ncols in 2..8: the few-column verify form (matrix cores).
hipError_t launch_gemv_multi(int type, const void *W, const void *x, void *y, int64_t N, int64_t K,
                             int ncols, const Epilogue &ep, hipStream_t stream);

// Chain of one-column steps in one persistent launch (see qk_kernels.hip).
struct ChainEntryIn {
    int type, f16;
    const void *W, *W2, *x;
    void *y;
    const void *res;
    int64_t N, K, row_bytes;
};
int64_t chain_plan_bytes(int nsteps, int nentries);
hipError_t chain_plan(const ChainEntryIn *entries, int nentries, const int *step_sizes, int nsteps, void *plan,
                      int64_t bytes);
int chain_steps(const void *plan_host);  // steps of a plan, or -1 if it is not one
hipError_t launch_chain(const void *plan_host, const void *plan_dev, uint32_t *sync, int64_t sync_words,
                        int64_t timeout_us, hipStream_t stream);
const char *chain_stage();  // the step of the calling thread's last failed launch_chain
// launch_chain with the counters in the library's own per-device array of
// CHAIN_SCRATCH_WORDS words (nsteps + 2 must fit); status: NULL or a device
// word that receives the run's flag word after the chain.
constexpr int CHAIN_SCRATCH_WORDS = 4096;
hipError_t launch_chain_noalloc(const void *plan_host, const void *plan_dev, void *status, int64_t timeout_us,
                                hipStream_t stream);

// fp32 dequantisation of the whole tensor (either layout).
hipError_t launch_dequant(int type, const void *W, void *out, int64_t N, int64_t K, hipStream_t stream);

// GGUF rows -> PLANAR rows (type without the flag).
hipError_t launch_repack(int type, const void *W, void *Wp, int64_t N, int64_t K, hipStream_t stream);

// ---- the attention side (qk_kv.hip): views and arrays as in the C ABI
struct Heads {
    void *p;
    int64_t row, head, elem;
    int f16;
};
struct KvCache {
    uint8_t *pool;
    int64_t num_pages;
    int hkv, D, ps_log2;
};
struct KvSeqs {
    int rows, nseq, max_pages;
    const int32_t *q_start, *kv_len, *pages;
};
struct RowPrep {  // norm + rotation of qk_norm_rope / qk_kv_append
    const float *q_norm, *k_norm, *inv_freq;
    const int32_t *positions;
    float eps;
    int rot_dim, interleaved;
};
// Bytes of one head's keys (or values) on a page, and of a page.
constexpr int64_t kv_block_bytes(int D, int ps) { return (int64_t)ps * D / 8 * 5; }
constexpr int64_t kv_page_bytes(int D, int hkv, int ps) { return 2 * hkv * kv_block_bytes(D, ps); }

// q and k heads through norm and rotation; with a cache, k and v into it
// (k_out then unused), without one k to k_out.
hipError_t launch_kv_rows(const KvCache *cache, const KvSeqs &seqs, const RowPrep &prep, int D, int hq, const Heads &q,
                          const Heads &q_out, int hkv, const Heads &k, const Heads &v, const Heads &k_out,
                          hipStream_t stream);
hipError_t launch_kv_read(const KvCache &cache, const KvSeqs &seqs, const Heads &k_out, const Heads &v_out,
                          hipStream_t stream);
int64_t kv_attn_workspace(const KvCache &cache, const KvSeqs &seqs, int hq);
hipError_t launch_kv_attn(const KvCache &cache, const KvSeqs &seqs, int hq, const Heads &q, const Heads &out,
                          float scale, int window, void *workspace, hipStream_t stream);

// ---- the rest of a token: block norms, recurrent layers, log probabilities
struct BlockNorm {
    const float *post, *pre;  // weights of the norms (NULL: none)
    float eps, scale;
    int act;                  // of the gate: 0 none, 1 SiLU, 2 logistic
};
// h = res + scale * post-norm(y) * act(gate); x = pre-norm(h).  gate, res, h, x: p may be NULL.
hipError_t launch_block_norm(const BlockNorm &b, int rows, int groups, int dim, const Heads &y, const Heads &gate,
                             const Heads &res, const Heads &h, const Heads &x, hipStream_t stream);

// Rows of sequences that carry a state (qk_state_seqs of the C ABI).
struct StateSeqs {
    int rows, nseq;
    const int32_t *q_start, *slots, *slots_out, *kv_len, *commit;
    int64_t num_slots;
};
struct ConvState {
    float *pool;              // [slots][taps - 1][channels]
    int channels, taps;
    const float *weight, *bias;  // [channels][taps], [channels] or NULL
};
// y.p may be NULL (the state alone).
hipError_t launch_conv(const StateSeqs &q, const ConvState &c, int act, const Heads &x, const Heads &y, hipStream_t stream);

struct DeltaState {
    float *pool;              // [slots][hv][dv][dk]
    int hk, hv, dk, dv;
};
struct DeltaIn {
    Heads q, k, v, alpha, beta;
    const float *A, *dt;      // NULL: alpha is the log decay, beta the step
    int norm;
    float eps, scale;
};
// What a call that goes in tiles takes, 0 for row by row; `norm` and `raw` (gates): of rows as they may be.
int64_t delta_workspace(const StateSeqs &q, const DeltaState &d, bool norm, bool raw);
// out.p may be NULL (the state alone).
hipError_t launch_delta(const StateSeqs &q, const DeltaState &d, const DeltaIn &in, const Heads &out, void *workspace,
                        hipStream_t stream);

// Element (t, v) of the logits at p[t * row + v * elem].
struct Probs {
    Heads z;
    int rows, vocab, ntok, top;
    float scale;
    const int32_t *tokens;    // [rows][ntok]
    float *token_lp, *lse, *entropy, *top_lp;
    int32_t *top_ids;
};
int64_t probs_workspace(const Probs &p);
hipError_t launch_probs(const Probs &p, void *workspace, hipStream_t stream);

}  // namespace qk
