// qk_kv_attn.hip -- attention over the paged 4-bit cache on matrix cores.
//
// Mathematics.  With K_ji = d_jg c_ji + m_jg (g = i / 32), the score of a
// query row is sum_g d_jg (sum_{i in g} q_i c_ji) + sum_g m_jg (sum_{i in g}
// q_i).  A group's inner sum is one 16x16x32 matrix instruction of 16
// positions by 16 query rows on exact operands: a nibble shifted and masked is
// an fp16 subnormal, code * 2^-21 (or 16 times that for the odd nibbles,
// whose queries carry 1/16), so a pair of codes costs a shift and a mask at
// most and nothing is converted or rounded.  The step d is one fp32 fma per
// result.  The minima's term is one more instruction for all groups, the
// queries' group sums as two fp16 terms.
// The values likewise: O_i = sum_j (p_j d_jg) c_ji + sum_j p_j m_jg, where
// p_j d_jg goes in as two fp16 terms (product, and its residual by fma plus the
// residual of p), so a probability is not rounded to 11 bits.  Two terms end
// where fp16 does, at 2^-24, whatever they stand for: probabilities are held
// up to 2^15 (2^13 at the running maximum) and steps times a power of two that
// has the largest one met so far in [1/16, 1), so that a position 16 nats below
// the maximum still has 11 bits or more, values of any scale alike.  A long tail
// under one high score is the ordinary state of a trained model; with 1 at the
// maximum and steps as they are, 32768 positions 12 nats down with values of
// 0.02 came out wrong by more than the output.  The power is chosen at a wave's
// first tile and lowered where a later one has a larger step: a maximum and a
// branch a tile, within the spread of the cases below but for 2% at 509 rows
// under a window.  It is 1 where the first tile allows it (values of 0.02, which
// are scaled: 2..4% more at 509 rows, 2% at 48 sequences and 17 drafts).
//
// Layout.  Scores are computed transposed (positions are the rows of the
// result, query rows its columns) and so is the output (dimensions by query
// rows): a lane holds the same query row in both, the probabilities of a
// lane are the operand of the second product as they are (slot j of quad a
// is position 16 (j / 4) + 4 a + j % 4 of a tile of 32), and the softmax
// statistics are one scalar per lane.  The page layout is made for this:
// the cache's bytes go from whole pieces in memory to operands in registers;
// LDS holds the queries where registers do not (D = 256, tiles of 16 rows) and
// joins the waves at the end.
//
// Bounds and figures (device time in a graph, of the floor that the bytes set
// at 5.1 TB/s or the products at 1150 TFLOP/s):
// - D = 256, 24 heads on 4, 1 token: 262139 positions 73 us, 336 MB, floor 66:
//   memory.  32773 positions 20 us, floor 8: start, one round trip a tile and
//   the joining launch (4 us).
// - D = 128, 48 sequences of 1..16384 positions: 46 us, 135 MB, floor 26: the
//   latency of 40 KB pages in any order (a copy that only loads: 39..42 us).
// - D = 64, 509 rows under a window: 59 us, 17 GFLOP, floor 15: vector
//   instructions (63% of the issue slots; the matrix cores are busy 25%).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "qk_kv.h"

namespace qk {
namespace attn {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int MAX_SPLIT = 256;   // splits of a sequence
constexpr float M_NONE = -3e38f; // running maximum before any visible position
// Two codes in an fp16 pair, as they lie after a shift: code * 2^-21 (a
// subnormal) and, 16 times that, code * 2^-17.  The sums inside a matrix
// instruction are aligned by the operands' exponent fields, so a subnormal
// that begins k bits below its field costs k bits of the sum: in the lowest
// place (code * 2^-24) it was 2^-18 of the largest product, toward zero; here
// it is 2^-21 and less.
constexpr uint32_t EVEN = 0x00780078u, ODD = 0x07800780u;
constexpr float TOP = 13.f;      // a probability is held as 2^TOP at the running maximum ...
constexpr float GROW = 15.f;     // ... and may reach 2^GROW (fp16 ends at 2^16) before the maximum is moved
constexpr int NEAR = 3;          // largest steps in [2^-(NEAR + 1), 1) are near enough to 1 as they are

__device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return (float)__builtin_bit_cast(h2, v).x; }
__device__ __forceinline__ float hi_f(uint32_t v) { return (float)__builtin_bit_cast(h2, v).y; }
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const h2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ h2 half_pair(float v) { return h2{(_Float16)v, (_Float16)v}; }
// the larger of each half's values (NaN where one is); three operands are one instruction
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_maximum(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b)));
}
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
}
// the value of the lane 8 columns on, in a row of 16 lanes
__device__ __forceinline__ float row_half_swap(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xf, 0xf, true));
}
// N dwords from an address aligned to min(4N, 16)
template <int N> __device__ __forceinline__ void load(uint32_t *r, const uint8_t *p) {
    if constexpr (N == 1) {
        r[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const u2 v = *reinterpret_cast<const u2 *>(p);
        r[0] = v.x; r[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u4 v = *reinterpret_cast<const u4 *>(p + 4 * i);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    }
}

// Inclusive sums over the lanes of a wave (DPP: rows of 16, then across rows).
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t lanes_below(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <typename T> __device__ __forceinline__ T scan(T v) {
    auto step = [&](auto from) { v += __builtin_bit_cast(T, from(__builtin_bit_cast(uint32_t, v))); };
    step([](uint32_t w) { return lanes_below<0x111, 0xf>(w); });
    step([](uint32_t w) { return lanes_below<0x112, 0xf>(w); });
    step([](uint32_t w) { return lanes_below<0x114, 0xf>(w); });
    step([](uint32_t w) { return lanes_below<0x118, 0xf>(w); });
    step([](uint32_t w) { return lanes_below<0x142, 0xa>(w); });
    step([](uint32_t w) { return lanes_below<0x143, 0xc>(w); });
    return v;
}

// Work.  Query rows of a sequence, its heads of one KV head side by side: row
// r is token r / grp, head r % grp of the group, in tiles of RT rows.  A
// tile's positions are cut into splits of about `chunk` tiles of 32, where
// chunk shares the whole call's work out over the compute units -- from the
// lengths themselves, so neither a page table made for longer contexts nor a
// batch of unlike lengths leaves units idle (48 sequences of 1..16384
// positions: 93 us with splits cut by the table's length, 46 with this).  A work item is one
// (tile, split); a sequence's items follow those of the sequences before it,
// which every workgroup sums up for itself (SHARE).  Where tiles alone fill
// the card (target 0) nothing is split and a tile's number says where it is
// (4000 sequences of 300 positions, D = 128: 2900 us with sums, 520 without);
// a kernel of its own, as the second way cost the first 5..7% in one.
struct AttnArgs {
    KvCache c;
    KvSeqs sq;
    Heads q, out;
    int hq, grp, window;
    int target;          // items per KV head to share the work out to (0: no splits)
    int min_chunk;       // tiles of 32 positions that a split has at least
    float per_target;    // 1 / target and a little
    int nitems;          // items per KV head at most
    float scale;
    int qvec;            // query rows are whole 16-byte pieces
    float *o;            // partial outputs [item * hkv + head][RT][D]
    float2 *ml;          // running maximum and sum [item * hkv + head][RT]
};
struct Item {
    int s, j, split, ns; // sequence, tile of it, split, splits of the sequence's tiles
    int first, n, len;   // the sequence's rows in the call, and its length
    int id0;             // item of the tile's first split
};

// One wave, uniform results.  by_row: the tile `j` of sequence `want`;
// otherwise the item number `want`.  false: there is none.
template <int RT, bool SHARE> __device__ __forceinline__ bool find_item(const AttnArgs &a, int want, bool by_row, int j, int lane,
                                                            Item &it) {
    if constexpr (!SHARE) {
        // a sequence's tiles are numbered from first * grp / RT + min(s, first)
        // on, a place of its own for each without a sum: the quotient and the
        // 1 that a sequence with rows adds cover its tiles, and empty ones,
        // however many, stay within rows * grp / RT + min(nseq, rows)
        if (!a.sq.q_start) {
            it.n = a.sq.rows / a.sq.nseq;
            const int per = (it.n * a.grp + RT - 1) / RT;
            it.s = __builtin_amdgcn_readfirstlane(want / per);
            it.j = want - it.s * per;
            it.first = it.s * it.n;
        } else {
            auto base_of = [&](int s, int first) { return (int)((int64_t)first * a.grp / RT) + min(s, first); };
            auto base = [&](int s) { return base_of(s, clamp_row(a.sq, a.sq.q_start[s])); };
            it.s = __builtin_amdgcn_readfirstlane(count_while(a.sq.nseq, lane, [&](int s) { return base(s) <= want; })) - 1;
            if (it.s < 0) return false;
            it.first = __builtin_amdgcn_readfirstlane(clamp_row(a.sq, a.sq.q_start[it.s]));
            it.n = __builtin_amdgcn_readfirstlane(clamp_row(a.sq, a.sq.q_start[it.s + 1])) - it.first;
            it.j = want - base_of(it.s, it.first);
        }
        it.len = __builtin_amdgcn_readfirstlane(a.sq.kv_len[it.s]);
        // (kept in scalar registers: 20 vector registers fewer)
        for (int *f : {&it.s, &it.j, &it.first, &it.n, &it.len}) *f = __builtin_amdgcn_readfirstlane(*f);
        it.split = it.id0 = 0;
        it.ns = 1;
        return it.n > 0 && it.j >= 0 && (int64_t)it.j * RT < (int64_t)it.n * a.grp;
    }
    struct Seq { int first, n, len, tiles, span; };
    const int even = a.sq.q_start ? 0 : a.sq.rows / a.sq.nseq;
    auto seq = [&](int s0) {
        const int s = min(s0 + lane, a.sq.nseq - 1);
        Seq v;
        if (a.sq.q_start) {
            v.first = clamp_row(a.sq, a.sq.q_start[s]);
            v.n = max(clamp_row(a.sq, a.sq.q_start[s + 1]) - v.first, 0);
        } else {
            v.first = s * even;
            v.n = even;
        }
        v.len = a.sq.kv_len[s];
        v.tiles = s0 + lane < a.sq.nseq ? (int)(((int64_t)v.n * a.grp + RT - 1) / RT) : 0;
        // tiles of 32 positions that the rows of its last tile see, about
        const int64_t end = min((int64_t)v.len, (int64_t)a.sq.max_pages << a.c.ps_log2);
        const int64_t seen = a.window ? min(end, (int64_t)a.window + min(v.n, RT / a.grp + 2)) : end;
        v.span = (int)((max(seen, (int64_t)0) + 31) >> 5);
        return v;
    };
    const Seq head = seq(0);  // (read once where one round has them all)
    // the call's work in fp32, and chunk at least work / target whatever that rounds
    float work = (float)head.tiles * (float)head.span;
    for (int s0 = 64; s0 < a.sq.nseq; s0 += 64) {
        const Seq v = seq(s0);
        work += (float)v.tiles * (float)v.span;
    }
    if (a.sq.nseq > 1) work = scan(work);
    work = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, work), a.sq.nseq > 1 ? 63 : 0));
    const int chunk = max(a.min_chunk, (int)fminf(work * a.per_target, 1e9f) + 1);
    int before = 0;
    for (int s0 = 0; s0 < a.sq.nseq; s0 += 64) {
        const Seq v = s0 ? seq(s0) : head;
        const int ns = min(MAX_SPLIT, max(1, v.span / chunk + (v.span % chunk ? 1 : 0)));
        int sum = v.tiles * ns;
        if (a.sq.nseq > 1) sum = scan(sum);
        int at;
        if (by_row) {
            at = want - s0;
            if (at < 0 || at > 63) at = -1;
        } else {
            const uint64_t past = __ballot(before + sum > want);
            at = past ? __builtin_ctzll(past) : -1;
        }
        if (at >= 0) {
            it.s = s0 + at;
            it.ns = __builtin_amdgcn_readlane(ns, at);
            it.first = __builtin_amdgcn_readlane(v.first, at);
            it.n = __builtin_amdgcn_readlane(v.n, at);
            it.len = __builtin_amdgcn_readlane(v.len, at);
            const int tiles = __builtin_amdgcn_readlane(v.tiles, at);
            const int id = before + __builtin_amdgcn_readlane(sum, at) - tiles * it.ns;
            it.j = by_row ? j : (want - id) / it.ns;
            it.split = by_row ? 0 : (want - id) % it.ns;
            it.id0 = id + it.j * it.ns;
            // (always so, but for starts that decrease)
            return it.s < a.sq.nseq && it.j >= 0 && it.j < tiles && it.id0 >= 0 && it.id0 + it.ns <= a.nitems;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

__device__ __forceinline__ void store_out(const Heads &o, int64_t i, float v) {
    if (o.f16) reinterpret_cast<_Float16 *>(o.p)[i] = (_Float16)v;
    else reinterpret_cast<float *>(o.p)[i] = v;
}

// Variants.  PAIR: tiles of 8 query rows, each twice among the 16 columns --
// columns 0..7 for the lower half of the groups, 8..15 for the upper -- so a
// lane keeps the steps of half of the groups and one fma scales two.  One
// score instruction then takes 16 dimensions of group p and 16 of group
// p + G/2 (the other half's query operand is 0), two make both sums, and the
// halves are added once per tile.  Otherwise tiles of 16 MT rows.
template <int MT, bool PAIR> struct Form {
    static constexpr int RT = PAIR ? 8 : 16 * MT;
};
// Waves of a workgroup.
constexpr int waves(int D, int rt) { return D == 256 && rt == 8 ? 8 : 4; }

// One workgroup: a tile of query rows, one KV head, one split of the
// positions; its waves take tiles of 32 positions in turn and join at the end.
template <int D, int MT, bool PAIR, bool SHARE>
__global__ void __launch_bounds__(64 * waves(D, Form<MT, PAIR>::RT), 2)
kv_attn_kernel(AttnArgs a) {
    using L = KvLayout<D>;
    constexpr int G = L::G, RT = Form<MT, PAIR>::RT, AW = waves(D, RT), NT = D / 16, OP = D + 4;
    constexpr int RC = PAIR ? 8 : 16;     // rows side by side in a wave's columns
    constexpr int GL = PAIR ? G / 2 : G;  // groups whose steps a lane keeps
    constexpr int VD = D >= 128 ? 4 : 2;  // dwords of a lane's four value pieces
    __shared__ float4 red4[AW * RC * OP / 4];
    __shared__ float2 st[AW][RT];
    float *red = reinterpret_cast<float *>(red4);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int hc = PAIR ? col >> 3 : 0;   // half of the groups, by column
    const int hk = blockIdx.x % a.c.hkv, bs = blockIdx.x / a.c.hkv;
    Item t;
    if (!find_item<RT, SHARE>(a, bs, false, 0, lane, t)) return;
    const int R = t.n * a.grp;
    const int64_t cap = (int64_t)a.sq.max_pages << a.c.ps_log2;
    // positions of the tile's first and last row, and the split's tiles of 32
    const int64_t p0 = (int64_t)t.len - t.n, pmin = p0 + t.j * RT / a.grp, pmax = p0 + (min(t.j * RT + RT, R) - 1) / a.grp;
    const int64_t end = min(pmax + 1, cap), begin = a.window ? max((int64_t)0, pmin - a.window + 1) : 0;
    const int64_t tb = begin >> 5, nt = end > begin ? ((end + 31) >> 5) - tb : 0;
    const int x0 = (int)(tb + nt * t.split / t.ns), x1 = (int)(tb + nt * (t.split + 1) / t.ns);
    const int32_t *table = a.sq.pages + (int64_t)t.s * a.sq.max_pages;
    const int tsh = a.c.ps_log2 - 5;
    const int64_t pstride = 2 * a.c.hkv * L::block(a.c.ps_log2);
    const uint8_t *pool = a.c.pool + (int64_t)hk * 2 * L::block(a.c.ps_log2);
    // Pages of the wave's next 64 tiles, one a lane: a page number is then a
    // register, not a load that the tile's loads would wait behind.  A page
    // that is not held is -1.
    int ahead = 0;
    auto look_ahead = [&](int x) {
        const int64_t at = min((int64_t)x + AW * lane, (int64_t)x1 - 1);
        const int page = table[at >> tsh];
        ahead = page >= 0 && page < a.c.num_pages ? page : -1;
    };

    uint32_t kc[2][G], kd[2][2 * GL], km[2][G / 2], vc[2][L::VW][VD], vd[2][2 * GL], vm[2][2];
    // a lane's offsets inside a tile; the tile's own place is uniform
    const uint32_t at_kc = col * L::ROW + (PAIR ? (quad & 1) * 4 * G + (quad >> 1) * 2 * G : quad * 4 * G);
    const uint32_t at_d = quad * 8 * G + hc * 4 * G, at_km = col * 2 * G;
    const uint32_t at_vc = (quad * L::VW * 16 + col) * 4 * VD, at_vm = (quad * G + min(col, G - 1)) * 8;
    const int d_off = L::d_off(a.c.ps_log2), m_off = L::m_off(a.c.ps_log2);
    auto load_k = [&](int page, int x) {
        const int p0 = (x & ((1 << tsh) - 1)) << 5;  // of the page
        const uint8_t *kb = pool + page * pstride, *c = kb + p0 * L::ROW, *d = kb + d_off + p0 * 2 * G,
                      *m = kb + m_off + p0 * 2 * G;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (PAIR) {
                load<G / 2>(kc[u], c + at_kc + u * 16 * L::ROW);
                load<G / 2>(kc[u] + G / 2, c + at_kc + u * 16 * L::ROW + 8 * G);
            } else {
                load<G>(kc[u], c + at_kc + u * 16 * L::ROW);
            }
            load<2 * GL>(kd[u], d + at_d + u * 32 * G);
            load<G / 2>(km[u], m + at_km + u * 32 * G);
        }
    };
    auto load_v = [&](int page, int x) {
        const int p0 = (x & ((1 << tsh) - 1)) << 5;
        const uint8_t *vb = pool + page * pstride + L::block(a.c.ps_log2);
        const uint8_t *c = vb + p0 * L::ROW, *d = vb + d_off + p0 * 2 * G, *m = vb + m_off + p0 * 2 * G;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int w = 0; w < L::VW; ++w) load<VD>(vc[u][w], c + at_vc + (u * 4 * L::VW + w) * 64 * VD);
            load<2 * GL>(vd[u], d + at_d + u * 32 * G);
            load<2>(vm[u], m + at_vm + u * 32 * G);
        }
    };
    int x = x0 + wave, page = -1;
    if (x < x1) look_ahead(x);

    // query rows as the second operand, scaled by a power of two per row so
    // that neither they nor their sixteenths are subnormal
    // D = 256 in tiles of 16 rows: 32 registers too many, so from LDS
    constexpr bool QLDS = D == 256 && !PAIR;
    u4 *const ql = reinterpret_cast<u4 *>(red4);  // [G][64], the same for every wave
    u4 qf[QLDS ? 1 : MT][QLDS ? 1 : G], qs[MT];
    int qat = lane;
    float sc1[MT], sc2[MT];
    int lim[MT], low[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = t.j * RT + mt * 16 + (col & (RC - 1)), rr = min(r, R - 1), tok = rr / a.grp;
        const int64_t pos = p0 + tok;
        lim[mt] = (int)max((int64_t)-1, min(pos, cap - 1));
        low[mt] = a.window ? (int)min(max((int64_t)0, pos - a.window + 1), (int64_t)INT32_MAX) : 0;
        const _Float16 *src = reinterpret_cast<const _Float16 *>(a.q.p) + (int64_t)(t.first + tok) * a.q.row +
                              (int64_t)(hk * a.grp + rr % a.grp) * a.q.head;
        // operand i of a lane: 8 dimensions from `dim(i)` on, or zeros
        const bool mine = !PAIR || (quad >> 1) == hc;
        auto dim = [&](int i) {
            return PAIR ? 32 * ((i >> 1) + hc * (G / 2)) + 16 * (i & 1) + 8 * (quad & 1) : 32 * i + 8 * quad;
        };
        u4 raw[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            raw[i] = u4{0, 0, 0, 0};
            if (mine) {
                if (a.qvec) {
                    raw[i] = *reinterpret_cast<const u4 *>(src + dim(i));
                } else {
                    h8 w;
#pragma unroll
                    for (int n = 0; n < 8; ++n) w[n] = src[(int64_t)(dim(i) + n) * a.q.elem];
                    raw[i] = __builtin_bit_cast(u4, w);
                }
            }
        }
        if (mt == 0 && x < x1) {  // the first tile's loads, before the queries are waited for
            page = __builtin_amdgcn_readlane(ahead, 0);
            if (!QLDS) {
                load_k(max(page, 0), x);
                load_v(max(page, 0), x);
            }
        }
        // row norm N: scaled by 2^e to N in [2^12, 2^13), as high as a group's
        // sum (at most sqrt(32) N) stays in fp16; the smallest elements'
        // sixteenths are then held to 2^-33 N.  Rows below 2^-18 by 2^30, which is exact;
        // infinite, NaN or zero rows as they are.
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) ss = dot2(raw[i][k], raw[i][k], ss);
        if (PAIR) ss += __shfl_xor(ss, 8);
        ss += __shfl_xor(ss, 16);
        ss += __shfl_xor(ss, 32);
        const int e = ss > 0.f && ss < 1e30f ? min(12 - (((int)(__float_as_uint(ss) >> 23) - 127) >> 1), 30) : 0;
        const float f = pow2(e);
        sc2[mt] = a.scale * 1.44269504088896340736f * pow2(-e);
        sc1[mt] = sc2[mt] * 2097152.f;  // 2^21, the codes' unit
        const h2 f1 = half_pair(pow2(min(e, 15))), f2 = half_pair(pow2(e - min(e, 15))), f16th = half_pair(0.0625f);
        const bool twice = __any(e > 15);  // (fp16 ends at 2^15)
        uint32_t sums[4] = {0, 0, 0, 0};
        float half = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            float s = 0.f;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t two = raw[i][k];
                s = dot2(two, 0x3c003c00u, s);
                h2 y = __builtin_bit_cast(h2, two) * f1;
                if (twice) y *= f2;
                w[k] = __builtin_bit_cast(uint32_t, y);
            }
            s *= f;
            // nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7: the odd ones' codes come 16 times too large
            auto pair = [&](uint32_t x, uint32_t y, uint32_t sel) { return __builtin_amdgcn_perm(y, x, sel); };
            auto sixteenth = [&](uint32_t x) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, x) * f16th); };
            const u4 op = u4{pair(w[0], w[2], 0x05040100u), sixteenth(pair(w[0], w[2], 0x07060302u)),
                             pair(w[1], w[3], 0x05040100u), sixteenth(pair(w[1], w[3], 0x07060302u))};
            if constexpr (QLDS) {
                if (wave == 0) ql[i * 64 + lane] = op;
            } else {
                qf[mt][i] = op;
            }
            // the group's sum as two fp16 terms, in two quads
            if (PAIR && (i & 1) == 0) {
                half = s;
                continue;
            }
            if (PAIR) s += half;
            s += __shfl_xor(s, 16);
            if (!PAIR) s += __shfl_xor(s, 32);
            const _Float16 hi = (_Float16)s, lo = (_Float16)(s - (float)hi);
            const int term = PAIR ? quad & 1 : quad;
            const _Float16 v = mine && term == 0 ? hi : mine && term == 1 ? lo : (_Float16)0.f;
            const uint32_t bits = __builtin_bit_cast(uint16_t, v);
            if constexpr (PAIR) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int g = (i >> 1) + h * (G / 2);
                    sums[g >> 1] |= (hc == h ? bits : 0u) << (16 * (g & 1));
                }
            } else {
                sums[i >> 1] |= bits << (16 * (i & 1));
            }
        }
        qs[mt] = u4{sums[0], sums[1], sums[2], sums[3]};
    }
    // (wave-uniform) tiles that every row sees whole, and positions that hold something
    const int64_t all_lo = a.window ? max((int64_t)0, pmax - a.window + 1) : 0, all_hi = min(pmin, cap - 1);
    const int held = (int)min((int64_t)t.len, cap), past = (int)min(begin, cap);  // (cap is at most 2^30)

    f4 o[MT][NT], om[MT];
    float m[MT], grow[MT];  // the maximum so far less TOP; how far a score may pass it before it moves (M_NONE: no score yet)
    int ve = 0;             // steps are taken times 2^ve, below 1 in every tile so far; wave-uniform
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < NT; ++i) o[mt][i] = f4{0.f, 0.f, 0.f, 0.f};
        om[mt] = f4{0.f, 0.f, 0.f, 0.f};
        m[mt] = 0.f;
        grow[mt] = M_NONE;
    }

    if (QLDS) __syncthreads();
    auto query = [&](int mt, int i) {
        if constexpr (QLDS) return ql[i * 64 + qat];
        else return qf[mt][i];
    };
    float minus1 = -1.f;
    asm("" : "+s"(minus1));

    // Keys of the next tile are asked for when this tile's are used up, and
    // values when this tile's are: each comes in under the other half's work.
    // A page that is not held is read as page 0 and counts for nothing; behind
    // the last tile the same tile is asked for again.
    for (int k = 1; x < x1; ++k, x += AW) {
        const bool live = page >= 0;
        int nx = x, np = page;
        if (x + AW < x1) {
            nx = x + AW;
            if ((k & 63) == 0) look_ahead(nx);
            np = __builtin_amdgcn_readlane(ahead, k & 63);
        }

        if constexpr (QLDS) {
            load_k(max(page, 0), x);
            load_v(max(page, 0), x);
            asm("" : "+v"(qat));  // read where they are used, not kept in registers
        }

        // scores
        float z[MT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f4 s[MT], acc[MT];
            u4 mo = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < G / 2; ++i) mo[i] = km[u][i];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[mt] = mfma(mo, qs[mt], f4{0.f, 0.f, 0.f, 0.f});
                acc[mt] = f4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int g = 0; g < GL; ++g) {
                u4 ko[2];
#pragma unroll
                for (int i = 0; i < (PAIR ? 2 : 1); ++i) {
                    const uint32_t w = kc[u][g + i * (G / 2)], a0 = w << 3, a1 = w >> 5;
                    ko[i] = u4{a0 & EVEN, a0 & ODD, a1 & EVEN, a1 & ODD};
                }
                const float d0 = lo_f(kd[u][2 * g]), d1 = hi_f(kd[u][2 * g]), d2 = lo_f(kd[u][2 * g + 1]),
                            d3 = hi_f(kd[u][2 * g + 1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    f4 r = mfma(ko[0], query(mt, PAIR ? 2 * g : g), f4{0.f, 0.f, 0.f, 0.f});
                    if constexpr (PAIR) r = mfma(ko[1], query(mt, 2 * g + 1), r);
                    acc[mt] = f4{fmaf(d0, r.x, acc[mt].x), fmaf(d1, r.y, acc[mt].y), fmaf(d2, r.z, acc[mt].z),
                                 fmaf(d3, r.w, acc[mt].w)};
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // less the maximum so far (each half of the columns takes half of it)
                    float y = fmaf(acc[mt][i], sc1[mt], fmaf(s[mt][i], sc2[mt], PAIR ? -0.5f * m[mt] : -m[mt]));
                    if constexpr (PAIR) y += row_half_swap(y);
                    z[mt][u][i] = y;
                }
        }
        if constexpr (!QLDS) {
            __builtin_amdgcn_sched_barrier(0);
            load_k(max(np, 0), nx);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!live || x * 32 < all_lo || x * 32 + 31 > all_hi) {
            const int base = x * 32 + 4 * quad;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = base + 16 * u + i;
                        z[mt][u][i] = live && p <= lim[mt] && p >= low[mt] ? z[mt][u][i] : -INFINITY;
                    }
        }

        // probabilities relative to the running maximum, as two fp16 terms
        uint32_t ph[MT][2][2], pl[MT][2][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float mx = z[mt][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) mx = fmaxf(mx, z[mt][i >> 2][i & 3]);
            if (__any(mx > grow[mt])) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const bool fresh = grow[mt] == M_NONE, some = mx > M_NONE;
                const float up = fresh ? (some ? mx - TOP : 0.f) : fmaxf(mx - TOP, 0.f);
                const float al = fresh ? 0.f : __builtin_amdgcn_exp2f(-up);
                m[mt] += up;
                if (some) grow[mt] = GROW;
                om[mt] *= al;
#pragma unroll
                for (int i = 0; i < NT; ++i) o[mt][i] *= al;
#pragma unroll
                for (int i = 0; i < 8; ++i) z[mt][i >> 2][i & 3] -= up;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    const float p0 = __builtin_amdgcn_exp2f(z[mt][u][2 * k2]);
                    const float p1 = __builtin_amdgcn_exp2f(z[mt][u][2 * k2 + 1]);
                    ph[mt][u][k2] = pack(p0, p1);
                    // (opaque, so that the residual is one mixed fma on the packed pair and not three conversions)
                    asm("" : "+v"(ph[mt][u][k2]));
                    pl[mt][u][k2] = pack(fmaf(lo_f(ph[mt][u][k2]), minus1, p0), fmaf(hi_f(ph[mt][u][k2]), minus1, p1));
                }
        }

        // values; of places that hold nothing yet or that no row's window
        // reaches, whatever their bytes say, the step and the minimum are 0
        // (a probability of 0 does not hide NaN).  Steps are to be below 1, and
        // not far below: those of a tile that holds a larger one are scaled,
        // and the sums so far with them.
        const bool edge = !live || x * 32 + 32 > held || x * 32 < past;
        auto largest = [&] {  // step in either half of a lane's
            uint32_t v = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 2 * GL; ++i) v = max2(v, vd[u][i]);
            return max(v & 0xffffu, v >> 16);
        };
        uint32_t top = largest();
        if (edge || ve != 0 || __any(top >= 0x3c00u) || (k == 1 && !__any(top >= (uint32_t)(14 - NEAR) << 10))) {
            if (edge) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const int p = x * 32 + 16 * u + 4 * quad + 2 * k2;
                        const uint32_t mask = (live && p >= past && p < held ? 0xffffu : 0u) |
                                              (live && p + 1 >= past && p + 1 < held ? 0xffff0000u : 0u);
#pragma unroll
                        for (int g = 0; g < GL; ++g) vd[u][2 * g + k2] &= mask;
                        vm[u][k2] &= mask;
                    }
                top = largest();
            }
            if (k == 1 || __any(top >= (uint32_t)(15 - ve) << 10)) {
                int field = 0;  // exponent of the wave's largest step (30 for what is not finite, as others may write)
#pragma unroll
                for (int bit = 16; bit; bit >>= 1)
                    if (__any(top >= (uint32_t)(field | bit) << 10)) field |= bit;
                int to = 14 - min(field, 30);
                if (to >= 0 && to <= NEAR) to = 0;
                if (k > 1) to = min(to, ve);
                const float down = pow2(to - ve);
                ve = to;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < NT; ++i) o[mt][i] *= down;
            }
            if (ve != 0) {
                const h2 vs = half_pair(pow2(ve));
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 2 * GL; ++i)
                        vd[u][i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, vd[u][i]) * vs);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            // row G of the minima is ones: its sum is the softmax's
            u4 mo = {vm[0][0], vm[0][1], vm[1][0], vm[1][1]};
            if (col == G) mo = u4{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
            om[mt] = mfma(mo, u4{ph[mt][0][0], ph[mt][0][1], ph[mt][1][0], ph[mt][1][1]}, om[mt]);
            om[mt] = mfma(mo, u4{pl[mt][0][0], pl[mt][0][1], pl[mt][1][0], pl[mt][1][1]}, om[mt]);
        }
#pragma unroll
        for (int gl = 0; gl < GL; ++gl) {
            u4 hi[MT], lo[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const h2 d = __builtin_bit_cast(h2, vd[u][2 * gl + k2]);
                        const h2 p = __builtin_bit_cast(h2, ph[mt][u][k2]), q = __builtin_bit_cast(h2, pl[mt][u][k2]);
                        const h2 y = p * d;
                        const h2 r = __builtin_elementwise_fma(p, d, -y);
                        hi[mt][2 * u + k2] = __builtin_bit_cast(uint32_t, y);
                        lo[mt][2 * u + k2] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(q, d, r));
                    }
#pragma unroll
            for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
                const int g = gl + h * (G / 2);
                u4 v0, v1;  // dimensions 32g .. 32g+15 and 32g+16 .. 32g+31 (those 16 times too large)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        uint32_t w;
                        if constexpr (D == 64) {
                            w = g ? vc[u][0][k2] >> 5 : vc[u][0][k2] << 3;
                        } else {
                            const uint32_t sel = 0x0c040c00u + 0x00010001u * (uint32_t)(g & 3);
                            w = __builtin_amdgcn_perm(vc[u][g >> 2][2 * k2 + 1], vc[u][g >> 2][2 * k2], sel) << 3;
                        }
                        v0[2 * u + k2] = w & EVEN;
                        v1[2 * u + k2] = w & ODD;
                    }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[mt][2 * g] = mfma(v0, hi[mt], o[mt][2 * g]);
                    o[mt][2 * g + 1] = mfma(v1, hi[mt], o[mt][2 * g + 1]);
                    o[mt][2 * g] = mfma(v0, lo[mt], o[mt][2 * g]);
                    o[mt][2 * g + 1] = mfma(v1, lo[mt], o[mt][2 * g + 1]);
                }
            }
        }
        if constexpr (!QLDS) {
            __builtin_amdgcn_sched_barrier(0);
            load_v(max(np, 0), nx);
            __builtin_amdgcn_sched_barrier(0);
        }
        page = np;
    }

    // join the waves: common maximum, then sums through LDS, RC rows at a time
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const float sum = om[mt][G & 3];  // row G, in quad G / 4
        if (grow[mt] == M_NONE) m[mt] = M_NONE;
        if (quad == G / 4 && hc == 0) st[wave][mt * 16 + col] = make_float2(m[mt], sum);
    }
    __syncthreads();
    const int64_t unit = ((int64_t)bs) * a.c.hkv + hk;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int row0 = col & (RC - 1);
        float mx = st[0][mt * 16 + row0].x;
#pragma unroll
        for (int w = 1; w < AW; ++w) mx = fmaxf(mx, st[w][mt * 16 + row0].x);
        const float f = __builtin_amdgcn_exp2f(m[mt] - mx);
        float *mine = red + (wave * RC + row0) * OP;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // the group's minima term: row g of om, held by quad g / 4
            const float mg = __shfl(om[mt][g & 3], (g >> 2) * 16 + col) * f;
            if (PAIR && hc != g / (G / 2)) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f4 v = o[mt][2 * g + k];
                const float s = (k ? 131072.f : 2097152.f) * f * pow2(-ve);  // 2^17, 2^21: the codes' units
                *reinterpret_cast<float4 *>(mine + 32 * g + 16 * k + 4 * quad) =
                    make_float4(fmaf(v.x, s, mg), fmaf(v.y, s, mg), fmaf(v.z, s, mg), fmaf(v.w, s, mg));
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < RC * D / 4; i += 64 * AW) {
            const int row = i / (D / 4), c4 = i % (D / 4), r = t.j * RT + mt * 16 + row;
            if (r >= R) continue;
            float4 s = *reinterpret_cast<const float4 *>(red + row * OP + 4 * c4);
#pragma unroll
            for (int w = 1; w < AW; ++w) {
                const float4 v = *reinterpret_cast<const float4 *>(red + (w * RC + row) * OP + 4 * c4);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
            float mm = st[0][mt * 16 + row].x, ll = 0.f;
#pragma unroll
            for (int w = 1; w < AW; ++w) mm = fmaxf(mm, st[w][mt * 16 + row].x);
#pragma unroll
            for (int w = 0; w < AW; ++w) ll = fmaf(__builtin_amdgcn_exp2f(st[w][mt * 16 + row].x - mm), st[w][mt * 16 + row].y, ll);
            if (t.ns == 1) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int64_t at = (int64_t)(t.first + r / a.grp) * a.out.row +
                                   (int64_t)(hk * a.grp + r % a.grp) * a.out.head + (int64_t)(4 * c4) * a.out.elem;
                store_out(a.out, at, s.x * inv);
                store_out(a.out, at + a.out.elem, s.y * inv);
                store_out(a.out, at + 2 * a.out.elem, s.z * inv);
                store_out(a.out, at + 3 * a.out.elem, s.w * inv);
            } else {
                reinterpret_cast<float4 *>(a.o + (unit * RT + mt * 16 + row) * D)[c4] = s;
                if (c4 == 0) a.ml[unit * RT + mt * 16 + row] = make_float2(mm, ll);
            }
        }
        __syncthreads();
    }
}

// Joins the splits of a row: one workgroup per row and query head.
template <int D, int RT>
__global__ void __launch_bounds__(256) kv_attn_join_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    __shared__ float wt[MAX_SPLIT], part[4][D], mx_s[4], sum_s[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = blockIdx.x / a.hq, h = blockIdx.x % a.hq;
    const RowSeq rs = row_seq(a.sq, row, lane);
    if (rs.s >= a.sq.nseq) return;
    const int hk = h / a.grp, r = (row - rs.first) * a.grp + h % a.grp;
    Item t;
    if (!find_item<RT, true>(a, rs.s, true, r / RT, lane, t) || t.ns == 1) return;  // (one split: written already)
    const int ns = t.ns;
    auto unit = [&](int s) { return ((int64_t)(t.id0 + s) * a.c.hkv + hk) * RT + r % RT; };
    const float2 v = tid < ns ? a.ml[unit(tid)] : make_float2(M_NONE, 0.f);
    // the first splits' outputs are asked for before their weights are known
    constexpr int FIRST = 16;
    float first[FIRST][E];
#pragma unroll
    for (int i = 0; i < FIRST; ++i) {
        const float *p = a.o + unit(min(wave + 4 * i, ns - 1)) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) first[i][e] = p[e];
    }
    float mx = v.x;
    for (int i = 1; i < 64; i <<= 1) mx = fmaxf(mx, __shfl_xor(mx, i));
    if (lane == 0) mx_s[wave] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(mx_s[0], mx_s[1]), fmaxf(mx_s[2], mx_s[3]));
    const float w = __builtin_amdgcn_exp2f(v.x - mx);
    float sum = tid < ns ? w * v.y : 0.f;
    wt[tid] = tid < ns ? w : 0.f;
    for (int i = 1; i < 64; i <<= 1) sum += __shfl_xor(sum, i);
    if (lane == 0) sum_s[wave] = sum;
    __syncthreads();
    sum = (sum_s[0] + sum_s[1]) + (sum_s[2] + sum_s[3]);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int i = 0; i < FIRST; ++i) {
        if (wave + 4 * i >= ns) break;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wt[wave + 4 * i], first[i][e], acc[e]);
    }
#pragma unroll 8
    for (int s = wave + 4 * FIRST; s < ns; s += 4) {
        const float *p = a.o + unit(s) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wt[s], p[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[wave][lane * E + e] = acc[e];
    __syncthreads();
    if (tid < D) {
        const float y = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        store_out(a.out, row * a.out.row + h * a.out.head + tid * a.out.elem, sum == 0.f ? 0.f : y / sum);
    }
}

// Launch shape: from sizes alone (the lengths are on the device).  Rows of a
// sequence by its heads of a KV head decide the tile: up to 8 the pair form;
// beyond, 16 (a form of 32 shares the unpacking of more rows but leaves one
// wave a SIMD at D = 128: 235 us against 195 at 509 rows x 4 heads, 8200
// positions), and 32 only for D = 64 and many rows (108 us against 129 at
// 2036, 56 against 52 at 512).  Workgroups of 8 waves where two waves fill a
// SIMD's registers (D = 256, pairs), else 4: fewer splits to join, against
// more of them to hide each other's start (48 sequences of 1..16384 positions,
// D = 128: 50 us with 4, 93 with 8; 1 token over 32773, D = 256: 24 and 21).
// A split has two tiles of 32 positions a wave or more (1 token over 32773:
// 21.7 us with one or two, 24.3 with four).  One sequence is cut into as many
// splits as fit at once, several into twice that, which evens out their unlike
// lengths (48 sequences: 49 us against 126; one sequence of 262139 and 32773
// positions: 81 and 33 us with twice, 74 and 22 with once).  (Both sides of
// each comparison are of one build; its split kernels were 2..7% slower than
// these.)
struct Shape {
    int rt, target, min_chunk, nitems;
};
Shape attn_shape(const KvCache &c, const KvSeqs &sq, int hq) {
    const int grp = hq / c.hkv;
    Shape s;
    const int64_t n = sq.rows / sq.nseq, per_seq = ((int64_t)sq.rows * grp + sq.nseq - 1) / sq.nseq;
    s.rt = per_seq <= 8 ? 8 : per_seq < 1024 || c.D > 64 ? 16 : 32;
    const int64_t tiles = sq.q_start ? (int64_t)sq.rows * grp / s.rt + std::min(sq.nseq, sq.rows)
                                     : sq.nseq * ((n * grp + s.rt - 1) / s.rt);
    const int aw = waves(c.D, s.rt);
    s.min_chunk = 2 * aw;
    const int64_t most = ((int64_t)sq.max_pages << c.ps_log2) / 32;  // tiles of 32 positions
    const int64_t slots = (int64_t)device_cus() * (c.D == 256 ? 8 : 12) / aw;  // workgroups that fit at once
    const int64_t share = slots * (sq.nseq > 1 ? 2 : 1) / c.hkv - tiles;
    // Every workgroup sums over all sequences, 0.03..0.045 us each; a context
    // in one piece takes 0.25 us a tile of 32 (D = 128, 8 KV heads; 1024
    // sequences, most of them without rows, tables of 8192 positions: 38 us
    // shared against 63 with one live sequence, 75 against 65 with 16; 8192
    // sequences: 236 against 64; tables of 131072: 63 against 895).
    // Nor are contexts shared where tiles alone are half of the workgroups that
    // fit: right for lengths alike (8000 positions, one of 16384: 209 us at 95
    // sequences, shared, 220 at 96), wrong for one of 131072 among others of
    // 300 (51 us at 95, 992 at 96), which the lengths alone would tell.
    s.target = most > s.min_chunk && share > tiles && sq.nseq <= 4 * most ? (int)share : 0;
    s.nitems = (int)(tiles + s.target);
    return s;
}

}  // namespace attn

using namespace attn;

int64_t kv_attn_workspace(const KvCache &c, const KvSeqs &sq, int hq) {
    const Shape s = attn_shape(c, sq, hq);
    return s.target ? (int64_t)s.nitems * c.hkv * s.rt * (4 * c.D + 8) : 0;
}

hipError_t launch_kv_attn(const KvCache &c, const KvSeqs &seqs, int hq, const Heads &q, const Heads &out, float scale,
                          int window, void *workspace, hipStream_t st) {
    const Shape s = attn_shape(c, seqs, hq);
    AttnArgs a{c, seqs, q, out, hq, hq / c.hkv, window, s.target, s.min_chunk,
               s.target ? 1.0001f / s.target : 0.f, s.nitems, scale, 0, nullptr, nullptr};
    a.qvec = q.elem == 1 && q.row % 8 == 0 && q.head % 8 == 0 && ((uintptr_t)q.p & 15) == 0;
    if (s.target) {
        a.o = (float *)workspace;
        a.ml = (float2 *)(a.o + (int64_t)s.nitems * c.hkv * s.rt * c.D);
    }
    auto go = [&](auto kern, auto join) -> hipError_t {
        hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)s.nitems * c.hkv)), dim3(64 * waves(c.D, s.rt)), 0, st, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !s.target) return e;
        hipLaunchKernelGGL(join, dim3((unsigned)(seqs.rows * hq)), dim3(256), 0, st, a);
        return hipGetLastError();
    };
    auto form = [&](auto share) {
        constexpr bool SHARE = decltype(share)::value;
        if (c.D == 256)
            return s.rt == 8 ? go(kv_attn_kernel<256, 1, true, SHARE>, kv_attn_join_kernel<256, 8>)
                             : go(kv_attn_kernel<256, 1, false, SHARE>, kv_attn_join_kernel<256, 16>);
        if (c.D == 128)
            return s.rt == 8 ? go(kv_attn_kernel<128, 1, true, SHARE>, kv_attn_join_kernel<128, 8>)
                             : go(kv_attn_kernel<128, 1, false, SHARE>, kv_attn_join_kernel<128, 16>);
        return s.rt == 8    ? go(kv_attn_kernel<64, 1, true, SHARE>, kv_attn_join_kernel<64, 8>)
               : s.rt == 16 ? go(kv_attn_kernel<64, 1, false, SHARE>, kv_attn_join_kernel<64, 16>)
                            : go(kv_attn_kernel<64, 2, false, SHARE>, kv_attn_join_kernel<64, 32>);
    };
    return s.target ? form(std::true_type{}) : form(std::false_type{});
}

}  // namespace qk
