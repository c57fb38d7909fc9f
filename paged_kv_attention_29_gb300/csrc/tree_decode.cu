// Attention of a tree of drafted tokens over the paged KV cache, on tcgen05
// tensor cores: the verification step of tree-structured speculative decoding,
// on the bf16 cache and on the 8-bit one.
//
// Sequence b has n_b nodes; their K/V rows are its last n_b positions, behind the
// P_b = L_b - n_b positions every node sees.  Node i also sees node j iff bit j of its
// mask is set:
//
//   out[i] = softmax_j(scale q_i . k_j) v_j   over j < P_b and the nodes of i's mask
//
// Unit: one sequence, one KV head and one tile of 128 / G nodes x the G query heads
// that share it (row r of the tile: node r / G, head G g + r % G).  Its keys go by in
// tiles of 64:
//
//   S = Q K^T   tcgen05.mma M=128 N=64, fp32 in TMEM, two buffers
//   P           masked online softmax by the warpgroup, bf16 over S
//   O += P V    tcgen05.mma with P from TMEM
//
// The tiles of all sequences, in order, are cut into runs of equal cost, and each run is
// taken by a CTA per KV head (two CTAs per SM, so that one's loads and products fill the
// other's waits; a run's CTAs are neighbours, so that the heads' rows of a token, which
// lie side by side in memory, are read at about the same time): a unit that a run does
// not hold whole leaves fp32 averages with their references and sums in the workspace, and
// a second kernel joins them in the order of the runs.  Results are deterministic.
//
// A node's row is as if masked keys were not there, whatever they hold: scores are
// selected, not added to, and infinities and NaN among the nodes' V rows, which a
// product with a weight of 0 would spread, are taken out of the tile and given back
// to the rows that see them.
//
// Trees of 16 rows or fewer on the 8-bit cache are another kernel's (tree_decode_rows.cu).
//
// Measured (calls in a graph, 8 KV heads): batch 64 with 512 to 4096 keys and 12 to 16
// nodes, G = 2, 575 MB: 98 us, 5.9 TB/s; 8 sequences of 16k to 40k keys, 60 nodes, 964 MB:
// 156 us, 6.2 TB/s: HBM.  32 sequences of 80 to 2999 keys, 33 to 64 nodes, G = 4, 46 GFLOP: 73
// us, bound by the steps of a tile (S, softmax, P, O), which wait on one another.  8-bit cache: the
// first case 99 us, 7 sequences of 16k to 40k keys, 13 to 29 nodes, G = 8: 128, bound by the same steps,
// whose waits and loads shared memory answers late (some 180 cycles beside the products' reads).  So
// each step of its softmax takes one pass over the scores, 32 at a time with their scales loaded a
// step ahead (two passes of 16: 110 and 156 us; one of 16: 107 and 142).  Its loops are kept rolled and
// rare paths out of line, since the roles share the schedulers' instruction caches.
//
// Warps 0-3: softmax and epilogue (TMEM lanes 0-127).  bf16 cache: warp 4 TMA producer,
// warp 5 TMEM allocation and MMA issue.  8-bit cache: warps 4-7 turn the codes that TMA
// has put into a slot of the ring into the bf16 values they stand for, in place; warp 8
// issues, warp 9 is the producer.
#include <algorithm>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int D = kHeadDim;
constexpr int ROWS = 128;                    // MMA M
constexpr int KT = 64;                       // keys per tile
constexpr int Q_HALF = ROWS * 64 * 2;        // 128B-swizzled box of 64 dims: 16 KiB of Q
constexpr int KV_HALF = KT * 64 * 2;         // 8 KiB of K or V
constexpr int KV_TILE = 2 * KV_HALF;
constexpr int TMEM_COLS = 256;
constexpr int O_COL = 128;                   // S / P buffers at columns 0 and 64
// A row's reference is put 2^16 above its largest score and moved again once the weights' sum has passed 1/4 (bf16: or one
// of the tile's weights 2^-8, and 64 of those make another 1/4).  So the sum stays below 1/2 and |O| below 2^127 for any
// finite V.  2^16, so that long contexts seldom move it (16384 equal keys); a lower one would leave O more of fp32's range at
// the lower end, where V of 2^-118 keeps 14 bits.  The sum is 2^-18 at least, and weights end at 2^-126: at 2^-108 of it.
constexpr float kLift = 16.0f;
constexpr float kMostWeightLog2 = -8.0f;
constexpr float kMostSum = 0.25f;
// 8 bits: the factor of a row whose query holds an infinity or a NaN.  Any number would do that is positive, finite and no
// other row's: a score that is not seen is -inf times the factor, and so that this is -inf no factor may be 0 or NaN.
constexpr float kBadRow = 0x1.000002p-126f;
constexpr int UNIT_COST = 2;                 // what starting and ending a unit costs, in tiles
constexpr int MIN_RUN = 4;                   // cost a CTA takes at least; above UNIT_COST, so that every run has a tile
static_assert(MIN_RUN > UNIT_COST, "a run has a tile");
constexpr int CTAS_PER_SM = 2;
constexpr int THREADS_BF16 = 192, THREADS_FP8 = 320;

// Shared memory.  bf16: rings of 3 K and 2 V tiles (a K tile is asked for two steps before its product, a V tile's
// product comes a step later).  8 bits: 3 tiles of K codes and 3 V tiles; the row scales of K as bytes and as floats, in
// rings so long that those of a tile are read before K's copies come round again (K of tile t + 5 is asked for when
// tile t is through); each query row's factor, of two segments.
template <bool FP8>
struct Layout {
    static constexpr int K_SLOTS = 3, V_SLOTS = FP8 ? 3 : 2, K_TILE = FP8 ? KT * D : KV_TILE, KS_SLOTS = 6;
    static constexpr int Q = 0, K = 2 * Q_HALF, V = K + K_SLOTS * K_TILE, VS = V + V_SLOTS * KV_TILE, KS = VS + (FP8 ? V_SLOTS * KT : 0);
    static constexpr int KSF = KS + (FP8 ? KS_SLOTS * KT : 0), QS = KSF + (FP8 ? KS_SLOTS * KT * 4 : 0);
    static constexpr int BAR = QS + (FP8 ? 2 * ROWS * 4 : 0);
    static constexpr int KF = 0, KE = KF + K_SLOTS, VF = KE + K_SLOTS, VE = VF + V_SLOTS, QF = VE + V_SLOTS, QE = QF + 1, SF = QE + 1, PF = SF + 2,
                         PV = PF + 2, OF = PV + 2, OE = OF + 1, WG = OE + 1, DRAIN = WG + 1, BF16_BARS = DRAIN + 1;
    static constexpr int VRAW = BF16_BARS, KSB = VRAW + V_SLOTS, KSR = KSB + KS_SLOTS, QR = KSR + KS_SLOTS, QG = QR + 1, FP8_BARS = QG + 1;
    static constexpr int NUM_BARS = FP8 ? FP8_BARS : BF16_BARS;
    static constexpr int MISC = (BAR + NUM_BARS * 8 + 15) & ~15;  // [0] TMEM base, [1] abort
    static constexpr int WILD = MISC + 16;                        // [2][4 warps][8]: nodes with infinities or NaN in V
    static constexpr int SCAN = WILD + 2 * 4 * 8 * 4;             // 16 x int64: set-up sums; what the run is; its start
    static constexpr int BYTES = SCAN + 16 * 8;
    static_assert(K % 1024 == 0 && V % 1024 == 0 && KSF % 16 == 0 && BAR % 8 == 0, "operand tiles and vectors need their alignment");
    static_assert(CTAS_PER_SM * (BYTES + 1024) <= 228 * 1024, "two CTAs share an SM's shared memory");
};

struct Params {
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_nodes;
    const unsigned long long* mask;
    uint16_t* out;
    float4* part_o;           // [CTA][2][32][128]: four columns of each row, over the sum
    float2* part_ml;          // [CTA][2][128]: reference (log2) and sum
    int4* meta;               // [CTA]: {last run of the unit that continues behind this one's or -1, first row's node, nodes, CTAs of a run}
    const uint8_t* v_codes;   // 8-bit cache, for the values taken out of a tile
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const uint16_t* v_cache;  // bf16 cache, for the values taken out of a tile
    int batch, max_blocks, num_heads, num_kv_heads, lg, block_size, num_blocks;
    int max_nodes, max_context, mask_words, total_nodes;
    int qtok;                 // nodes of a tile: 128 / G
    float scale_log2;
    int* err;
};

struct Ctl {
    volatile uint32_t* abort;
    int* err;
};

// Waits for a phase, asleep between tries; gives up when another warp has, or after the limit.  What a wait that lasts
// does is out of line: the roles' loops share small instruction caches.
__device__ __noinline__ bool wait_long(volatile uint32_t* abort, int* err, uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, 500000u)) return true;
        if (*abort) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort = 1u;
            record_error(err, PKV_DEVERR_TIMEOUT, static_cast<int>(blockIdx.x));
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_phase(const Ctl& c, uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || mbar_try_wait_sleep(bar, parity, 100000u) || wait_long(c.abort, c.err, bar, parity);
}
__device__ __forceinline__ bool wait_warp(const Ctl& c, uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_phase(c, bar, parity));
}
// Both phases, asked for side by side: shared memory answers late beside the products' reads.
__device__ __forceinline__ bool wait_both(const Ctl& c, uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1) {
    const bool x = mbar_try_wait(bar0, parity0), y = mbar_try_wait(bar1, parity1);
    return (x || wait_phase(c, bar0, parity0)) && (y || wait_phase(c, bar1, parity1));
}
__device__ __noinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait_sleep(bar, parity, 500000u))
        if (global_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

__device__ __noinline__ void complain(int* err, int code, int info) { record_error(err, code, info); }

struct Seq {
    int q0, n, len;       // first node's row, nodes (0: nothing to do), keys
    bool bad;
};
__device__ __forceinline__ Seq sequence(const Params& p, int b) {
    Seq s;
    s.q0 = __ldg(p.cu_nodes + b);
    const int q1 = __ldg(p.cu_nodes + b + 1);
    s.len = __ldg(p.context_lens + b);
    const long long n = static_cast<long long>(q1) - s.q0;
    const bool fits = s.q0 >= 0 && n > 0 && q1 <= p.total_nodes && n <= p.max_nodes && n <= s.len && s.len <= p.max_context &&
                      s.len <= static_cast<long long>(p.max_blocks) * p.block_size;
    s.bad = n != 0 && !fits;
    s.n = fits ? static_cast<int>(n) : 0;
    return s;
}
__device__ __forceinline__ int tiles_of(const Params& p, const Seq& s) { return (s.n + p.qtok - 1) / p.qtok; }      // of rows
__device__ __forceinline__ int cost_of(const Seq& s) { return s.n ? (s.len + KT - 1) / KT + UNIT_COST : 0; }           // of each

// A CTA's run, segment by segment: tiles [j0, j1) of the unit (sequence b, row tile rt).  Runs are cut in
// cost: a unit is UNIT_COST steps without a tile and then a step per tile.  Every role walks by itself.
// only: the one row tile of each sequence that is walked, or -1 for all of them.
struct Walk {
    const Params& p;
    Seq s;
    int b, rt, j0, j1, only;
    long long left;                          // cost of the run behind this segment

    __device__ __forceinline__ Walk(const Params& params, int b0, long long off, long long cost, int only_rt) : p(params), b(b0), only(only_rt) {
        j0 = j1 = 0;
        rt = max(0, only);
        left = cost;
        if (cost <= 0) return;
        s = sequence(p, b);
        const int per = nt() + UNIT_COST, before = static_cast<int>(off / per);
        const int at = static_cast<int>(off - static_cast<long long>(before) * per);
        rt += before;                        // 0 where one row tile is walked
        j0 = max(0, at - UNIT_COST);
        clip(max(0, UNIT_COST - at));
        if (j0 == j1) next();                // nothing of the last unit's steps but its first ones
    }
    __device__ __forceinline__ int nt() const { return (s.len + KT - 1) / KT; }        // tiles of the unit
    __device__ __forceinline__ void clip(int before) {
        j1 = static_cast<int>(min(static_cast<long long>(nt()), max(static_cast<long long>(j0), j0 + left - before)));
        left -= before + (j1 - j0);
    }
    __device__ __forceinline__ bool last() const { return left <= UNIT_COST; }     // no tile of this run lies behind this segment
    __device__ __forceinline__ bool more() const { return j1 > j0; }
    __device__ __forceinline__ void next() {
        j1 = j0 = 0;
        if (last()) return;
        if (only >= 0 || ++rt == tiles_of(p, s)) {
            rt = max(0, only);
            do {
                if (++b >= p.batch) return;
                s = sequence(p, b);
            } while (s.n == 0);
        }
        clip(UNIT_COST);
    }
    __device__ __forceinline__ int tokens() const { return min(p.qtok, s.n - rt * p.qtok); }
    // the physical block of logical block lb; negative: no such block
    __device__ __forceinline__ int block_of(int lb) const {
        const int phys = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks + lb);
        if (phys >= 0 && phys < p.num_blocks) return phys;
        complain(p.err, PKV_DEVERR_BLOCK_ID, b);
        return -1;
    }
};

// A tile's products, issued by one elected lane in one piece: with the descriptors advanced by constants (1% of a call against an
// election for each).
// S = Q K^T, bf16: 8 steps of 16 dims, 64 dims to a half of each tile.
__device__ __forceinline__ void issue_qk_bf16(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
    static_assert(Q_HALF >> 4 == 1024 && KV_HALF >> 4 == 512, "offsets below");
    asm volatile(
        "{\n\t"
        ".reg .pred e, f, t;\n\t"
        ".reg .b32 r;\n\t"
        ".reg .b64 a, b;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.u32 f, 0, 0;\n\t"
        "setp.eq.u32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
        "add.u64 a, %1, 2;\n\t"
        "add.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 4;\n\t"
        "add.u64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 6;\n\t"
        "add.u64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1024;\n\t"
        "add.u64 b, %2, 512;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1026;\n\t"
        "add.u64 b, %2, 514;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1028;\n\t"
        "add.u64 b, %2, 516;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1030;\n\t"
        "add.u64 b, %2, 518;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "}" :: "r"(d), "l"(q), "l"(k), "r"(idesc)
        : "memory");
}

// S = (Q's two parts) K^T, e4m3: 4 steps of 32 dims for each part.
__device__ __forceinline__ void issue_qk_e4m3(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
    asm volatile(
        "{\n\t"
        ".reg .pred e, f, t;\n\t"
        ".reg .b32 r;\n\t"
        ".reg .b64 a, b;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.u32 f, 0, 0;\n\t"
        "setp.eq.u32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
        "add.u64 a, %1, 2;\n\t"
        "add.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 4;\n\t"
        "add.u64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 6;\n\t"
        "add.u64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1024;\n\t"
        "add.u64 b, %2, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1026;\n\t"
        "add.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1028;\n\t"
        "add.u64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 1030;\n\t"
        "add.u64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "}" :: "r"(d), "l"(q), "l"(k), "r"(idesc)
        : "memory");
}

// O (+)= P V, P in TMEM: `steps` (1 to 4) of 16 keys.
__device__ __forceinline__ void issue_pv_ts(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t accumulate, uint32_t steps) {
    asm volatile(
        "{\n\t"
        ".reg .pred e, f, t;\n\t"
        ".reg .b32 r, a;\n\t"
        ".reg .b64 b;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.u32 f, %4, 0;\n\t"
        "setp.eq.u32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
        "setp.gt.and.u32 e, %5, 1, e;\n\t"
        "add.u32 a, %1, 8;\n\t"
        "add.u64 b, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "setp.gt.and.u32 e, %5, 2, e;\n\t"
        "add.u32 a, %1, 16;\n\t"
        "add.u64 b, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "setp.gt.and.u32 e, %5, 3, e;\n\t"
        "add.u32 a, %1, 24;\n\t"
        "add.u64 b, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "}" :: "r"(d), "r"(p), "l"(v), "r"(idesc), "r"(accumulate), "r"(steps)
        : "memory");
}

// Arrive on two barriers, and on a third if it is not 0, once all products issued before are through.
__device__ __forceinline__ void commit3(uint32_t a, uint32_t b, uint32_t c) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t"
        "setp.ne.and.u32 e, %2, 0, e;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%2];\n\t}" ::"r"(a), "r"(b), "r"(c)
        : "memory");
}

// Which of a tile's keys a node sees: bit e for key 64 j + e.
__device__ __forceinline__ unsigned long long visible(const unsigned long long (&w)[4], int rel, int keys) {
    // rel: node of the tile's first key (negative before the tree); keys: keys of the sequence in this tile
    unsigned long long m;
    if (rel < 0) {
        m = rel <= -64 ? ~0ull : (w[0] << -rel) | ((1ull << -rel) - 1ull);
    } else {
        const int i = rel >> 6, sh = rel & 63;
        const unsigned long long lo = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
        const unsigned long long hi = i == 0 ? w[1] : i == 1 ? w[2] : i == 2 ? w[3] : 0ull;
        m = sh ? (lo >> sh) | (hi << (64 - sh)) : lo;
    }
    return keys >= 64 ? m : m & ((1ull << keys) - 1ull);
}

// Two bf16 of which at least one is an infinity or a NaN.
__device__ __forceinline__ bool wild2(uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four numbers rounded to e4m3, the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// Two bytes of w, each as 16 bits with its sign in the upper eight: bytes 0 and 1 by the selector 0x9180, 2 and 3 by 0xb3a2.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(d) : "r"(w), "n"(SEL));
    return d;
}

// 16 e4m3 codes and their row's scale byte as 16 bf16.  A code's bits, set one exponent field further, read as a bf16
// 2^-120 times its value (its subnormals as bf16's), so a product with 2^120 times the scale is exact where bf16 holds that
// factor, scales of 2^-119 to 2^7.  Rows with other scales or with a NaN code (ODD) go by way of f16 and fp32.
__device__ __forceinline__ bool odd_row(const uint4& c, uint32_t byte) {      // a NaN code, or a scale outside 2^-119 .. 2^7
    const uint32_t nan = ((c.x & 0x7f7f7f7fu) + 0x01010101u) | ((c.y & 0x7f7f7f7fu) + 0x01010101u) | ((c.z & 0x7f7f7f7fu) + 0x01010101u) |
                         ((c.w & 0x7f7f7f7fu) + 0x01010101u);
    return (nan & 0x80808080u) != 0u || byte - 8u > 126u;
}
template <bool ODD>
__device__ __forceinline__ void bf16_of_row(const uint4& c, uint32_t byte, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    const uint32_t f = (byte + 120u) * 0x00800080u;                  // 2^(120 + e) twice
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ODD) {
            const uint2 x = bf16_of_codes(w[i], e8m0_value(byte));
            o[2 * i] = x.x;
            o[2 * i + 1] = x.y;
        } else {
            o[2 * i] = hmul2((widen<0x9180u>(w[i]) << 4) & 0x87f087f0u, f);
            o[2 * i + 1] = hmul2((widen<0xb3a2u>(w[i]) << 4) & 0x87f087f0u, f);
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// A query row for the product with codes.  With f the power of two that takes the row's largest |q| to [128, 256), q f
// is a sum of two e4m3 numbers, the nearest one and what is left: exactly where |q| is 2^-9 of the largest or more (8 bits
// are 4 + 4, the last one 2^-9), and to 2^-17 of the largest otherwise (half of e4m3's smallest step, 2^-9, beside 128).  The row is replaced by its two parts, each laid out as 128
// bytes of a K-major tile; *factor gets scale / f, or kBadRow for a row with an infinity or a NaN.  Eight lanes take a row, lane v
// dims 16 v .. 16 v + 15; all of a warp's lanes call.
__device__ __forceinline__ void split_row(uint8_t* q, int row, int v, float scale, float* factor) {
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 c = *reinterpret_cast<const uint4*>(q + (v >> 2) * Q_HALF + row * 128 + ((((2 * v + i) & 7) ^ (row & 7)) * 16));
        x[4 * i] = c.x;
        x[4 * i + 1] = c.y;
        x[4 * i + 2] = c.z;
        x[4 * i + 3] = c.w;
    }
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = x[i] & 0x7fff7fffu;
        asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(a));
    }
    most = max(most & 0xffffu, most >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));      // the row is read, too
    const uint32_t e = max(8u, most >> 7);                                       // exponent field of the largest
    const float f = __uint_as_float((261u - e) << 23);                           // 2^(134 - e)
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t a = x[2 * k], b = x[2 * k + 1];
        const float y0 = bf16_lo(a) * f, y1 = bf16_hi(a) * f, y2 = bf16_lo(b) * f, y3 = bf16_hi(b) * f;
        hi[k] = e4m3x4(y0, y1, y2, y3);
        uint32_t h0, h1;
        f16_of_codes(hi[k], h0, h1);
        const float2 z0 = __half22float2(*reinterpret_cast<const __half2*>(&h0)), z1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        lo[k] = e4m3x4(y0 - z0.x, y1 - z0.y, y2 - z1.x, y3 - z1.y);
    }
    uint8_t* at = q + row * 128 + ((v ^ (row & 7)) * 16);
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + Q_HALF) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (v == 0) {
        // a factor below fp32's range is one of scores next to 0 (the products are below 2^125): the smallest number does as well
        const float x = fmaxf(scale * __uint_as_float((e - 7u) << 23), 0x1p-149f);
        *factor = e == 255u ? kBadRow : x == kBadRow ? 0x1p-126f : x;
    }
}

// The infinities and NaN that were taken out of the V rows of a segment's nodes, added to O in the rows that see the
// node: wild holds a bit for every node of which something was taken, four sets that the warps found.
template <bool FP8>
__device__ __noinline__ void give_back(const Params& p, int seq, int n, int len, int j0, int j1, int g, const uint32_t* wild, unsigned long long m0, unsigned long long m1,
                                       unsigned long long m2, unsigned long long m3, bool live, uint32_t o_tmem) {
    for (int i = 0; i < n; ++i) {
        const uint32_t* x = wild + (i >> 5);
        if (!(((x[0] | x[8] | x[16] | x[24]) >> (i & 31)) & 1u)) continue;
        const int pos = len - n + i, lb = pos / p.block_size;
        const int phys = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks + lb);
        if (pos / KT < j0 || pos / KT >= j1 || phys < 0 || phys >= p.num_blocks) continue;
        const bool sees = live && ((i < 64 ? m0 : i < 128 ? m1 : i < 192 ? m2 : m3) >> (i & 63)) & 1ull;
        const int64_t head = static_cast<int64_t>(phys) * p.num_kv_heads + g;
        const int64_t row = (static_cast<int64_t>(phys) * p.block_size + (pos - lb * p.block_size)) * p.num_kv_heads + g;
        const float f = FP8 ? e8m0_value(__ldg(p.v_scale + head * p.block_size + (pos - lb * p.block_size))) : 1.f;
        for (int d = 0; d < D; ++d) {
            const float v = FP8 ? bf16_lo(bf16_of_codes(__ldg(p.v_codes + row * D + d), f).x)
                                : __uint_as_float(static_cast<uint32_t>(__ldg(p.v_cache + row * D + d)) << 16);
            if (fabsf(v) <= 3.4028235e38f) continue;
            const float o = __uint_as_float(tmem_ld1(o_tmem + d));
            tmem_ld_wait();
            tmem_st1(o_tmem + d, __float_as_uint(sees ? o + v : o));
            tmem_st_wait();
        }
    }
}

template <bool FP8>
__global__ void __launch_bounds__(FP8 ? THREADS_FP8 : THREADS_BF16, CTAS_PER_SM)
tree_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const Params p) {
    constexpr int THREADS = FP8 ? THREADS_FP8 : THREADS_BF16, LOAD_WARP = FP8 ? 9 : 4, MMA_WARP = FP8 ? 8 : 5;
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_u32(gbase);
    using L = Layout<FP8>;
    const uint32_t sQ = base + L::Q, bars = base + L::BAR;
    auto bar = [&](int i) { return bars + 8u * i; };
    uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + L::MISC);
    long long* scan = reinterpret_cast<long long*>(gbase + L::SCAN);
    Ctl ctl{reinterpret_cast<volatile uint32_t*>(misc + 1), p.err};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < L::NUM_BARS; ++i) {
            const bool per_warp = i == L::PF || i == L::PF + 1 || i == L::OE || i == L::WG || (FP8 && ((i >= L::VF && i < L::VE) || i == L::QR));
            mbar_init(bar(i), per_warp ? 4 : FP8 && i >= L::KSR && i < L::QR ? 2 : 1);
        }
        misc[1] = 0u;
        fence_barrier_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == MMA_WARP) {
        tmem_alloc(base + L::MISC, TMEM_COLS);
        tmem_relinquish();
    }
    // everything above overlaps the kernel before this one; global memory is read and written from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The run: all tiles are counted, then the sequence in which this CTA's share starts is searched, a
    // block of sequences at a time.
    constexpr int WARPS = THREADS / 32;
    auto block_scan = [&](long long v, long long& total) {      // inclusive sums over the CTA's threads
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = v;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll 1
        for (int i = 0; i < WARPS; ++i) {
            const long long x = scan[i];
            before += i < warp ? x : 0;
            total += x;
        }
        return before + v;
    };
    // Sums over the sequences of a row tile's cost, alone (x) and times the row tiles (y).  Where every sequence has the same
    // number of row tiles, more than one, they are taken side by side like the KV heads, by neighbouring CTAs: what one
    // reads from memory the other finds in L2 (33 to 64 nodes of 4 heads, batch of 32: 73 us and 270 MB read).  Elsewhere
    // they go one after the other (the same with one tree of one node: 85 us and 398 MB).
    long long x = 0, y = 0, x_first = 0, y_first = 0;
    int least = 0x7fffffff, most = 0;
#pragma unroll 1
    for (int b = tid; b < p.batch; b += THREADS) {
        const Seq s = sequence(p, b);
        if (s.bad && blockIdx.x == 0) complain(p.err, PKV_DEVERR_SEQLENS, b);
        const long long cost = cost_of(s);
        const int tiles = tiles_of(p, s);
        if (tiles > 0) {
            least = min(least, tiles);
            most = max(most, tiles);
        }
        if (b < THREADS) {
            x_first = cost;
            y_first = cost * tiles;
        }
        x += cost;
        y += cost * tiles;
    }
    long long W, Wx;
    long long upto = block_scan(y, W);
    int rts = 1;                                              // row tiles side by side
    if (p.max_nodes > p.qtok) {
        const long long upto_x = block_scan(x, Wx);
        const int r = Wx > 0 ? static_cast<int>(W / Wx) : 1;
        if (r > 1 && static_cast<int>(gridDim.x) >= r * p.num_kv_heads && __syncthreads_and(most == 0 || (least == r && most == r))) {
            rts = r;
            W = Wx;
            upto = upto_x;
        }
    }
    const int lanes = rts * p.num_kv_heads;                   // CTAs that walk the same run
    const long long C = max(1ll, min(static_cast<long long>(gridDim.x / lanes), W / MIN_RUN));
    const long long c = blockIdx.x / lanes;
    const int rt_mine = static_cast<int>(blockIdx.x - c * lanes) / p.num_kv_heads;
    const int g = static_cast<int>(blockIdx.x - c * lanes) - rt_mine * p.num_kv_heads;
    const long long t0 = c < C ? c * W / C : 0, t1 = c < C ? (c + 1) * W / C : 0;
    if (t1 > t0) {
        long long before = 0;
#pragma unroll 1
        for (int base_b = 0; base_b < p.batch; base_b += THREADS) {
            const int b = base_b + tid;
            long long v = 0, total = W;
            if (p.batch <= THREADS) {
                v = rts > 1 ? x_first : y_first;             // one block: its sums are known
            } else {
                if (b < p.batch) {
                    const Seq s = sequence(p, b);
                    v = static_cast<long long>(cost_of(s)) * (rts > 1 ? 1 : tiles_of(p, s));
                }
                upto = block_scan(v, total);
            }
            const long long at = before + upto;
            if (t0 >= at - v && t0 < at) {
                scan[14] = b;
                scan[15] = t0 - (at - v);
            }
            before += total;
            if (before > t0) break;
        }
    }
    if (tid == 0) {                                           // what the end of a unit asks for, out of the registers until then
        scan[10] = lanes;
        scan[11] = t1;
        scan[12] = C;
        scan[13] = W;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const bool busy = t1 > t0;
    Walk w(p, busy ? static_cast<int>(scan[14]) : 0, busy ? scan[15] : 0, t1 - t0, rts > 1 ? rt_mine : -1);

    if (warp == LOAD_WARP) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0 && busy) {
            int kt = 0, vt = 0, segs = 0;                     // K, V and Q tiles issued
            bool ok = true;
            auto load_k = [&](int phys, int off) {
                const int slot = kt % L::K_SLOTS;
                if (kt >= L::K_SLOTS && !(ok = wait_phase(ctl, bar(L::KE + slot), ((kt / L::K_SLOTS) - 1) & 1))) return;
                const uint32_t dst = base + L::K + slot * L::K_TILE, full = bar(L::KF + slot);
                mbar_arrive_expect_tx(full, L::K_TILE);
                tma_load_4d(dst, &tm_k, full, 0, g, off, phys);
                if (FP8) {
                    const int64_t at = (static_cast<int64_t>(max(phys, 0)) * p.num_kv_heads + g) * p.block_size + off;
                    const int s = kt % L::KS_SLOTS;
                    mbar_arrive_expect_tx(bar(L::KSB + s), KT);
                    bulk_load(base + L::KS + s * KT, p.k_scale + at, KT, bar(L::KSB + s));
                } else {
                    tma_load_4d(dst + KV_HALF, &tm_k, full, 64, g, off, phys);
                }
                ++kt;
            };
            auto load_v = [&](int phys, int off) {
                const int slot = vt % L::V_SLOTS;
                if (vt >= L::V_SLOTS && !(ok = wait_phase(ctl, bar(L::VE + slot), ((vt / L::V_SLOTS) - 1) & 1))) return;
                const uint32_t dst = base + L::V + slot * KV_TILE, full = bar((FP8 ? L::VRAW : L::VF) + slot);
                if (FP8) {
                    // codes to the slot's second half, where the warp that decodes a row finds and overwrites it
                    const int64_t at = (static_cast<int64_t>(max(phys, 0)) * p.num_kv_heads + g) * p.block_size + off;
                    mbar_arrive_expect_tx(full, KV_HALF + KT);
                    tma_load_4d(dst + KV_HALF, &tm_v, full, 0, g, off, phys);
                    bulk_load(base + L::VS + slot * KT, p.v_scale + at, KT, full);
                } else {
                    mbar_arrive_expect_tx(full, KV_TILE);
                    tma_load_4d(dst, &tm_v, full, 0, g, off, phys);
                    tma_load_4d(dst + KV_HALF, &tm_v, full, 64, g, off, phys);
                }
                ++vt;
            };
            auto load_q = [&] {
                if (segs >= 1 && !(ok = wait_phase(ctl, bar(L::QE), (segs - 1) & 1))) return;
                mbar_arrive_expect_tx(bar(L::QF), 2 * Q_HALF);
                const int row = w.s.q0 + w.rt * p.qtok, head = g << p.lg;
                tma_load_3d(sQ, &tm_q, bar(L::QF), 0, head, row);
                tma_load_3d(sQ + Q_HALF, &tm_q, bar(L::QF), 64, head, row);
                ++segs;
            };
            // K of a tile, then V of the one before; a segment's queries behind the first K.  Tile j lies in logical
            // block lb, at key off.
            int j = w.j0, lb = j * KT / p.block_size, off = j * KT - lb * p.block_size, phys = w.block_of(lb), v_phys = 0, v_off = 0;
            bool more = true;
#pragma unroll 1
            for (int t = 0; ok; ++t) {
                if (more) load_k(phys, off);
                if (ok && t > 0) load_v(v_phys, v_off);
                if (!ok || !more) break;
                if (j == w.j0) load_q();
                v_phys = phys;
                v_off = off;
                off += KT;
                if (++j == w.j1) {
                    more = !w.last();
                    if (more) {                               // every segment behind a run's first starts at its first key
                        w.next();
                        j = lb = off = 0;
                        phys = w.block_of(0);
                    }
                } else if (off == p.block_size) {
                    off = 0;
                    phys = w.block_of(++lb);
                }
            }
            if (*ctl.abort) {
                // copies in flight land before shared memory is released
                if (segs > 0) wait_drain(bar(L::QF), (segs - 1) & 1);
                for (int i = max(0, kt - L::K_SLOTS); i < kt; ++i) wait_drain(bar(L::KF + i % L::K_SLOTS), (i / L::K_SLOTS) & 1);
                for (int i = max(0, vt - L::V_SLOTS); i < vt; ++i) wait_drain(bar((FP8 ? L::VRAW : L::VF) + i % L::V_SLOTS), (i / L::V_SLOTS) & 1);
                if (FP8)
                    for (int i = max(0, kt - L::KS_SLOTS); i < kt; ++i)
                        wait_drain(bar(L::KSB + i % L::KS_SLOTS), (i / L::KS_SLOTS) & 1);
            }
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    } else if (FP8 && warp >= 4 && warp < 8) {
        // ---------------------------------------------------------------- 8-bit V rows to bf16 tiles
        // Warp x decodes rows 16 x .. 16 x + 15 of each tile.  Their codes lie where the second half of their values
        // will, so a warp that has read its rows may write them.  Eight lanes take half of two rows whose numbers
        // differ in bits 0 and 2: with the chunks of the codes (as TMA has put them) and of the values at an exclusive
        // or with the row, neither the loads nor the stores meet in a bank.
        const int half = (lane >> 3) & 1, vec = half * 4 + (lane & 3);
        // per tile: its K scales to floats, by the first two warps; V of the tile before; and, where it is a segment's
        // first, the segment's queries
        int j = w.j0, seg = 0;
        bool more = busy, ok = true;
#pragma unroll 1
        for (int t = 0; ok; ++t) {
            if (more && warp < 6) {
                const int s = t % L::KS_SLOTS, key = tid - 4 * 32;
                if (!(ok = wait_warp(ctl, bar(L::KSB + s), (t / L::KS_SLOTS) & 1))) break;
                reinterpret_cast<float*>(gbase + L::KSF)[s * KT + key] = e8m0_value(gbase[L::KS + s * KT + key]);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::KSR + s));
            }
            if (t > 0) {
                const int u = t - 1;
                const int slot = u % L::V_SLOTS;
                if (!(ok = wait_warp(ctl, bar(L::VRAW + slot), (u / L::V_SLOTS) & 1))) break;
                uint8_t* tile = gbase + L::V + slot * KV_TILE;
                const uint8_t* scales = gbase + L::VS + slot * KT;
                // rolled, four rows at a time: this code and the softmax's share the schedulers' instruction caches
#pragma unroll 1
                for (int i = 0; i < 16; i += 4) {
                    const int row = (warp - 4) * 16 + ((2 * (lane >> 4) + i) ^ (lane & 4 ? 5 : 0)), ch = (lane & 3) * 2;
                    const uint4 c = *reinterpret_cast<const uint4*>(tile + KV_HALF + row * 128 + ((vec ^ (row & 7)) * 16));
                    const uint32_t byte = scales[row];
                    uint4 lo, hi;
                    if (__any_sync(0xffffffffu, odd_row(c, byte)))       // and every lane has read its part of these rows
                        bf16_of_row<true>(c, byte, lo, hi);
                    else
                        bf16_of_row<false>(c, byte, lo, hi);
                    uint8_t* dst = tile + half * KV_HALF + row * 128;
                    *reinterpret_cast<uint4*>(dst + ((ch ^ (row & 7)) * 16)) = lo;
                    *reinterpret_cast<uint4*>(dst + (((ch + 1) ^ (row & 7)) * 16)) = hi;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::VF + slot));
            }
            if (!more) break;
            if (j == w.j0) {
                if (!(ok = wait_warp(ctl, bar(L::QF), seg & 1))) break;
                const int rows = w.tokens() << p.lg;
                float* factors = reinterpret_cast<float*>(gbase + L::QS) + (seg & 1) * ROWS;
#pragma unroll 1
                for (int r = (warp - 4) * 4 + (lane >> 3); r - (lane >> 3) < rows; r += 16) split_row(gbase + L::Q, r, lane & 7, p.scale_log2, factors + r);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::QR));
                ++seg;
            }
            if (++j == w.j1) {
                more = !w.last();
                if (more) w.next();
                j = w.j0;
            }
        }
        tc_fence_before();
        __syncthreads();
    } else if (warp == MMA_WARP) {
        // ---------------------------------------------------------------- MMA
        // The whole warp runs this loop in step; each tcgen05 instruction is issued by one elected lane.
        constexpr uint32_t idesc_qk = idesc_bf16_f32(ROWS, KT, 0, 0);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(ROWS, D, 0, 1);
        const uint64_t dq = smem_desc(sQ, 16, 1024, 2);
        int segs = 0;                                         // segments whose S has begun
        int oseg = 0;                                         // segments whose O has begun
        bool ok = busy;
        auto issue_s = [&](int t, bool seg_first, bool seg_last) {
            if (seg_first) {
                if (!(ok = wait_warp(ctl, bar(FP8 ? L::QR : L::QF), segs & 1))) return;
                if (FP8 && lane == 0) mbar_arrive(bar(L::QG));        // the rows' factors, to the softmax
                __syncwarp();
                ++segs;
            }
            const int slot = t % L::K_SLOTS;
            if (!(ok = wait_warp(ctl, bar(L::KF + slot), (t / L::K_SLOTS) & 1))) return;
            tc_fence_after();
            const uint64_t dk = smem_desc(base + L::K + slot * L::K_TILE, 16, 1024, 2);
            if (FP8)
                issue_qk_e4m3(tmem + (t & 1) * KT, dq, dk, idesc_e4m3_f32(ROWS, KT));     // the codes themselves, and Q's two parts
            else
                issue_qk_bf16(tmem + (t & 1) * KT, dq, dk, idesc_qk);
            commit3(bar(L::SF + (t & 1)), bar(L::KE + slot), seg_last ? bar(L::QE) : 0u);
        };
        // S of a tile goes ahead of the product with V of the tile before it, as long as both are of one segment
        int j = w.j0, t = 0, s = 0;
#pragma unroll 1
        while (ok) {
            if (s == t) {
                issue_s(s, true, j + 1 == w.j1);
                ++s;
                if (!ok) break;
            }
            if (j + 1 < w.j1) {
                issue_s(s, false, j + 2 == w.j1);
                ++s;
                if (!ok) break;
            }
            const bool first_here = j == w.j0, last_here = j + 1 == w.j1, end = last_here && w.last();
            const int keys = min(KT, w.s.len - j * KT);
            if (first_here) {
                if (oseg >= 1 && !(ok = wait_warp(ctl, bar(L::OE), (oseg - 1) & 1))) break;
                ++oseg;
            }
            const int slot = t % L::V_SLOTS;
            if (!(ok = __all_sync(0xffffffffu, wait_both(ctl, bar(L::VF + slot), (t / L::V_SLOTS) & 1, bar(L::PF + (t & 1)), (t >> 1) & 1)))) break;
            tc_fence_after();
            const uint64_t dv = smem_desc(base + L::V + slot * KV_TILE, KV_HALF, 1024, 2);
            issue_pv_ts(tmem + O_COL, tmem + (t & 1) * KT, dv, idesc_pv, first_here ? 0u : 1u, (keys + 15) >> 4);
            commit3(bar(L::PV + (t & 1)), bar(L::VE + slot), last_here ? bar(L::OF) : 0u);
            if (end) break;
            if (last_here) w.next();
            j = last_here ? w.j0 : j + 1;
            ++t;
        }
        mma_commit_warp(bar(L::DRAIN));
        wait_drain(bar(L::DRAIN), 0);
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    } else {
        // ---------------------------------------------------------------- softmax and epilogue
        const int row = tid;                                  // TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const int qtok = p.qtok;
        int t = 0, seg = 0;
        bool ok = true;
        int4 meta = make_int4(-1, 0, 0, 0);
        uint32_t* wild = reinterpret_cast<uint32_t*>(gbase + L::WILD);
        uint32_t meets = 0;
        auto meet = [&] {                                     // a barrier of the four warps that gives up with the others
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::WG));
            ok = wait_warp(ctl, bar(L::WG), meets++ & 1u);
            return ok;
        };
        for (; w.more() && ok; w.next(), ++seg) {
            const int tokens = w.tokens();
            const int tok = row >> p.lg;
            const bool live = tok < tokens;                   // rows behind are computed by nobody
            const bool warp_live = (warp * 32) >> p.lg < tokens;
            const int tree0 = w.s.len - w.s.n;                // position of the first node
            const int node_row = w.s.q0 + w.rt * qtok + tok;
            unsigned long long words[4];
            auto load_words = [&] {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    words[i] = live && i < p.mask_words ? __ldg(p.mask + static_cast<int64_t>(node_row) * p.mask_words + i) : 0ull;
            };
            if (!FP8) load_words();
            float m_used = -INFINITY, l = 0.f, sc = p.scale_log2;
            // 8 bits: what the sum of weights may be: more moves the reference, and so does anything where nothing has been seen yet
            float most = live ? -1.f : INFINITY;
            bool had_tree = false;
            if (FP8) {
                ok = wait_warp(ctl, bar(L::QG), seg & 1);
                if (!ok) break;
                sc = reinterpret_cast<const float*>(gbase + L::QS)[(seg & 1) * ROWS + row];
            }
            for (int j = w.j0; j < w.j1; ++j, ++t) {
                const int keys = min(KT, w.s.len - j * KT), rel = j * KT - tree0;
                const bool tree = rel + KT > 0;               // nodes among the keys: on no more than the last few tiles
                const uint32_t ksf = base + L::KSF + (t % L::KS_SLOTS) * KT * 4;
                // K scales of the first 16 of the 32 columns that are read next: beside the products' own reads of shared
                // memory a load takes some 180 cycles
                uint4 kf[4];
                auto fetch = [&](int c0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) kf[e] = ld_shared_v4(ksf + 4 * ((c0 & (KT - 1)) + 4 * e));
                };
                if (FP8 && warp_live)
                    ok = __all_sync(0xffffffffu, wait_both(ctl, bar(L::KSR + t % L::KS_SLOTS), (t / L::KS_SLOTS) & 1, bar(L::SF + (t & 1)), (t >> 1) & 1));
                else
                    ok = wait_warp(ctl, bar(L::SF + (t & 1)), (t >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                if (warp_live) {
                    const uint32_t s_tmem = tmem + lane_off + (t & 1) * KT;
                    if (FP8 && tree) load_words();
                    const unsigned long long see = tree ? visible(words, rel, keys) : ~0ull;
                    // bf16: all of S in registers.  8 bits: CH columns at a time, in rolled loops.
                    constexpr int CH = FP8 ? 32 : KT;
                    float s[CH];
                    auto read = [&](int c0) {
                        if constexpr (FP8) {
                            uint32_t r[32];
                            tmem_ld32(s_tmem + c0, r);
                            uint4 k2[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) k2[e] = ld_shared_v4(ksf + 4 * (c0 + 16 + 4 * e));
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const uint4 f = e < 16 ? kf[(e >> 2) & 3] : k2[(e >> 2) & 3];
                                fmul2(s[e], s[e + 1], __uint_as_float(r[e]), __uint_as_float(r[e + 1]), __uint_as_float(f.x), __uint_as_float(f.y));
                                fmul2(s[e + 2], s[e + 3], __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]), __uint_as_float(f.z), __uint_as_float(f.w));
                            }
                            fetch(c0 + 32);
                        } else {
                            uint32_t r[2][32];
                            tmem_ld32(s_tmem, r[0]);
                            tmem_ld32(s_tmem + 32, r[1]);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < KT; ++e) s[e] = __uint_as_float(r[e >> 5][e & 31]);
                        }
                        if (tree) {
                            const unsigned long long m = see >> c0;
                            const uint32_t lo = static_cast<uint32_t>(m), hi = static_cast<uint32_t>(m >> 32);
#pragma unroll
                            for (int e = 0; e < CH; ++e) s[e] = ((e < 32 ? lo : hi) >> (e & 31)) & 1u ? s[e] : -INFINITY;
                        }
                    };
                    auto largest = [&] {
                        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                        for (int e = 0; e < CH; e += 4) {
                            mx0 = fmax3(mx0, s[e + 0], s[e + 1]);
                            mx1 = fmax3(mx1, s[e + 2], s[e + 3]);
                        }
                        return fmaxf(mx0, mx1) * sc;
                    };
                    // O times alpha, once PV(t - 1) is through
                    auto rescale = [&](float alpha) {
                        ok = wait_warp(ctl, bar(L::PV + ((t - 1) & 1)), ((t - 1) >> 1) & 1);
                        if (!ok) return;
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < 4; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(tmem + lane_off + O_COL + 32 * cc, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tmem + lane_off + O_COL + 32 * cc, o);
                        }
                        tmem_st_wait();
                    };
                    // The reference of a row's weights is moved, and O rescaled, only when its own weights become large.  The warp
                    // does it together, but each row decides for itself: what another row sees may not decide when this one is
                    // rounded.  A row that is nobody's does not ask for it.
                    float r0 = 0.f, r1 = 0.f, r2 = 0.f, r3 = 0.f, neg_m;
                    if constexpr (!FP8) {
                        read(0);
                        const float m_new = largest();
                        const bool full = l > kMostSum, large = m_new > m_used + kMostWeightLog2;
                        if (j == w.j0) {
                            m_used = m_new + kLift;
                        } else if (__any_sync(0xffffffffu, live && (full || large))) {
                            const float m_tgt = full ? fmaxf(m_used, m_new) + kLift : large ? m_new + kLift : m_used;
                            const float alpha = m_tgt == m_used ? 1.f : ex2_ftz(m_used - m_tgt);
                            rescale(alpha);
                            if (!ok) break;
                            l *= alpha;
                            m_used = m_tgt;
                        }
                        neg_m = m_used == -INFINITY ? 0.f : -m_used;         // a row that has seen nothing yet
                    } else {
                        neg_m = m_used == -INFINITY ? 0.f : -m_used;
                        fetch(0);
                    }
#pragma unroll 1
                    for (int c0 = 0; c0 < KT; c0 += CH) {
                        if constexpr (FP8) read(c0);
                        uint32_t pk[CH / 2];
                        auto weigh = [&](float& x0, float& x1, float& x2, float& x3) {
#pragma unroll
                            for (int e = 0; e < CH; e += 4) {
                                float a0, a1, a2, a3;
                                ffma2(a0, a1, s[e], s[e + 1], sc, sc, neg_m, neg_m);
                                ffma2(a2, a3, s[e + 2], s[e + 3], sc, sc, neg_m, neg_m);
                                const float p0 = ex2_ftz(a0), p1 = ex2_ftz(a1), p2 = ex2_ftz(a2), p3 = ex2_ftz(a3);
                                if (FP8 && e == 0) {
                                    x0 = p0, x1 = p1, x2 = p2, x3 = p3;
                                } else {
                                    fadd2(x0, x1, x0, x1, p0, p1);
                                    fadd2(x2, x3, x2, x3, p2, p3);
                                }
                                pk[e >> 1] = pack_bf16x2(p0, p1);
                                pk[(e >> 1) + 1] = pack_bf16x2(p2, p3);
                            }
                        };
                        if constexpr (!FP8) {
                            weigh(r0, r1, r2, r3);
                            tmem_st32(s_tmem, pk);
                        } else {
                            // One pass: the sum with 32 more weights tells, before they are stored, that it has become too large.
                            // Then the rest of the tile is looked through for the new reference, a power of two, so that the
                            // weights that lie over S by then are scaled exactly.
                            float x0, x1, x2, x3;
                            weigh(x0, x1, x2, x3);
                            float x = (x0 + x1) + (x2 + x3);
                            const bool full = l + x > most;
                            if (__any_sync(0xffffffffu, full)) {
                                fetch(c0);
                                float m_new = -INFINITY;
#pragma unroll 1
                                for (int c = c0; c < KT; c += CH) {
                                    read(c);
                                    m_new = fmaxf(m_new, largest());
                                }
                                const float m_tgt = full ? fmaxf(m_used, ceilf(m_new)) + kLift : m_used, d = m_used - m_tgt;
                                const float alpha = m_tgt == m_used ? 1.f : d < -126.f ? 0.f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(d) + 127) << 23);
                                const uint32_t alpha2 = (__float_as_uint(alpha) >> 16) * 0x00010001u;
                                if (j > w.j0) {
                                    rescale(alpha);
                                    if (!ok) break;
                                }
                                tmem_st_wait();
#pragma unroll 1
                                for (int c = 0; c < c0; c += CH) {
                                    tmem_ld16(s_tmem + c / 2, pk);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) pk[e] = hmul2(pk[e], alpha2);
                                    tmem_st16(s_tmem + c / 2, pk);
                                }
                                l *= alpha;
                                m_used = m_tgt;
                                neg_m = m_used == -INFINITY ? 0.f : -m_used;
                                if (live && m_used != -INFINITY) most = kMostSum;
                                fetch(c0);
                                read(c0);
                                weigh(x0, x1, x2, x3);
                                x = (x0 + x1) + (x2 + x3);
                            }
                            l += x;
                            tmem_st16(s_tmem + c0 / 2, pk);         // P's columns end before the ones of S that are still to be read
                        }
                    }
                    if (!ok) break;
                    if (!FP8) l += (r0 + r1) + (r2 + r3);
                    tmem_st_wait();
                }
                if (tree) {
                    // Infinities and NaN among the nodes' V rows leave the tile, and so does what the block holds
                    // behind the last key: weights of 0 would spread them.
                    const int slot = t % L::V_SLOTS;
                    ok = wait_warp(ctl, bar(L::VF + slot), (t / L::V_SLOTS) & 1);
                    if (!ok) break;
                    uint32_t* mine = wild + ((seg & 1) * 4 + warp) * 8;
                    if (!had_tree && lane < 8) mine[lane] = 0u;
                    __syncwarp();
                    had_tree = true;
                    uint8_t* vt = gbase + L::V + slot * KV_TILE;
                    const int lo = max(0, -rel), hi = (keys + 15) & ~15;
                    for (int i = lo * 16 + tid; i < hi * 16; i += 128) {
                        const int r = i >> 4;
                        uint4* at = reinterpret_cast<uint4*>(vt + ((i >> 3) & 1) * KV_HALF + r * 128 + (i & 7) * 16);
                        if (r >= keys) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else {
                            const uint4 x = *at;
                            if (wild2(x.x) || wild2(x.y) || wild2(x.z) || wild2(x.w)) {
                                uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u;
                                    if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0x0000ffffu;
                                }
                                *at = make_uint4(y[0], y[1], y[2], y[3]);
                                atomicOr(mine + ((rel + r) >> 5), 1u << ((rel + r) & 31));
                            }
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::PF + (t & 1)));
            }
            if (!ok) break;
            ok = wait_warp(ctl, bar(L::OF), seg & 1);
            if (!ok) break;
            tc_fence_after();
            if (had_tree && !meet()) break;                   // every warp's bits are there; those of the segment before are read
            const bool whole = w.j0 == 0 && w.j1 == w.nt();
            const int part = w.j0 > 0 ? 0 : 1;                // 0: the unit began before this run, 1: it goes on behind it
            if (!whole && part == 1) {
                // its last run: that of the unit's last tile, which lies nt - j1 steps behind this run's end
                const long long end = scan[11] + (w.nt() - w.j1);
                meta = make_int4(static_cast<int>((end * scan[12] - 1) / scan[13]), w.s.q0 + w.rt * qtok, tokens, static_cast<int>(scan[10]));
            }
            if (warp_live) {
                if (FP8 && sc == kBadRow && l != 0.f) l = __uint_as_float(0x7fc00000u);      // it has seen a key
                if (had_tree) {
                    // what was taken out of the tiles, to the rows that see it
                    uint32_t any = 0u;
#pragma unroll 1
                    for (int i = 0; i < 32; ++i) any |= wild[(seg & 1) * 32 + i];
                    if (FP8 && any != 0u) load_words();
                    if (any != 0u) give_back<FP8>(p, w.b, w.s.n, w.s.len, w.j0, w.j1, g, wild + (seg & 1) * 32, words[0], words[1], words[2], words[3], live, tmem + lane_off + O_COL);
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + part;
                uint16_t* orow = p.out + (static_cast<int64_t>(node_row) * p.num_heads + (g << p.lg) + (row & ((1 << p.lg) - 1))) * D;
                if (!whole) p.part_ml[slot * ROWS + row] = make_float2(m_used, l);
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t o[32];
                    tmem_ld32(tmem + lane_off + O_COL + 32 * cc, o);
                    tmem_ld_wait();
                    if (whole) {
                        if (live) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint4 x;
                                x.x = pack_bf16x2(__uint_as_float(o[8 * q + 0]) * inv, __uint_as_float(o[8 * q + 1]) * inv);
                                x.y = pack_bf16x2(__uint_as_float(o[8 * q + 2]) * inv, __uint_as_float(o[8 * q + 3]) * inv);
                                x.z = pack_bf16x2(__uint_as_float(o[8 * q + 4]) * inv, __uint_as_float(o[8 * q + 5]) * inv);
                                x.w = pack_bf16x2(__uint_as_float(o[8 * q + 6]) * inv, __uint_as_float(o[8 * q + 7]) * inv);
                                *reinterpret_cast<uint4*>(orow + 32 * cc + 8 * q) = x;
                            }
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            p.part_o[(slot * 32 + 8 * cc + q) * ROWS + row] =
                                make_float4(__uint_as_float(o[4 * q]) * inv, __uint_as_float(o[4 * q + 1]) * inv, __uint_as_float(o[4 * q + 2]) * inv,
                                            __uint_as_float(o[4 * q + 3]) * inv);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::OE));
        }
        if (tid == 0) p.meta[blockIdx.x] = ok ? meta : make_int4(-1, 0, 0, 0);
        tc_fence_before();
        __syncthreads();
    }
}

// The units that several runs share: block (CTA, y) joins 32 columns of the unit that starts in the CTA's run and goes on
// behind it, a thread 16 columns of one row.
constexpr int JOIN_THREADS = 2 * ROWS, JOIN_SPLIT = 4;
// The pointers promise nothing (no __restrict__): the kernel is resident while the one before it still writes what they point at,
// and loads of memory that is constant as far as the compiler knows may be moved ahead of the wait.
__global__ void __launch_bounds__(JOIN_THREADS) tree_join_kernel(const float4* part_o, const float2* part_ml, const int4* meta, uint16_t* out, int num_heads,
                                                                 int num_kv_heads, int lg) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 u = meta[blockIdx.x];
    if (u.x < 0) return;
    const int lanes = u.w, c = blockIdx.x / lanes, in_run = blockIdx.x - c * lanes, g = in_run % num_kv_heads;
    const int row = threadIdx.x & (ROWS - 1), c4 = (blockIdx.y * 2 + (threadIdx.x >> 7)) * 4;
    if ((row >> lg) >= u.z) return;
    // the unit's first part is its run's second slot, all others are their runs' first
    auto slot = [&](int i) { return (static_cast<int64_t>(i) * lanes + in_run) * 2 + (i == c ? 1 : 0); };
    // The reference, the sum and the columns in one pass, two runs' loads at a time.  Parts are averages, and what is held is
    // the average of those that have gone by: no sum of theirs leaves fp32's range.
    float M = -INFINITY, l = 0.f, o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    for (int i0 = c; i0 <= u.x; i0 += 2) {
        float2 ml[2];
        float4 x[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t at = slot(min(i0 + i, u.x));
            ml[i] = i0 + i <= u.x ? part_ml[at * ROWS + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[i][k] = i0 + i <= u.x ? part_o[(at * 32 + c4 + k) * ROWS + row] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float now = fmax3(M, ml[0].x, ml[1].x);
        const float l0 = ml[0].x == now ? ml[0].y : ml[0].y * ex2_ftz(ml[0].x - now), l1 = ml[1].x == now ? ml[1].y : ml[1].y * ex2_ftz(ml[1].x - now);
        const float before = M == now ? l : l * ex2_ftz(M - now);
        M = now;
        l = before + l0 + l1;
        const float inv = l == 0.f ? 0.f : __fdividef(1.f, l), keep = before * inv, w0 = l0 * inv, w1 = l1 * inv;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[4 * k] = o[4 * k] * keep + x[0][k].x * w0 + x[1][k].x * w1;
            o[4 * k + 1] = o[4 * k + 1] * keep + x[0][k].y * w0 + x[1][k].y * w1;
            o[4 * k + 2] = o[4 * k + 2] * keep + x[0][k].z * w0 + x[1][k].z * w1;
            o[4 * k + 3] = o[4 * k + 3] * keep + x[0][k].w * w0 + x[1][k].w * w1;
        }
    }
    uint4* to = reinterpret_cast<uint4*>(out + (static_cast<int64_t>(u.y + (row >> lg)) * num_heads + (g << lg) + (row & ((1 << lg) - 1))) * D + 4 * c4);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        to[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                           pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
}

constexpr size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// As many CTAs as the bounds allow runs: never fewer than the lengths themselves ask for, so that how a batch is cut, and
// with it every rounding, does not depend on how tight the bounds are.
int64_t max_ctas(int num_kv_heads) {
    return std::max(1, CTAS_PER_SM * sm_count() / num_kv_heads) * static_cast<int64_t>(num_kv_heads);
}
int64_t grid_of(int batch, int max_nodes, int max_context, int num_kv_heads, int qtok) {
    const int64_t cost = static_cast<int64_t>(batch) * ((static_cast<int64_t>(max_context) + KT - 1) / KT + UNIT_COST) * ((max_nodes + qtok - 1) / qtok);
    return std::min<int64_t>(max_ctas(num_kv_heads), std::max<int64_t>(1, cost / MIN_RUN) * num_kv_heads);
}

template <bool FP8>
bool allow_smem() {
    return cudaFuncSetAttribute(tree_decode_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<FP8>::BYTES) == cudaSuccess;
}
template <bool FP8>
cudaError_t launch(int grid, cudaStream_t stream, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = programmatic(dim3(grid), FP8 ? THREADS_FP8 : THREADS_BF16, Layout<FP8>::BYTES, stream, attr);
    return cudaLaunchKernelEx(&cfg, tree_decode_kernel<FP8>, tm_q, tm_k, tm_v, p);
}

}  // namespace

size_t tree_decode_workspace_bytes(int num_kv_heads) {
    const size_t ctas = static_cast<size_t>(max_ctas(num_kv_heads));
    return std::max(align256(ctas * 2 * ROWS * D * 4) + align256(ctas * 2 * ROWS * 8) + align256(ctas * 16), tree_rows_workspace_bytes(num_kv_heads));
}

pkv_status launch_tree_decode(const TreeDecodeArgs& a, int* err, cudaStream_t stream) {
    const bool fp8 = a.k_scale != nullptr;
    const int lg = group_log2(a.num_heads, a.num_kv_heads);
    if (lg < 0) return PKV_ERR_UNSUPPORTED;
    const int qtok = ROWS >> lg;
    if (a.workspace == nullptr || a.workspace_bytes < tree_decode_workspace_bytes(a.num_kv_heads)) return PKV_ERR_WORKSPACE;
    if (!setup_once(kSetupTreeDecode, [] { return allow_smem<false>() && allow_smem<true>(); }))
        return PKV_ERR_CUDA;
    // by the bounds, not by the trees themselves
    if (tree_rows_fits(a, lg)) return launch_tree_rows(a, lg, err, stream);
    CUtensorMap tm_q, tm_k, tm_v;
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.num_heads), static_cast<uint64_t>(a.total_nodes)};
        const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.num_heads) * D * 2};
        const uint32_t box[3] = {64u, static_cast<uint32_t>(1 << lg), static_cast<uint32_t>(qtok)};
        if (encode_tiled(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return PKV_ERR_INVALID_ARG;
    }
    {
        const uint64_t row = static_cast<uint64_t>(D) * (fp8 ? 1 : 2);
        const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.num_kv_heads), static_cast<uint64_t>(a.block_size),
                                  static_cast<uint64_t>(a.num_blocks)};
        const uint64_t strides[3] = {row, a.num_kv_heads * row, static_cast<uint64_t>(a.block_size) * a.num_kv_heads * row};
        const uint32_t box[4] = {fp8 ? 128u : 64u, 1u, static_cast<uint32_t>(KT), 1u};
        // a head's row of codes is 128 bytes: wider fetches would bring the next head's too
        const CUtensorMapL2promotion promotion = fp8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
        const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        if (encode_tiled(&tm_k, type, 4, const_cast<void*>(a.k_cache), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, promotion) != CUDA_SUCCESS ||
            encode_tiled(&tm_v, type, 4, const_cast<void*>(a.v_cache), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, promotion) != CUDA_SUCCESS)
            return PKV_ERR_INVALID_ARG;
    }
    const size_t ctas = static_cast<size_t>(max_ctas(a.num_kv_heads));
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    Params p{};
    p.part_o = reinterpret_cast<float4*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + align256(ctas * 2 * ROWS * D * 4));
    p.meta = reinterpret_cast<int4*>(ws + align256(ctas * 2 * ROWS * D * 4) + align256(ctas * 2 * ROWS * 8));
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.cu_nodes = a.cu_nodes;
    p.mask = reinterpret_cast<const unsigned long long*>(a.tree_mask);
    p.out = a.out;
    p.v_codes = static_cast<const uint8_t*>(a.v_cache);
    p.v_cache = static_cast<const uint16_t*>(a.v_cache);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.batch = a.batch;
    p.max_blocks = a.max_blocks;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.lg = lg;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.max_nodes = a.max_nodes;
    p.max_context = a.max_context;
    p.mask_words = a.mask_words;
    p.total_nodes = a.total_nodes;
    p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
    p.err = err;
    p.qtok = qtok;
    const int grid = static_cast<int>(grid_of(a.batch, a.max_nodes, a.max_context, a.num_kv_heads, qtok));
    if ((fp8 ? launch<true>(grid, stream, tm_q, tm_k, tm_v, p) : launch<false>(grid, stream, tm_q, tm_k, tm_v, p)) != cudaSuccess) return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = programmatic(dim3(grid, JOIN_SPLIT), JOIN_THREADS, 0, stream, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_join_kernel, static_cast<const float4*>(p.part_o), static_cast<const float2*>(p.part_ml),
                                             static_cast<const int4*>(p.meta), a.out, a.num_heads, a.num_kv_heads, lg);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
