// Sampling with temperature, top-k, top-p and min-p: the exponential race among the tokens that
// a row's filters keep.
//
// With z_v = (l_v - max l) / T and w_v = e^z_v, tokens ordered by logit (equal logits: lower
// column first), a row keeps
//   top-k   the first k;
//   top-p   of those, every token whose weights before it in the order sum to less than
//           p * (the weights of all of those) -- the shortest prefix that reaches p;
//   min-p   of those, the tokens with z_v >= ln(min_p);
// and the winner is argmax z_v - ln e_v, e_v = -ln u_v, with pkv_sample's noise.  Since
// -ln e_v lies in (-2.82, 16.64), a token more than 19.6 below the maximum cannot beat the
// maximum's own key: it counts in the sums but takes no part in the race.
//
// One cluster of CTAs takes a row, each an equal slice of it; pass 1 reads it from HBM, later
// sweeps mostly find it in L2 and skip a quad of logits at one comparison of its maximum.
// The work below pass 1 is bound by latency (cluster barriers, dependent shared-memory steps), so
// each kind of row takes the shortest way that is exact for it:
//
//   pass 1  every thread's maximum and, for top-p, its sum of weights relative to a maximum; one
//           exchange gives every CTA the row's first token (top_k = 1 ends here) and the sum Z.
//           Without top-k and min-p the pass races every token too, so the exchange has the winner.
//   top-k   (k at most the threads, and 1024.)  A thread keeps its two largest quads of logits and
//           the third's maximum.  The k-th largest of those quads' maxima bounds the k-th logit
//           from below: a 128-bin histogram of the maxima gives the bound, and what reaches the
//           bound (a little over k tokens) is collected from those, rarely by another look at a
//           thread's share, in the first CTA, which ends the row on that list: one warp if it is
//           short.
//   top-p   A token that wins a race among all that min-p allows is the filters' winner if it is one
//           of their tokens: if the weights before it in the order sum to less than p Z.  If it is
//           not, it and what comes after it are out, and the race's next token is the candidate, so
//           long as it is known: every warp brings its two best.  One sweep sums the weights before
//           the best CANDS tokens (one of them is in with probability 1 - (1 - p)^CANDS; a single
//           row, for which the wait counts, examines one).  If none is, the tokens before them are
//           collected in the first CTA, which ends the row, or raced again, if they are more than
//           fit.  Where that fails TRIES times, the border itself is looked for:
//   border  A token lighter than (1 - p) Z / vocab is outside (all of those together weigh less
//           than 1 - p of Z).  Each warp lists its quads that hold others, and those are counted
//           into 2048 bins of 1/64 octave of weight.  A bin's weights lie within 1.1% of one
//           another, so the counts bound the running sum from both sides and leave a few bins where
//           it may reach p Z (if they hold too many, they are counted once more, into 2048 bins of
//           their own).  The tokens above those bins are summed and raced, the bins' members
//           collected in the first CTA, which sorts them, finds the border by their running sum and
//           races what is above it.
//   else    (a larger k, or more members than fit: a flat row, thousands of equal logits.)  The
//           same histogram over every token, and the range of candidates halved, by (logit bits,
//           column), until it fits; the race then sweeps the slices once more.
//
// Counts are integers, the weights of every thread are summed in a fixed tree (Z) or in 64-bit fixed
// point (2^-38), so neither atomics nor the order of the list can change a result.  A thread's share
// of a sum (19, 74 or 148 weights of a row of 151,936, in clusters of 16 x 512, 8 x 256 and 4 x 256
// threads) is fp32: a running sum is within about 1e-6 of itself at up to 200,000 logits, and the token at the border is decided as in exact arithmetic except when a border lies
// that near to it.
//
// Rows that cannot all run at once are taken in an order that starts the longest first (row_in_order).
//
// Measured on rows of 151,936 logits: 256 rows with settings of their own 87 us (156 MB, 1.8 TB/s; the average
// of sixteen seeds, 103 at most), all top-k = 50 62 us, all top-p = 0.9 127 us, no filter 82 us; one row 14,
// 16 and 14 us (top-p 18 us when its code has to come from DRAM).  The same batch of 256 before: with the border
// looked for in every top-p row and lists sorted 111 us; with one candidate examined 105 us on average and 179 at
// most; with rows in their own order 94.  What else was tried: the slices kept in shared memory (435 us), one loop
// for every sweep instead of a batched and a last one, five CTAs to an SM, a repeated race by only those warps
// whose best tokens are out, the last rows on larger clusters beside the others (all slower).
//
// The race's keys are fp32 with an error below 2e-5; when the two best are within 1e-4 they are
// ranked again in fp64.
#include <cooperative_groups.h>

#include <type_traits>
#include <utility>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_noise.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int BINS = 2048;
constexpr int TAIL = BINS - 1;               // the last bin: everything from 2047/64 octaves down
constexpr int COARSE = 128;                  // bins of the threads' maxima, 16 fine bins each
constexpr int CAP = 2048;                    // members collected at once
constexpr int BORDER = 512;                  // of those, around top-p's border
constexpr int LISTED = 10240;                // quads of a CTA's warps' lists
constexpr int WARP_LIST = 128;               // members that one warp ends a row with
constexpr int RANK_MAX = 256;                // members sorted by counting
constexpr int LOADS = 4;                     // 16-byte loads in flight per thread of a sweep (pass 1, from HBM: LOADS1)
constexpr int RACE_LOADS = 2;                // and of a race over all tokens
constexpr int CHECK_LOADS = 8;               // and of the check of a race's winner
constexpr int MAX_CLUSTER = 16;
constexpr float BINS_PER_OCTAVE = 64.f;
constexpr float RACE_Z = 19.6f;              // reach of the race (see above): 28.3 octaves, inside the fine bins
constexpr int CANDS = 3;                     // best tokens of a race that are examined, at most (TRIED)
constexpr float REF_REACH = 32.f;            // how far a race's reference may lie below a logit, in units of T
constexpr int TRIES = 6;                     // winners of top-p races examined before the border is looked for
constexpr float NEAR = 1e-4f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float FIX = 274877906944.f;        // 2^38: a weight of 1 in fixed point

struct Shared {
    uint32_t hist[BINS];         // this CTA's counts; top-k: every CTA's coarse counts
    uint32_t tot[BINS];          // the cluster's counts
    union {
        uint64_t list[CAP];      // first CTA: members, as composites
        uint16_t quads[LISTED];  // top-p and races: each warp's quads, from the slice's first
    };
    union {
        uint64_t border[BORDER];                     // first CTA, top-p: members
        uint64_t parts[MAX_CLUSTER * 8][2];          // races: the two best of every part
    };
    uint64_t sorted[RANK_MAX];
    uint64_t slot[2][MAX_CLUSTER];             // cluster-wide sums, alternating
    uint64_t lo[2][MAX_CLUSTER], hi[2][MAX_CLUSTER];   // cluster-wide ranges, alternating
    uint64_t top[MAX_CLUSTER];   // pass 1: first token of each CTA, and its sum of weights relative to it
    float z[MAX_CLUSTER];
    float wz[32];                // per warp
    uint64_t win[MAX_CLUSTER][2];   // border: the two best of each CTA
    uint64_t lists[MAX_CLUSTER][CANDS + 1];
    int list_part[MAX_CLUSTER][CANDS + 1];
    uint64_t cand[CANDS + 1];       // the race's best, in the order of their keys, with their parts and logits
    int cand_part[CANDS + 1];
    float cand_x[CANDS];
    uint64_t cand_at[CANDS];        // their places in the row's order
    uint64_t wsum[32][CANDS];       // weights before each of them: per warp, per CTA
    uint64_t csum[MAX_CLUSTER][CANDS];
    uint32_t ccnt[MAX_CLUSTER];
    uint64_t threshold;
    uint64_t list_sum;
    uint64_t wred[32];           // per warp
    uint64_t wlo[32], whi[32];
    float2 wscan[32];
    uint64_t wwin[32][2];
    int first[3];
    uint32_t list_n;
};
static_assert(MAX_CLUSTER * COARSE <= BINS, "the coarse counts fit the histogram");
static_assert(sizeof(Shared) <= 48 * 1024, "no opt-in to more shared memory");

// Order of the tokens as an unsigned number: larger = earlier.  -0 and +0 are one logit.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t composite(float x, int col) {
    return (static_cast<uint64_t>(key_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ float composite_x(uint64_t c) { return value_of(static_cast<uint32_t>(c >> 32)); }
__device__ __forceinline__ int composite_col(uint64_t c) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(c)); }

// Depth below the maximum in bins; non-decreasing as the logit falls, inf for -inf.
__device__ __forceinline__ int bin_of(float depth) { return static_cast<int>(fminf(depth, static_cast<float>(TAIL))); }
__device__ __forceinline__ float weight_of(float depth) { return ex2_ftz(depth * (-1.f / BINS_PER_OCTAVE)); }
__device__ __forceinline__ uint64_t fixed_of(float w) { return __float2ull_rn(w * FIX); }

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int off) {
    return static_cast<uint64_t>(__shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(v), off));
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// The two best of a race, as composites of key and column (larger key first, then lower column); 0: none.
struct Best {
    uint64_t b1, b2;
    __device__ __forceinline__ void clear() { b1 = b2 = 0; }
    __device__ __forceinline__ void add(uint64_t c) {
        b2 = max(b2, min(b1, c));
        b1 = max(b1, c);
    }
    __device__ __forceinline__ void merge(uint64_t o1, uint64_t o2) {
        b2 = max(max(b2, o2), min(b1, o1));
        b1 = max(b1, o1);
    }
    // keys shifted by d
    __device__ __forceinline__ void rebase(float d) {
        if (b1) b1 = composite(composite_x(b1) + d, composite_col(b1));
        if (b2) b2 = composite(composite_x(b2) + d, composite_col(b2));
    }
    __device__ __forceinline__ float key() const { return b1 ? composite_x(b1) : -INFINITY; }
};

// The smallest fp32 number not below M + c in exact arithmetic (c <= 0): the sum rounded to nearest and, where the
// rounding took it down (its error is exact in fp32), the next one.  A limit on logits, compared as it would be on
// their differences from M: M + c rounded to nearest is off by half a step of M, 3e-5 for logits near 1000.
__device__ __forceinline__ float not_below(float M, float c) {
    const float s = __fadd_rn(M, c), b = __fsub_rn(s, M);
    const float low = __fadd_rn(__fsub_rn(M, __fsub_rn(s, b)), __fsub_rn(c, b));      // M + c - s
    return low > 0.f ? nextafterf(s, INFINITY) : s;
}

// Steps that several ways share are functions, not inlined: a row runs most of this kernel's code once, so its
// time is in good part that of fetching it.

// n members sorted, earliest first, by the CTA.
template <int THREADS>
__device__ __noinline__ void sort_members(Shared& sh, uint64_t* list, int n) {
    const int tid = threadIdx.x;
    if (n <= RANK_MAX) {
        for (int i = tid; i < n; i += THREADS) {
            const uint64_t c = list[i];
            int at = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) at += list[j] > c ? 1 : 0;
            sh.sorted[at] = c;
        }
        __syncthreads();
        for (int i = tid; i < n; i += THREADS) list[i] = sh.sorted[i];
        __syncthreads();
        return;
    }
    int n2 = RANK_MAX;
    while (n2 < n) n2 <<= 1;
    for (int i = n + tid; i < n2; i += THREADS) list[i] = 0ull;
    __syncthreads();
    for (int size = 2; size <= n2; size <<= 1)
        for (int half = size >> 1; half >= 1; half >>= 1) {
            for (int i = tid; i < (n2 >> 1); i += THREADS) {
                const int x = (i & ~(half - 1)) * 2 + (i & (half - 1)), y = x + half;
                const uint64_t cx = list[x], cy = list[y];
                if ((x & size) == 0 ? cx < cy : cx > cy) {
                    list[x] = cy;
                    list[y] = cx;
                }
            }
            __syncthreads();
        }
}

// How many of the first n members of a sorted list have less than `goal` weight before them, `above` in
// front, and their weight (without `above`).  By every thread of the CTA.
struct Kept {
    uint64_t sum;
    int count;
};
template <int THREADS>
__device__ __noinline__ Kept kept_members(Shared& sh, const uint64_t* list, int n, uint64_t above, uint64_t goal, float M,
                                          float per_logit) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (n + THREADS - 1) / THREADS, i0 = tid * each, i1 = min(n, i0 + each);
    auto weight = [&](int i) { return fixed_of(weight_of((M - composite_x(list[i])) * per_logit)); };
    uint64_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += weight(i);
    uint64_t s = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t x = static_cast<uint64_t>(__shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(s), off));
        if (lane >= off) s += x;
    }
    __syncthreads();
    if (lane == 31) sh.wred[warp] = s;
    __syncthreads();
    uint64_t before = above + s - mine;
    for (int w = 0; w < warp; ++w) before += sh.wred[w];
    Kept r{0, 0};
    for (int i = i0; i < i1; ++i) {
        const uint64_t w = weight(i);
        if (before < goal) {
            ++r.count;
            r.sum += w;
        }
        before += w;
    }
    r.count = __reduce_add_sync(0xffffffffu, r.count);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) r.sum += shfl_xor64(r.sum, off);
    __syncthreads();
    if (lane == 0) { sh.wred[warp] = r.sum; sh.wlo[warp] = static_cast<uint64_t>(r.count); }
    __syncthreads();
    r = Kept{0, 0};
    for (int w = 0; w < WARPS; ++w) { r.count += static_cast<int>(sh.wlo[w]); r.sum += sh.wred[w]; }
    __syncthreads();
    return r;
}

__device__ __noinline__ uint4 noise_quad(uint32_t quad, PhiloxRow row) {
    const RoundKeys unused = {};
    return philox_row_at<false>(quad, row, unused);
}

__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

// The key of a token whose logit exceeds the reference's by d, relative to a key of 0 there.
__device__ __forceinline__ float key_of_token(float d, float inv_t, uint32_t noise) {
    // e = -ln u from the exact w = 1 - u where u is near 1, from the hardware logarithm elsewhere
    const float w = one_minus_u_of(noise);
    const float e = w < 0.015625f ? w * fmaf(w, fmaf(w, fmaf(w, 0.25f, 0.333333343f), 0.5f), 1.0f)
                                  : -__logf(__uint2float_rn(2u * (noise >> 9) + 1u) * 5.9604644775390625e-08f);
    return d * inv_t - __logf(e);
}

// The tokens of a quad that are above -inf, raced, with keys relative to `base`.  A token can beat the warp's
// best `bar` only if 1 - u < e^(z - bar) (since -ln u >= 1 - u), which spares most keys: the quad's smallest
// 1 - u against the bound of its largest logit, then each token's; the bound carries a margin of 1e-3.  False:
// nothing was added.
__device__ __forceinline__ bool race_quad(Best& best, int qd, const float (&l)[4], float lmax, float base, float bar, float inv_t,
                                          float l2, const uint4& w) {
    const float cb = (1e-3f - bar) * LOG2E + 1.4419741739064e-3f;                      // + log2 1.001
    const uint32_t wmax = max(max(w.x, w.y), max(w.z, w.w));
    const bool any = one_minus_u_of(wmax) < ex2_ftz(fmaf(lmax - base, l2, cb));
    if (any) {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (one_minus_u_of(ws[e]) < ex2_ftz(fmaf(l[e] - base, l2, cb)))
                best.add(composite(key_of_token(l[e] - base, inv_t, ws[e]), 4 * qd + e));
    }
    return any;
}

// A key that at least two tokens of the warp reach: what is pruned against it is not among the warp's two best.
__device__ __forceinline__ float warp_second(const Best& best) {
    const float k1 = best.key(), m = warp_max(k1);
    return warp_max(k1 == m ? (best.b2 ? composite_x(best.b2) : -INFINITY) : k1);
}

// Whole quads are one aligned 16-byte load; absent columns and NaN read as -inf.
__device__ __forceinline__ float4 clean(const float4& v) {
    return make_float4(fmaxf(v.x, -INFINITY), fmaxf(v.y, -INFINITY), fmaxf(v.z, -INFINITY), fmaxf(v.w, -INFINITY));
}
// kOnce: the row is not swept again, so its lines may leave L2 first (152 rows at once are 92 MB: without it, later
// looks at the other rows missed L2; 256 rows with settings of their own 91 -> 87 us).
template <bool kOnce = false>
__device__ __forceinline__ float4 load_whole_quad(const float* row, int qd) {
    const float4* at = reinterpret_cast<const float4*>(row) + qd;
    return clean(kOnce ? __ldcs(at) : __ldg(at));
}
__device__ __forceinline__ float4 load_columns(const float* row, int qd, int vocab) {
    const int col = qd * 4;
    float4 v;
    v.x = __ldg(row + col);
    v.y = col + 1 < vocab ? __ldg(row + col + 1) : -INFINITY;
    v.z = col + 2 < vocab ? __ldg(row + col + 2) : -INFINITY;
    v.w = col + 3 < vocab ? __ldg(row + col + 3) : -INFINITY;
    return clean(v);
}
__device__ __forceinline__ float max_of(const float4& v) { return fmaxf(fmax3(v.x, v.y, v.z), v.w); }

// f(quad, its logits) over quads [q0, q1) of a row by whole warps, N loads in flight; lanes without a quad get -inf.
template <int THREADS, int N, bool kOnce = false, typename F>
__device__ __forceinline__ void sweep_warps(const float* row, int q0, int q1, int whole, int vocab, F f) {
    const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    const int tid = threadIdx.x;
    int base = q0;
    for (; base + N * THREADS <= min(q1, whole); base += N * THREADS) {
        float4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = load_whole_quad<kOnce>(row, base + i * THREADS + tid);
#pragma unroll
        for (int i = 0; i < N; ++i) f(base + i * THREADS + tid, v[i]);
    }
    for (; base < q1; base += N * THREADS) {
        float4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int qd = base + i * THREADS + tid;
            v[i] = whole > 0 ? load_whole_quad<kOnce>(row, min(qd, whole - 1)) : none;
            if (qd >= q1) v[i] = none;
            else if (qd >= whole) v[i] = load_columns(row, qd, vocab);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (base + i * THREADS < q1) f(base + i * THREADS + tid, v[i]);
    }
}

// A race among all tokens of a slice, read once, with its maximum and (kSum) the sum of its weights.  Sums and
// keys are relative to a reference the warp shares, which moves when a logit exceeds it by REF_REACH.
struct RaceAll {
    Best best;
    float mx, zs, ref;
    int mx_quad;
};
template <bool kSum, bool kTwo, int THREADS>
__device__ __noinline__ RaceAll race_all_of(const float* row, int q0, int q1, int whole, int vocab, float T, float inv_t,
                                            PhiloxRow prow) {
    RaceAll r;
    r.best.clear();
    r.mx = r.ref = -INFINITY;
    r.zs = 0.f;
    r.mx_quad = q0;
    const float l2 = fminf(inv_t * LOG2E, 3.4028235e38f);
    const RoundKeys unused = {};
    float ref_end = -INFINITY, bar = -INFINITY;
    sweep_warps<THREADS, RACE_LOADS, !kSum>(row, q0, q1, whole, vocab, [&](int qd, const float4& v) {
        const float m4 = max_of(v);
        if (m4 > r.mx) { r.mx = m4; r.mx_quad = qd; }
        if (__any_sync(0xffffffffu, m4 > ref_end)) {
            const float up = warp_max(m4), d = r.ref - up;
            if (r.ref > -INFINITY) {
                r.zs *= ex2_ftz(d * l2);
                r.best.rebase(d * inv_t);
                bar += d * inv_t;
            }
            r.ref = up;
            ref_end = up + REF_REACH * T;
        }
        if (r.ref > -INFINITY) {
            if (kSum)
                r.zs += (ex2_ftz((v.x - r.ref) * l2) + ex2_ftz((v.y - r.ref) * l2)) +
                        (ex2_ftz((v.z - r.ref) * l2) + ex2_ftz((v.w - r.ref) * l2));
            const float l[4] = {v.x, v.y, v.z, v.w};
            const uint4 w = philox_row_at<false>(static_cast<uint32_t>(qd), prow, unused);
            const bool any = race_quad(r.best, qd, l, m4, r.ref, bar, inv_t, l2, w);
            if (!kTwo) bar = warp_max(r.best.key());
            else if (__any_sync(0xffffffffu, any)) bar = warp_second(r.best);
        }
    });
    return r;
}

// A quad's weights added to the sums of those that come before each candidate, and its tokens before `top_c` counted.
struct Before {
    float w[CANDS];
    uint32_t count;
};
__device__ __noinline__ Before add_before(Before s, const Shared& sh, float4 v, int qd, float M, float per_logit, uint64_t top_c) {
    const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t c = composite(l[e], 4 * qd + e);
        const float w = weight_of((M - l[e]) * per_logit);
#pragma unroll
        for (int j = 0; j < CANDS; ++j)
            if (c > sh.cand_at[j]) s.w[j] += w;
        if (c > top_c) ++s.count;
    }
    return s;
}

__device__ __forceinline__ uint32_t noise_of(int col, const PhiloxRow& prow) {
    const uint4 w = noise_quad(static_cast<uint32_t>(col) >> 2, prow);
    const int e = col & 3;
    return e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
}

// The column that wins among the two best: their fp64 keys decide where fp32 ones are too near.
__device__ __noinline__ int winner_of(Best best, const float* row, float M, float T, PhiloxRow prow) {
    int c1 = best.b1 ? composite_col(best.b1) : -1;       // (a row that changes under the call may have none)
    if (best.b2 && composite_x(best.b1) - composite_x(best.b2) <= NEAR) {
        const int c2 = composite_col(best.b2);
        double d[2];
        for (int i = 0; i < 2; ++i) {
            const int col = i ? c2 : c1;
            const double e = -log1p(-static_cast<double>(one_minus_u_of(noise_of(col, prow))));
            d[i] = (static_cast<double>(__ldg(row + col)) - static_cast<double>(M)) / static_cast<double>(T) - log(e);
        }
        if (d[1] > d[0] || (d[1] == d[0] && c2 < c1)) c1 = c2;
    }
    return c1;
}

// top_p of a fixed-point sum (p < 1), at least 1.
__device__ __forceinline__ uint64_t goal_of_sum(uint64_t z, float p) {
    return max(__umul64hi(z, __float2ull_rz(p * 9223372036854775808.f)) << 1, static_cast<unsigned long long>(1));
}

// The winner among the n members of the list, which begins the row's order: their first `count`, and (by_weight)
// of those the ones before which the weights sum to less than the goal (goal 0: p of the `count` ones' sum).
// By GROUP threads, a warp or the whole CTA; each holds its share of up to CAPACITY members in registers.  The
// members are not sorted: the count-th is selected, and a race's winner stands if the weights before it are less
// than the goal; if they are not, neither it nor what comes after it is a member, and the rest is raced again.
template <int GROUP, int CAPACITY>
__device__ __noinline__ int list_winner(Shared& sh, const float* row, int n, int count, bool by_weight, uint64_t goal, float p, float M,
                                        float T, float inv_t, float per_logit, float min_x, PhiloxRow prow) {
    constexpr int WARPS = GROUP / 32, PER = CAPACITY / GROUP, DIGITS = 256;
    auto sync = [] { if (WARPS == 1) __syncwarp(); else __syncthreads(); };
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t c[PER], keep = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = tid + i * GROUP < n ? sh.list[tid + i * GROUP] : 0;      // no member's is 0
    if (count < n) {
        // the need-th, from the top, of `in` members that are compared with one another
        const uint64_t* among = sh.list;
        int need = count, in = n;
        if (CAPACITY > RANK_MAX && n > RANK_MAX) {
            uint64_t lo = ~0ull, hi = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (c[i]) { lo = min(lo, c[i]); hi = max(hi, c[i]); }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                lo = min(lo, shfl_xor64(lo, off));
                hi = max(hi, shfl_xor64(hi, off));
            }
            sync();
            if (lane == 0) { sh.wlo[warp] = lo; sh.whi[warp] = hi; }
            sync();
            for (int w = 0; w < WARPS; ++w) { lo = min(lo, sh.wlo[w]); hi = max(hi, sh.whi[w]); }
            // [lo, hi] holds it; 256 equal parts at a time
            while (in > RANK_MAX) {
                const int shift = max(0, 56 - __clzll(static_cast<long long>(hi - lo)));
                if (tid < DIGITS) sh.hist[tid] = 0u;
                sync();
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (c[i] >= lo && c[i] <= hi) atomicAdd(&sh.hist[(c[i] - lo) >> shift], 1u);
                sync();
                const int digit = DIGITS - 1 - tid, mine = tid < DIGITS ? static_cast<int>(sh.hist[digit]) : 0;
                int upto = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, upto, off);
                    if (lane >= off) upto += x;
                }
                if (lane == 31) sh.wlo[warp] = static_cast<uint64_t>(upto);
                sync();
                for (int w = 0; w < warp; ++w) upto += static_cast<int>(sh.wlo[w]);
                if (upto - mine < need && upto >= need) { sh.first[0] = digit; sh.first[1] = need - (upto - mine); sh.first[2] = mine; }
                sync();
                lo += static_cast<uint64_t>(sh.first[0]) << shift;
                hi = min(hi, lo + ((static_cast<uint64_t>(1) << shift) - 1));
                need = sh.first[1];
                in = sh.first[2];
                sync();
            }
            if (tid == 0) sh.first[0] = 0;
            sync();
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (c[i] >= lo && c[i] <= hi) {
                    const int at = atomicAdd(&sh.first[0], 1);
                    if (at < RANK_MAX) sh.sorted[at] = c[i];
                }
            sync();
            among = sh.sorted;
        }
        for (int i = tid; i < in; i += GROUP) {
            const uint64_t x = among[i];
            int before = 0;
#pragma unroll 4
            for (int j = 0; j < in; ++j) before += among[j] > x ? 1 : 0;
            if (before == need - 1) sh.threshold = x;
        }
        sync();
        keep = sh.threshold;
    }
    auto block_sum = [&](uint64_t v) -> uint64_t {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) v += shfl_xor64(v, off);
        sync();
        if (lane == 0) sh.wred[warp] = v;
        sync();
        v = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += sh.wred[w];
        return v;
    };
    auto weight = [&](uint64_t m) { return fixed_of(weight_of((M - composite_x(m)) * per_logit)); };
    auto weights_from = [&](uint64_t first) {              // of the members from `first` up
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (c[i] && c[i] >= first) s += weight(c[i]);
        return block_sum(s);
    };
    float key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (c[i] < keep || !(composite_x(c[i]) >= min_x)) key[i] = -INFINITY;      // (an absent member's x is NaN)
        else key[i] = key_of_token(composite_x(c[i]) - M, inv_t, noise_of(composite_col(c[i]), prow));
    }
    if (by_weight && goal == 0) goal = goal_of_sum(weights_from(keep), p);
    for (;;) {
        Best best;
        best.clear();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (c[i] >= keep && key[i] > -INFINITY) best.add(composite(key[i], composite_col(c[i])));
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) best.merge(shfl_xor64(best.b1, off), shfl_xor64(best.b2, off));
        if (lane == 0) { sh.wwin[warp][0] = best.b1; sh.wwin[warp][1] = best.b2; }
        sync();
        best.clear();
        if (lane < WARPS) best.merge(sh.wwin[lane][0], sh.wwin[lane][1]);
#pragma unroll
        for (int off = WARPS / 2; off >= 1; off >>= 1) best.merge(shfl_xor64(best.b1, off), shfl_xor64(best.b2, off));
        best.b1 = static_cast<uint64_t>(__shfl_sync(0xffffffffu, static_cast<unsigned long long>(best.b1), 0));
        best.b2 = static_cast<uint64_t>(__shfl_sync(0xffffffffu, static_cast<unsigned long long>(best.b2), 0));
        const int col = winner_of(best, row, M, T, prow);
        if (!by_weight || col < 0) return col;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (c[i] && composite_col(c[i]) == col) sh.threshold = c[i];
        sync();
        keep = sh.threshold + 1;
        if (weights_from(keep) < goal) return col;
    }
}

struct Args {
    SampleFilteredArgs a;
    int vec_ok;
    int ordered;             // rows that take long first
    int* err;
};

// The row that the i-th cluster takes where rows do not all run at once: those that take long first, so that the
// batch does not end with one of them: without top-k and with top-p, without both, with a large k, a small one, 1.
constexpr int ORDERED_ROWS = 4095;           // counted in 12 bits each
template <int THREADS>
__device__ __noinline__ int row_in_order(Shared& sh, const SampleFilteredArgs& a, int i) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto field = [&](int b) {
        const int k = a.top_k ? __ldg(a.top_k + b) : 0;
        const float p = a.top_p ? __ldg(a.top_p + b) : 1.f;
        if (k <= 0 || k >= a.vocab) return p < 1.f ? 0 : 12;
        return k > WARP_LIST ? 24 : k > 1 ? 36 : 48;
    };
    const int per = (a.batch + THREADS - 1) / THREADS, b0 = tid * per, b1 = min(a.batch, b0 + per);
    uint64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += static_cast<uint64_t>(1) << field(b);
    uint64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t x = static_cast<uint64_t>(__shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(upto), off));
        if (lane >= off) upto += x;
    }
    if (lane == 31) sh.wred[warp] = upto;
    __syncthreads();
    uint64_t all = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) upto += sh.wred[w];
        all += sh.wred[w];
    }
    int f = 0;
    for (; f < 48 && i >= static_cast<int>((all >> f) & 4095u); f += 12) i -= static_cast<int>((all >> f) & 4095u);
    i -= static_cast<int>(((upto - mine) >> f) & 4095u);
    if (i >= 0 && i < static_cast<int>((mine >> f) & 4095u))
        for (int b = b0; b < b1; ++b)
            if (field(b) == f && i-- == 0) sh.first[2] = b;
    __syncthreads();
    return sh.first[2];
}

template <int CLUSTER, int THREADS, int LOADS1, int MIN_CTAS, int TRIED>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS, MIN_CTAS) sample_filtered_kernel(const Args args) {
    constexpr int WARPS = THREADS / 32;
    constexpr int BINS_PER_THREAD = BINS / THREADS;
    constexpr int BINS_PER_RANK = BINS / CLUSTER;
    constexpr int FAST_K = CLUSTER * THREADS < CAP / 2 ? CLUSTER * THREADS : CAP / 2;
    static_assert(BINS % THREADS == 0 && CLUSTER <= MAX_CLUSTER && CLUSTER <= WARPS && WARPS <= 32 && TRIED <= CANDS &&
                      CLUSTER * (TRIED > 1 ? WARPS : 1) <= MAX_CLUSTER * 8 && COARSE <= THREADS, "tables fit");
    const SampleFilteredArgs& a = args.a;
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = args.ordered ? row_in_order<THREADS>(sh, a, blockIdx.y) : static_cast<int>(blockIdx.y);

    const float T = __ldg(a.temperatures + row);
    const int k = a.top_k ? __ldg(a.top_k + row) : 0;
    const float p = a.top_p ? __ldg(a.top_p + row) : 1.f;
    const float mp = a.min_p ? __ldg(a.min_p + row) : 0.f;
    const bool t_ok = T > 0.f && T < INFINITY;
    const bool f_ok = p > 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f;
    if (!t_ok || !f_ok) {
        if (rank == 0 && tid == 0) {
            record_error(args.err, t_ok ? PKV_DEVERR_FILTER : PKV_DEVERR_TEMPERATURE, row);
            a.out_ids[row] = -1;
        }
        return;
    }
    auto started = cluster.barrier_arrive();              // waited for before the first access to another CTA
    const bool need_k = k > 0 && k < a.vocab;
    const bool need_p = p < 1.f;
    const bool fast_k = need_k && k <= FAST_K;
    const float inv_t = fminf(1.0f / T, 3.4028235e38f);
    const float l2 = fminf(inv_t * LOG2E, 3.4028235e38f);
    const float per_logit = fminf(inv_t * (LOG2E * BINS_PER_OCTAVE), 3.4028235e38f);    // bins per unit of logit

    // ---- this CTA's slice: whole quads [q0, q1) of the row; absent columns and NaN read as -inf
    const float* lrow = a.logits + static_cast<int64_t>(row) * a.row_stride;
    const int nquads = (a.vocab + 3) >> 2;
    const int per = (nquads + CLUSTER - 1) / CLUSTER;
    const int q0 = min(nquads, rank * per), q1 = min(nquads, q0 + per);
    const int whole = args.vec_ok ? a.vocab >> 2 : 0;     // quads below it are whole
    const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    auto load_whole = [&](int qd) -> float4 { return load_whole_quad(lrow, qd); };
    auto load_quad = [&](int qd) -> float4 { return qd < whole ? load_whole(qd) : load_columns(lrow, qd, a.vocab); };
    // f(quad, its logits) over the slice, LOADS loads in flight per thread
    auto sweep_quads_by = [&](auto in_flight, auto f, auto once) {
        constexpr int N = decltype(in_flight)::value;
        constexpr bool kOnce = decltype(once)::value;
        int qd = q0 + tid;
        const int end = min(q1, whole);
        for (; qd + (N - 1) * THREADS < end; qd += N * THREADS) {
            float4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = load_whole_quad<kOnce>(lrow, qd + i * THREADS);
#pragma unroll
            for (int i = 0; i < N; ++i) f(qd + i * THREADS, v[i]);
        }
        if (qd < end) {                                   // the rest of the whole quads, together as well
            float4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = load_whole_quad<kOnce>(lrow, min(qd + i * THREADS, end - 1));
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (qd + i * THREADS < end) f(qd + i * THREADS, v[i]);
            qd += ((end - qd + THREADS - 1) / THREADS) * THREADS;
        }
        for (; qd < q1; qd += THREADS) f(qd, load_quad(qd));
    };
    auto sweep_quads = [&](auto f) { sweep_quads_by(std::integral_constant<int, LOADS>{}, f, std::false_type{}); };
    const int iters = (q1 - q0 + THREADS - 1) / THREADS;  // uniform
    // f(column, logit) for every logit of the slice from x_min up, and above -inf
    auto sweep_from = [&](float x_min, auto f) {
        sweep_quads([&](int qd, const float4& v) {
            const float m = max_of(v);
            if (!(m >= x_min && m > -INFINITY)) return;
            const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (l[e] >= x_min && l[e] > -INFINITY) f(4 * qd + e, l[e]);
        });
    };

    // ---- noise and keys
    uint64_t seed = a.seed, offset = a.offset;
    if (a.seed_offset) {
        seed = __ldg(a.seed_offset);
        offset = __ldg(a.seed_offset + 1);
    }
    const uint64_t rr = static_cast<uint64_t>(row) + offset;
    const PhiloxRow prow = philox_row(static_cast<uint32_t>(rr), static_cast<uint32_t>(rr >> 32), static_cast<uint32_t>(seed),
                                      static_cast<uint32_t>(seed >> 32));
    Best best;
    best.clear();
    auto warp_best = [&]() {                              // of the warp's lanes, in each of them
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) best.merge(shfl_xor64(best.b1, off), shfl_xor64(best.b2, off));
    };
    // the CTA's two best, in the lanes of its first warp
    auto block_best = [&]() {
        warp_best();
        if (lane == 0) { sh.wwin[warp][0] = best.b1; sh.wwin[warp][1] = best.b2; }
        __syncthreads();
        if (warp == 0) {
            best.clear();
            if (lane < WARPS) best.merge(sh.wwin[lane][0], sh.wwin[lane][1]);
#pragma unroll
            for (int off = WARPS / 2; off >= 1; off >>= 1) best.merge(shfl_xor64(best.b1, off), shfl_xor64(best.b2, off));
        }
    };
    auto put_best = [&](int to) {                         // by a lane of the first warp, after block_best
        uint64_t* w = cluster.map_shared_rank(&sh.win[rank][0], to);
        w[0] = best.b1;
        w[1] = best.b2;
    };
    // what the race's best are taken from, to every CTA
    constexpr int PUT = TRIED > 1 ? WARPS : 1;            // parts of a CTA whose two best are known
    auto gather_best = [&]() {
        if (PUT == 1) block_best();
        else warp_best();
        if (PUT == 1 ? tid < CLUSTER : lane < CLUSTER) {
            uint64_t* w = cluster.map_shared_rank(&sh.parts[rank * PUT + (PUT == 1 ? 0 : warp)][0], lane);
            w[0] = best.b1;
            w[1] = best.b2;
        }
    };

    // ---- pass 1
    for (int b = tid; b < BINS; b += THREADS) sh.hist[b] = 0u;
    if (tid < COARSE) sh.tot[tid] = 0u;                   // the coarse counts, first
    if (tid == 0) sh.list_n = 0u;
    float mx = -INFINITY, zs = 0.f;
    int mx_quad = q0;                                     // the first quad that holds this thread's maximum
    float m2 = -INFINITY, m3 = -INFINITY;                 // top-k: the second and third largest quads' maxima
    int m2_quad = q0;
    const bool online = need_p && !fast_k;
    const bool race_all = !need_k && mp == 0.f;           // every token is raced as it is read
    float ref = -INFINITY;                                // race_all: what the warp's sums and keys are relative to
    if (race_all) {
        const RaceAll r = online ? race_all_of<true, (TRIED > 1), THREADS>(lrow, q0, q1, whole, a.vocab, T, inv_t, prow)
                                 : race_all_of<false, false, THREADS>(lrow, q0, q1, whole, a.vocab, T, inv_t, prow);
        mx = r.mx;
        mx_quad = r.mx_quad;
        zs = r.zs;
        ref = r.ref;
        best = r.best;
    } else if (online) {
        sweep_quads_by(std::integral_constant<int, LOADS1>{}, [&](int qd, const float4& v) {
            const float m4 = max_of(v);
            if (m4 > mx) {
                zs *= ex2_ftz((mx - m4) * l2);            // 0 for the first
                mx = m4;
                mx_quad = qd;
            }
            if (mx > -INFINITY)
                zs += (ex2_ftz((v.x - mx) * l2) + ex2_ftz((v.y - mx) * l2)) + (ex2_ftz((v.z - mx) * l2) + ex2_ftz((v.w - mx) * l2));
        }, std::false_type{});
    } else if (fast_k) {
        sweep_quads_by(std::integral_constant<int, LOADS1>{}, [&](int qd, const float4& v) {
            const float m4 = max_of(v);
            const bool a1 = m4 > mx, a2 = m4 > m2;
            m3 = a2 ? m2 : fmaxf(m3, m4);
            m2_quad = a1 ? mx_quad : a2 ? qd : m2_quad;
            m2 = a1 ? mx : a2 ? m4 : m2;
            mx_quad = a1 ? qd : mx_quad;
            mx = a1 ? m4 : mx;
        }, std::true_type{});
    } else {
        sweep_quads_by(std::integral_constant<int, LOADS1>{}, [&](int qd, const float4& v) {
            const float m4 = max_of(v);
            if (m4 > mx) { mx = m4; mx_quad = qd; }
        }, std::false_type{});
    }
    uint64_t top = 0;                                     // the first token: largest logit, lowest column
    if (mx > -INFINITY) {
        const float4 v = load_quad(mx_quad);
        const int e = v.x == mx ? 0 : v.y == mx ? 1 : v.z == mx ? 2 : 3;
        top = composite(mx, 4 * mx_quad + e);
    }
    {
        uint64_t t = top;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) t = max(t, shfl_xor64(t, off));
        if (lane == 0) sh.whi[warp] = t;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) t = max(t, sh.whi[w]);
        float z = 0.f;
        if (online) {
            // fixed trees of fp32 sums; infinite maxima end the row below, whatever their sum
            const float m_cta = t ? composite_x(t) : 0.f, m_own = race_all ? ref : mx;
            z = m_own > -INFINITY && m_cta < INFINITY ? zs * ex2_ftz((m_own - m_cta) * l2) : 0.f;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
            if (lane == 0) sh.wz[warp] = z;
            __syncthreads();
            z = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) z += sh.wz[w];
        }
        if (race_all) best.rebase((ref - composite_x(t)) * inv_t);
        cluster.barrier_wait(std::move(started));
        if (race_all) gather_best();
        if (tid < CLUSTER) {
            *cluster.map_shared_rank(&sh.top[rank], tid) = t;
            *cluster.map_shared_rank(&sh.z[rank], tid) = z;
        }
    }
    cluster.sync();                                       // also publishes the cleared tables
    uint64_t first_token = 0, Z = 0;
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) first_token = max(first_token, sh.top[r]);
    const float M = composite_x(first_token);
    if (first_token == 0 || k == 1 || M == INFINITY) {    // nothing above -inf; or no choice: infinite logits win
        if (rank == 0 && tid == 0) a.out_ids[row] = first_token == 0 ? -1 : static_cast<int64_t>(composite_col(first_token));
        return;
    }
    if (online) {
        float z = 0.f;
#pragma unroll
        for (int r = 0; r < CLUSTER; ++r)
            if (sh.top[r]) z = fmaf(sh.z[r], ex2_ftz((composite_x(sh.top[r]) - M) * l2), z);
        Z = fixed_of(z);
    }
    // the smallest logit in the race: min-p's limit, and the race's reach
    const float min_x = fmaxf(mp > 0.f ? not_below(M, T * logf(mp)) : -INFINITY, M - RACE_Z * T);
    auto depth = [&](float x) { return (M - x) * per_logit; };
    // a logit not above any whose bin is <= b: M minus b + 1 bins and a margin for its own rounding
    auto x_at_end_of = [&](int b) {
        const float x = M - static_cast<float>(b + 1) / per_logit;
        return x - (fabsf(M) + fabsf(x)) * 1e-6f;
    };

    // ---- cluster-wide reductions; every CTA ends with the same values
    int phase = 0;
    auto cluster_sum = [&](uint64_t v) -> uint64_t {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) v += shfl_xor64(v, off);
        if (lane == 0) sh.wred[warp] = v;
        __syncthreads();
        if (tid < CLUSTER) {
            uint64_t s = 0;
            for (int w = 0; w < WARPS; ++w) s += sh.wred[w];
            *cluster.map_shared_rank(&sh.slot[phase][rank], tid) = s;
        }
        cluster.sync();
        uint64_t s = 0;
#pragma unroll
        for (int r = 0; r < CLUSTER; ++r) s += sh.slot[phase][r];
        phase ^= 1;
        return s;
    };
    int rphase = 0;
    auto cluster_range = [&](uint64_t& lo, uint64_t& hi) {   // the smallest and the largest
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            lo = min(lo, shfl_xor64(lo, off));
            hi = max(hi, shfl_xor64(hi, off));
        }
        if (lane == 0) { sh.wlo[warp] = lo; sh.whi[warp] = hi; }
        __syncthreads();
        if (tid < CLUSTER) {
            for (int w = 0; w < WARPS; ++w) { lo = min(lo, sh.wlo[w]); hi = max(hi, sh.whi[w]); }
            *cluster.map_shared_rank(&sh.lo[rphase][rank], tid) = lo;
            *cluster.map_shared_rank(&sh.hi[rphase][rank], tid) = hi;
        }
        cluster.sync();
        lo = sh.lo[rphase][0];
        hi = sh.hi[rphase][0];
        for (int r = 1; r < CLUSTER; ++r) { lo = min(lo, sh.lo[rphase][r]); hi = max(hi, sh.hi[rphase][r]); }
        rphase ^= 1;
    };
    // the cluster's counts from every CTA's (complete before the call's first barrier)
    auto cluster_hist = [&]() {
        cluster.sync();
        for (int i = tid; i < BINS_PER_RANK; i += THREADS) {
            const int b = rank * BINS_PER_RANK + i;
            uint32_t s = 0;
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) s += *cluster.map_shared_rank(&sh.hist[b], r);
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) *cluster.map_shared_rank(&sh.tot[b], r) = s;
        }
        cluster.sync();
    };
    // exclusive prefix over the CTA's threads of two fp32 numbers
    auto scan2 = [&](float2 v) -> float2 {
        float2 s = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, s.x, off), y = __shfl_up_sync(0xffffffffu, s.y, off);
            if (lane >= off) { s.x += x; s.y += y; }
        }
        __syncthreads();
        if (lane == 31) sh.wscan[warp] = s;
        __syncthreads();
        float2 before = make_float2(0.f, 0.f);
        for (int w = 0; w < warp; ++w) { before.x += sh.wscan[w].x; before.y += sh.wscan[w].y; }
        return make_float2(before.x + s.x - v.x, before.y + s.y - v.y);
    };

    auto winner = [&]() -> int { return winner_of(best, lrow, M, T, prow); };

    // ---- each warp's list of its quads that reach x_min; f(quad, its logits) over the warp's list, 32 at a
    // time.  Order and shares are fixed.  A slice too long for the lists is walked instead.
    constexpr int PER_WARP = LISTED / WARPS;
    const bool listable = iters * 32 <= PER_WARP && q1 - q0 <= 65536;
    int n_quads = 0;
    float listed_x = -INFINITY;
    auto list_quads = [&](float x_min) {
        listed_x = x_min;
        if (!listable) return;
        n_quads = 0;
        uint16_t* mine = sh.quads + warp * PER_WARP;
        auto put = [&](int qd, const float4& v) {
            const float m = max_of(v);
            const uint32_t in = __ballot_sync(0xffffffffu, m >= x_min && m > -INFINITY);
            if ((in >> lane) & 1u) mine[n_quads + __popc(in & ((1u << lane) - 1u))] = static_cast<uint16_t>(qd - q0);
            n_quads += __popc(in);
        };
        sweep_warps<THREADS, LOADS>(lrow, q0, q1, whole, a.vocab, put);
        __syncwarp();
    };
    // f is called by whole warps (quad -1 and -inf logits for lanes without one)
    auto for_quads = [&](auto f) {
        if (!listable) {
            for (int i = 0; i < iters; ++i) {
                const int qd = q0 + i * THREADS + tid;
                const float4 v = qd < q1 ? load_quad(qd) : none;
                f(max_of(v) >= listed_x ? qd : -1, v);
            }
            return;
        }
        const uint16_t* mine = sh.quads + warp * PER_WARP;
        for (int i0 = 0; i0 < n_quads; i0 += 32 * LOADS) {
            float4 v[LOADS];
            int qd[LOADS];
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int at = i0 + i * 32 + lane;
                qd[i] = q0 + mine[min(at, n_quads - 1)];
                v[i] = whole > 0 ? load_whole(min(qd[i], whole - 1)) : none;
                if (at >= n_quads) {
                    qd[i] = -1;
                    v[i] = none;
                } else if (qd[i] >= whole) {
                    v[i] = load_quad(qd[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                if (i0 + i * 32 < n_quads) f(qd[i], v[i]);
        }
    };

    // ---- the list in the first CTA
    uint64_t* list0 = cluster.map_shared_rank(sh.list, 0);
    uint32_t* n0 = cluster.map_shared_rank(&sh.list_n, 0);
    auto collect = [&](uint64_t c) {
        const uint32_t at = atomicAdd(n0, 1u);
        if (at < CAP) list0[at] = c;
    };
    auto sort_list = [&](uint64_t* list, int n) { sort_members<THREADS>(sh, list, n); };
    auto kept_by_weight = [&](const uint64_t* list, int n, uint64_t above, uint64_t goal, uint64_t* sum) -> int {
        const Kept r = kept_members<THREADS>(sh, list, n, above, goal, M, per_logit);
        *sum = r.sum;
        return r.count;
    };
    auto goal_of = [&](uint64_t z) { return goal_of_sum(z, p); };
    auto race_list = [&](const uint64_t* list, int n) {
        for (int i = tid; i < n; i += THREADS) {
            const uint64_t c = list[i];
            if (composite_x(c) < min_x) break;
            best.add(composite(key_of_token(composite_x(c) - M, inv_t, noise_of(composite_col(c), prow)), composite_col(c)));
        }
    };

    // ---- top-k
    if (fast_k) {
        if (mx > -INFINITY) atomicAdd(&sh.tot[bin_of(depth(mx)) / (BINS / COARSE)], 1u);
        if (m2 > -INFINITY) atomicAdd(&sh.tot[bin_of(depth(m2)) / (BINS / COARSE)], 1u);
        __syncthreads();
        if (tid < COARSE) {
            const uint32_t cnt = sh.tot[tid];
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) *cluster.map_shared_rank(&sh.hist[rank * COARSE + tid], r) = cnt;
        }
        cluster.sync();
        float2 mine = make_float2(0.f, 0.f);
        if (tid < COARSE)
            for (int r = 0; r < CLUSTER; ++r) mine.x += static_cast<float>(sh.hist[r * COARSE + tid]);
        if (tid == 0) sh.first[0] = COARSE;
        const float2 run = scan2(mine);
        if (tid < COARSE && run.x < static_cast<float>(k) && run.x + mine.x >= static_cast<float>(k)) sh.first[0] = tid;
        __syncthreads();
        const int bound = sh.first[0];                    // COARSE: fewer than k maxima
        const int last_bin = bound < COARSE - 1 ? (bound + 1) * (BINS / COARSE) - 1 : BINS;
        // Collected by their bins, exactly; a row with fewer than k maxima above -inf, or with the k-th in the
        // last bins, collects everything it has (which fits if the vocabulary does).
        if (last_bin < BINS || a.vocab <= CAP) {
            const float x_end = last_bin < BINS ? x_at_end_of(last_bin) : -INFINITY;
            auto collect_quad = [&](int qd, const float4& v) {
                const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (l[e] > -INFINITY && (last_bin == BINS || bin_of(depth(l[e])) <= last_bin)) collect(composite(l[e], 4 * qd + e));
            };
            const bool two = m2 >= x_end && m2 > -INFINITY;
            if (mx >= x_end && mx > -INFINITY) {
                const float4 v1 = load_quad(mx_quad);
                const float4 v2 = load_quad(two ? m2_quad : mx_quad);
                collect_quad(mx_quad, v1);
                if (two) collect_quad(m2_quad, v2);
            }
            if (m3 >= x_end && m3 > -INFINITY)            // a third quad: this thread's share again
                sweep_quads([&](int qd, const float4& v) {
                    if (qd != mx_quad && qd != m2_quad && max_of(v) >= x_end) collect_quad(qd, v);
                });
            cluster.sync();
            const int n = static_cast<int>(*n0);
            if (n <= CAP) {
                if (rank != 0) return;
                auto read = cluster.barrier_arrive();     // the others leave once they have read the counter
                int col = 0;
                if (n > WARP_LIST)
                    col = list_winner<THREADS, CAP>(sh, lrow, n, min(k, n), need_p, 0, p, M, T, inv_t, per_logit, min_x, prow);
                else if (warp == 0)
                    col = list_winner<32, WARP_LIST>(sh, lrow, n, min(k, n), need_p, 0, p, M, T, inv_t, per_logit, min_x, prow);
                if (tid == 0) a.out_ids[row] = static_cast<int64_t>(col);
                cluster.barrier_wait(std::move(read));
                return;
            }
            cluster.sync();
            if (rank == 0 && tid == 0) sh.list_n = 0u;
        }
        for (int b = tid; b < BINS; b += THREADS) sh.hist[b] = 0u;
        cluster.sync();
    }

    // ---- thresholds by histogram
    uint64_t keep = 0;                                    // a token is kept if its composite is >= keep
    // From a range of members (bins [b_lo, b_hi] and composites >= keep, n of them) to the threshold.
    // By count: the goal-th member, in order.  By weight: the last member before which the weights,
    // those above the range in front, sum to less than the goal.  Sets `keep`; returns the weight of
    // every kept token (weigh: also when selecting by count).
    auto select = [&](bool by_weight, bool weigh, int b_lo, int b_hi, uint32_t n, uint64_t goal) -> uint64_t {
        float ws = 0.f;
        uint64_t cmin = ~0ull, cmax = 0ull;
        const bool fits = n <= CAP;
        sweep_from(b_hi < TAIL ? x_at_end_of(b_hi) : -INFINITY, [&](int col, float x) {
            const float d = depth(x);
            const int b = bin_of(d);
            if (b < b_lo) {
                if (weigh) ws += weight_of(d);
            } else if (b <= b_hi) {
                const uint64_t c = composite(x, col);
                if (c < keep) return;
                if (fits) collect(c);
                cmin = min(cmin, c);
                cmax = max(cmax, c);
            }
        });
        uint64_t above = cluster_sum(fixed_of(ws));
        if (!fits) {
            cluster_range(cmin, cmax);
            for (int half = 0; half < 64 && n > CAP; ++half) {          // composites differ: 64 halvings leave one
                const uint64_t mid = cmin + ((cmax - cmin) >> 1);       // upper half: (mid, cmax]
                ws = 0.f;
                uint32_t cnt = 0;
                sweep_from(composite_x(mid), [&](int col, float x) {
                    const uint64_t c = composite(x, col);
                    if (c <= mid || c > cmax) return;
                    ++cnt;
                    if (weigh) ws += weight_of(depth(x));
                });
                const uint32_t upper = static_cast<uint32_t>(cluster_sum(cnt));
                const uint64_t w_upper = weigh ? cluster_sum(fixed_of(ws)) : 0ull;
                if (by_weight ? above + w_upper >= goal : upper >= goal) {
                    cmin = mid + 1;
                    n = upper;
                } else {
                    above += w_upper;
                    if (!by_weight) goal -= upper;
                    cmax = mid;
                    n -= upper;
                }
            }
            sweep_from(composite_x(cmin), [&](int col, float x) {
                const uint64_t c = composite(x, col);
                if (c >= cmin && c <= cmax) collect(c);
            });
            cluster.sync();
        }
        if (rank == 0) {
            n = min(sh.list_n, static_cast<uint32_t>(CAP));              // as counted
            __syncthreads();
            sort_list(sh.list, static_cast<int>(n));
            uint64_t sum = 0;
            int kept = static_cast<int>(min(goal, static_cast<uint64_t>(n)));
            if (by_weight) kept = kept_by_weight(sh.list, static_cast<int>(n), above, goal, &sum);
            else if (weigh) kept_by_weight(sh.list, kept, 0, ~0ull, &sum);
            if (tid < CLUSTER) {
                // none kept: just above the range
                *cluster.map_shared_rank(&sh.threshold, tid) = kept > 0 ? sh.list[kept - 1] : n > 0 ? sh.list[0] + 1 : cmax + 1;
                *cluster.map_shared_rank(&sh.list_sum, tid) = above + sum;
            }
            if (tid == 0) sh.list_n = 0u;
        }
        cluster.sync();
        keep = sh.threshold;
        return sh.list_sum;
    };

    // ---- races.  `exact`: `keep` is where the filters end, but for min-p's.  Until then a winner is one of the
    // filters' if the weights before it are less than the goal, and if it is not, neither is what comes after it.
    bool exact = !need_k && !need_p;
    int tries = need_k ? 0 : TRIES;
    bool raced = race_all;
    for (;; raced = false) {
        if (!exact && tries == 0) {
            keep = 0;
            best.clear();
            int k_bin = BINS;                                 // the bin of the last token top-k keeps
            uint32_t k_left = 0;                              // tokens it keeps in that bin
            int end = TAIL;                                   // bins that top-p's border can lie in, or that the race reaches
            if (need_k) {
                float ws = 0.f;
                uint32_t tail = 0;
                sweep_from(-INFINITY, [&](int, float x) {
                    const float d = depth(x);
                    const int b = bin_of(d);
                    if (b == TAIL) ++tail; else atomicAdd(&sh.hist[b], 1u);
                    if (need_p) ws += weight_of(d);
                });
                tail = __reduce_add_sync(0xffffffffu, tail);
                if (lane == 0 && tail) atomicAdd(&sh.hist[TAIL], tail);
                Z = cluster_sum(fixed_of(ws));
                cluster_hist();
                // exact in fp32: the vocabulary is limited to 2^24
                float2 mine = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < BINS_PER_THREAD; ++i) mine.x += static_cast<float>(sh.tot[tid * BINS_PER_THREAD + i]);
                float2 run = scan2(mine);
                if (tid == 0) { sh.first[0] = BINS; sh.first[1] = 0; }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < BINS_PER_THREAD; ++i) {
                    const int b = tid * BINS_PER_THREAD + i;
                    const float before = run.x;
                    run.x += static_cast<float>(sh.tot[b]);
                    if (before < static_cast<float>(k) && run.x >= static_cast<float>(k)) {
                        sh.first[0] = b;
                        sh.first[1] = k - static_cast<int>(before);
                    }
                }
                __syncthreads();
                k_bin = sh.first[0];
                k_left = static_cast<uint32_t>(sh.first[1]);
                __syncthreads();
                // every token of the tail is out of the race's reach: without top-p its order does not matter
                if (k_bin < TAIL || (k_bin == TAIL && need_p))
                    Z = select(false, need_p, k_bin, k_bin, sh.tot[k_bin], k_left);
            } else {
                // tokens lighter than (1 - p) Z / vocab are outside; the limit in bins, with a margin
                const float z_f = static_cast<float>(Z) * (1.f / FIX);
                const float limit = (log2f(static_cast<float>(a.vocab)) - log2f((1.f - p) * z_f)) * BINS_PER_OCTAVE * 1.00001f + 2.f;
                end = limit < static_cast<float>(TAIL) ? max(1, static_cast<int>(limit)) : TAIL;
                list_quads(x_at_end_of(end));
                for_quads([&](int, const float4& v) {
                    const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int b = bin_of(depth(l[e]));
                        if (b < end) atomicAdd(&sh.hist[b], 1u);
                    }
                });
                cluster_hist();
            }
            if (need_p) {
                const uint64_t goal = goal_of(Z);
                const float goal_f = static_cast<float>(goal) * (1.f / FIX);
                auto kept_in = [&](int b) { return b < k_bin ? sh.tot[b] : b == k_bin ? k_left : 0u; };   // after top-k
                // The bins [b_lo, b_hi] in which the running sum may reach what is left of the goal, from counts(b) and
                // the largest and smallest weight of a bin; thread t holds bins BINS_PER_THREAD t ...; and their members.
                int b_lo = 0, b_hi = 0;
                uint32_t n_in = 0;
                auto find = [&](float left, int last, auto counts, auto weight_at) {
                    float up[BINS_PER_THREAD], dn[BINS_PER_THREAD];
                    float2 mine = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < BINS_PER_THREAD; ++i) {
                        const int b = tid * BINS_PER_THREAD + i;
                        const float cnt = static_cast<float>(counts(b));
                        up[i] = cnt * weight_at(b);
                        dn[i] = cnt * weight_at(b + 1);
                        mine.x += up[i];
                        mine.y += dn[i];
                    }
                    float2 run = scan2(mine);
                    if (tid == 0) sh.first[0] = sh.first[1] = BINS;
                    __syncthreads();
                    const float at_up = left * (1.f - 1e-4f), at_dn = left * (1.f + 1e-4f);
                    // the threads whose sums reach a mark from below it, or from so little above that rounding may be
                    // what put the prefix there
                    int b_up = BINS, b_dn = BINS;
                    const bool mine_up = run.x < at_up * 1.0001f, mine_dn = run.y < at_dn * 1.0001f;
#pragma unroll
                    for (int i = 0; i < BINS_PER_THREAD; ++i) {
                        run.x += up[i];
                        run.y += dn[i];
                        if (run.x >= at_up) b_up = min(b_up, tid * BINS_PER_THREAD + i);
                        if (run.y >= at_dn) b_dn = min(b_dn, tid * BINS_PER_THREAD + i);
                    }
                    if (mine_up && b_up < BINS) atomicMin(&sh.first[0], b_up);
                    if (mine_dn && b_dn < BINS) atomicMin(&sh.first[1], b_dn);
                    __syncthreads();
                    b_lo = sh.first[0];
                    b_hi = min(max(b_lo, sh.first[1]), last);
                    n_in = 0;
                    for (int b = b_lo + lane; b <= b_hi; b += 32) n_in += counts(b);
                    n_in = __reduce_add_sync(0xffffffffu, n_in);
                    __syncthreads();
                };
                find(goal_f, end - 1, kept_in, [&](int b) { return b > TAIL ? 0.f : weight_of(static_cast<float>(b)); });
                if (b_lo <= b_hi && !need_k) {
                    // the depths of the range, and what lies above it; a second histogram if the range holds too many
                    float d_lo = static_cast<float>(b_lo), d_hi = static_cast<float>(b_hi + 1), sub = 0.f;
                    const uint32_t n_range = n_in;
                    int s_lo = 0, s_hi = 0;
                    if (n_in > BORDER) {
                        for (int b = tid; b < BINS; b += THREADS) sh.hist[b] = 0u;
                        __syncthreads();
                        sub = static_cast<float>(BINS) / (d_hi - d_lo);
                        auto sub_of = [&](float d) { return min(static_cast<int>((d - d_lo) * sub), BINS - 1); };
                        float ws = 0.f;
                        for_quads([&](int, const float4& v) {
                            const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float d = depth(l[e]);
                                if (d < d_lo) ws += weight_of(d);
                                else if (d < d_hi) atomicAdd(&sh.hist[sub_of(d)], 1u);
                            }
                        });
                        const uint64_t above = cluster_sum(fixed_of(ws));
                        cluster_hist();
                        // (a sum that rounding puts past the goal already leaves the first members as the range)
                        const float left = goal > above ? static_cast<float>(goal - above) * (1.f / FIX) : 0.f;
                        find(fmaxf(left, 1e-30f), BINS - 1, [&](int b) { return sh.tot[b]; },
                             [&](int b) { return weight_of(d_lo + static_cast<float>(b) / sub); });
                        s_lo = b_lo;
                        s_hi = b_hi;
                    }
                    if (n_in <= BORDER && b_lo <= b_hi) {
                        // sum and race what is above the range, collect the range
                        uint64_t* border0 = cluster.map_shared_rank(sh.border, 0);
                        float ws = 0.f, bar = -INFINITY;
                        for_quads([&](int qd, const float4& v) {
                            float l[4] = {v.x, v.y, v.z, v.w}, lmax = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float d = depth(l[e]);
                                bool sure = d < d_lo, in = !sure && d < d_hi;
                                if (in && sub > 0.f) {
                                    const int b = min(static_cast<int>((d - d_lo) * sub), BINS - 1);
                                    sure = b < s_lo;
                                    in = b >= s_lo && b <= s_hi;
                                }
                                if (sure) ws += weight_of(d);
                                if (in) {
                                    const uint32_t at = atomicAdd(n0, 1u);
                                    if (at < BORDER) border0[at] = composite(l[e], 4 * qd + e);
                                }
                                if (!(sure && l[e] >= min_x)) l[e] = -INFINITY;
                                lmax = fmaxf(lmax, l[e]);
                            }
                            if (lmax > -INFINITY) race_quad(best, qd, l, lmax, M, bar, inv_t, l2, noise_quad(static_cast<uint32_t>(qd), prow));
                            bar = warp_max(best.key());
                        });
                        block_best();
                        if (tid == 0) put_best(0);
                        const uint64_t above = cluster_sum(fixed_of(ws));
                        if (rank != 0) return;
                        const int members = static_cast<int>(min(sh.list_n, static_cast<uint32_t>(BORDER)));     // n_in
                        sort_list(sh.border, members);
                        uint64_t sum;
                        const int kept = kept_by_weight(sh.border, members, above, goal, &sum);
                        best.clear();
                        race_list(sh.border, kept);
                        block_best();
                        if (warp == 0) {
                            if (lane != 0) best.clear();      // the border's best counts once
                            if (lane < CLUSTER) best.merge(sh.win[lane][0], sh.win[lane][1]);
                            warp_best();
                            if (lane == 0) a.out_ids[row] = winner();
                        }
                        return;
                    }
                    // thousands of equal logits at the border: halve it
                    b_lo = static_cast<int>(d_lo);
                    b_hi = static_cast<int>(d_hi) - 1;
                    n_in = n_range;
                }
                if (b_lo <= b_hi) select(true, true, b_lo, b_hi, n_in, goal);
            }
            exact = true;
        }
        if (!raced) {
            const float x_keep = keep ? composite_x(keep) : -INFINITY, x_from = fmaxf(min_x, x_keep);
            const uint32_t col_keep = keep ? static_cast<uint32_t>(composite_col(keep)) : 0xffffffffu;    // at x_keep itself: columns up to this
            float bar = -INFINITY;
            best.clear();
            list_quads(x_from);
            for_quads([&](int qd, const float4& v) {
                float l[4] = {v.x, v.y, v.z, v.w}, lmax = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!(l[e] >= x_from && (l[e] > x_keep || static_cast<uint32_t>(4 * qd + e) <= col_keep))) l[e] = -INFINITY;
                    lmax = fmaxf(lmax, l[e]);
                }
                bool any = false;
                if (lmax > -INFINITY) any = race_quad(best, qd, l, lmax, M, bar, inv_t, l2, noise_quad(static_cast<uint32_t>(qd), prow));
                if (__any_sync(0xffffffffu, any)) bar = TRIED > 1 ? warp_second(best) : warp_max(best.key());
            });
            gather_best();
            cluster.sync();
        }
        // the race's best tokens: the best of 32 by a warp each, of those by the first
        constexpr int LISTS = CLUSTER * PUT * 2 / 32, EACH = (LISTS * (TRIED + 1) + 31) / 32;
        const int wanted = exact ? 2 : TRIED + 1;
        if (warp < LISTS) {
            const int at = warp * 32 + lane;
            uint64_t e = sh.parts[at >> 1][at & 1];
            if (raced && e) e = composite(composite_x(e) + (composite_x(sh.top[at / (2 * PUT)]) - M) * inv_t, composite_col(e));
#pragma unroll 1
            for (int j = 0; j < wanted; ++j) {
                const uint64_t m = warp_max64(e);
                if (e == m) {
                    (LISTS > 1 ? sh.lists[warp] : sh.cand)[j] = m;
                    (LISTS > 1 ? sh.list_part[warp] : sh.cand_part)[j] = at >> 1;
                    e = 0;
                }
            }
        }
        if (LISTS > 1) __syncthreads();
        else __syncwarp();
        if (warp == 0) {
            if (LISTS > 1) {
                uint64_t e[EACH];
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    const int at = i * 32 + lane;
                    e[i] = at < LISTS * (TRIED + 1) && at % (TRIED + 1) < wanted ? sh.lists[at / (TRIED + 1)][at % (TRIED + 1)] : 0;
                }
#pragma unroll 1
                for (int j = 0; j < wanted; ++j) {
                    uint64_t m = e[0];
#pragma unroll
                    for (int i = 1; i < EACH; ++i) m = max(m, e[i]);
                    m = warp_max64(m);
                    if (lane == 0) sh.cand[j] = m;
#pragma unroll
                    for (int i = 0; i < EACH; ++i)
                        if (m && e[i] == m) {
                            e[i] = 0;
                            sh.cand_part[j] = sh.list_part[(i * 32 + lane) / (TRIED + 1)][(i * 32 + lane) % (TRIED + 1)];
                        }
                }
                __syncwarp();
            }
            if (lane < CANDS && !exact) {
                const int col = composite_col(sh.cand[lane]);
                const float x = lane < TRIED && sh.cand[lane] ? __ldg(lrow + col) : -INFINITY;
                sh.cand_x[lane] = x;
                sh.cand_at[lane] = x > -INFINITY ? composite(x, col) : ~0ull;
            }
        }
        __syncthreads();
        int first = 0, next = 1;                          // the first candidate that stands, and the next
        if (!exact) {
            float x_low = INFINITY;
            uint64_t top_c = 0;                           // the candidate that comes first in the order
#pragma unroll 1
            for (int j = 0; j < TRIED && sh.cand[j]; ++j) {
                x_low = fminf(x_low, sh.cand_x[j]);
                top_c = max(top_c, sh.cand_at[j]);
            }
            Before sums = {};                             // before each of them; and the tokens before that one
            sweep_quads_by(std::integral_constant<int, CHECK_LOADS>{}, [&](int qd, const float4& v) {
                if (max_of(v) >= x_low) sums = add_before(sums, sh, v, qd, M, per_logit, top_c);
            }, std::false_type{});
            const uint32_t before = __reduce_add_sync(0xffffffffu, sums.count);
#pragma unroll
            for (int j = 0; j < TRIED; ++j) {
                uint64_t f = fixed_of(sums.w[j]);
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) f += shfl_xor64(f, off);
                if (lane == 0) sh.wsum[warp][j] = f;
            }
            if (lane == 0) sh.wlo[warp] = before;
            __syncthreads();
            if (tid < CLUSTER * TRIED) {
                const int to = tid / TRIED, j = tid % TRIED;
                uint64_t f = 0, n = 0;
                for (int w = 0; w < WARPS; ++w) { f += sh.wsum[w][j]; n += sh.wlo[w]; }
                *cluster.map_shared_rank(&sh.csum[rank][j], to) = f;
                if (j == 0) *cluster.map_shared_rank(&sh.ccnt[rank], to) = static_cast<uint32_t>(n);
            }
            cluster.sync();
            const uint64_t goal = goal_of(Z);
            uint64_t out = 0;                             // the excluded candidate that comes first in the order
            bool known = true;                            // no part had both of its two best excluded
            int stands[2] = {-1, -1};
#pragma unroll 1
            for (int j = 0; j < TRIED && sh.cand[j]; ++j) {
                uint64_t f = 0;
#pragma unroll
                for (int r = 0; r < CLUSTER; ++r) f += sh.csum[r][j];
                if (f < goal) {
                    if (stands[0] < 0) stands[0] = j;
                    else if (stands[1] < 0) stands[1] = j;
                } else if (stands[0] < 0) {
                    for (int i = 0; i < j; ++i) known = known && sh.cand_part[i] != sh.cand_part[j];
                    out = max(out, sh.cand_at[j]);
                }
            }
            first = stands[0];
            next = stands[1] < 0 ? TRIED + 1 : stands[1];
            // none stands, or a token of a part whose two best are out might beat it: race again what is left; or one
            // that was not examined is too near it: the border decides
            const bool near = first >= 0 && stands[1] < 0 && sh.cand[TRIED] &&
                              composite_x(sh.cand[first]) - composite_x(sh.cand[TRIED]) <= NEAR;
            if (first < 0 || !known || near) {
                uint32_t n = 0;
                for (int r = 0; r < CLUSTER; ++r) n += sh.ccnt[r];
                keep = out + 1;
                // (decided by what every CTA has from the same exchange, so that a row that is written under the call
                // cannot part them)
                if (first < 0 && n <= CAP) {              // out is top_c: the first CTA ends it
                    sweep_from(composite_x(out), [&](int other, float x) {
                        if (composite(x, other) > out) collect(composite(x, other));
                    });
                    cluster.sync();
                    if (rank != 0) return;
                    n = min(sh.list_n, static_cast<uint32_t>(CAP));
                    const int last = list_winner<THREADS, CAP>(sh, lrow, static_cast<int>(n), static_cast<int>(n), true, goal, p, M, T,
                                                               inv_t, per_logit, min_x, prow);
                    if (tid == 0) a.out_ids[row] = static_cast<int64_t>(last);
                    return;
                }
                tries = near ? 0 : tries - 1;
                continue;
            }
        }
        if (rank == 0 && tid == 0) {
            best.b1 = sh.cand[first];
            best.b2 = next <= TRIED ? sh.cand[next] : 0;
            a.out_ids[row] = static_cast<int64_t>(winner());
        }
        return;
    }
}

template <int CLUSTER, int THREADS, int LOADS1, int MIN_CTAS, int TRIED>
struct Rows {
    static constexpr auto kernel = sample_filtered_kernel<CLUSTER, THREADS, LOADS1, MIN_CTAS, TRIED>;
    static cudaError_t launch(const Args& args, cudaStream_t stream) {
        kernel<<<dim3(CLUSTER, args.a.batch), THREADS, 0, stream>>>(args);
        return cudaGetLastError();
    }
};
using FewRows = Rows<16, 512, 5, 1, 1>;
using SomeRows = Rows<8, 256, 8, 4, CANDS>;
using ManyRows = Rows<4, 256, 8, 4, CANDS>;

}  // namespace

pkv_status launch_sample_filtered(const SampleFilteredArgs& a, int* err, cudaStream_t stream) {
    if (a.batch == 0) return PKV_OK;
    if (!setup_once(kSetupSampleFiltered, [] {
            return cudaFuncSetAttribute(FewRows::kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
        }))
        return PKV_ERR_CUDA;
    Args args;
    args.a = a;
    args.vec_ok = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && (a.batch == 1 || a.row_stride % 4 == 0);
    args.err = err;
    // The more CTAs to a row, the sooner it is done; the fewer, the less of its time goes into their barriers.  7
    // clusters of 16 x 512 threads run at once, half as many rows as there are SMs on clusters of 8 x 256 (four CTAs to
    // an SM), as many rows as SMs on clusters of 4.  Rows of 151,936 with settings of their own, us: 8 rows 22 on 16 and
    // 28 on 8, 10 rows 22 and 28, 12 rows 35 and 29; 120 rows 53 on 8 and 70 on 4, 228 rows 84 and 78, 512 rows 162 and
    // 119 (256 rows without filters 109 and 82).  Their order: 120 rows 61 without it, 512 rows 136; equal rows lose
    // 3 us to it.  Other vocabularies, L2 flushed before each call: 262,144 logits 8 rows 29 on 16 and 42 on 8, 12 rows 33
    // and 40, 190 rows 87 on 8 and 115 on 4, 300 rows 122 and 142; 32,000 logits 8 rows 25 and 24, 10 rows 28 and 24, 120
    // rows 36 on 8 and 34 on 4, 300 rows 73 and 50.  So the limits, which go by rows alone, are right within a few
    // us around 151,936 logits, and at 262,144 clusters of 8 would win past 300 rows still.
    constexpr int kWideRows = 10;
    const int sms = sm_count();
    const bool wide = a.batch <= kWideRows, some = 4 * a.batch <= 5 * sms;
    args.ordered = !wide && a.batch > (some ? sms / 2 : sms) && a.batch <= ORDERED_ROWS;
    const cudaError_t e = wide ? FewRows::launch(args, stream) : some ? SomeRows::launch(args, stream) : ManyRows::launch(args, stream);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
