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
// One cluster of 8 CTAs takes a row: each CTA copies its eighth of the row into shared memory
// once (151,936 logits: 76 KB, two CTAs per SM) and every later step reads that copy, so HBM sees
// each logit once.  A kept set is an upper set of the order, so top-k and top-p each come down to
// one threshold (logit, column):
//
//   1  Histogram of z over 2048 bins of width 0.01 (integer counts, so the order of the atomics
//      does not matter), summed over the cluster.
//   2  Top-k: the bin where the count reaches k.  Top-p: a bin holds weights within 1% of one
//      another, so the counts bound the running sum from both sides and leave a few bins where
//      it may reach its goal.
//   3  One sweep sums the weights above those bins (fixed order: threads, then CTAs in rank order)
//      and collects the bins' members, at most 1024, in the first CTA, which sorts them and finds
//      the threshold.  More members than that (a flat row, thousands of equal logits) are first
//      halved, by (logit bits, column), as often as it takes.
//
// Sums: weights in fp32 (ex2.approx), a thread's share (37 of 151,936 terms) in fp32, everything
// across threads in fp64: a running sum is within about 1e-7 of itself, so the token at the
// border is decided as in exact arithmetic except when a border lies that near to it.
//
// The race's keys are fp32 with an error below 2e-5; when the two best are within 1e-4 the
// candidates are ranked again in fp64.
#include <cooperative_groups.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_noise.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int CLUSTER = 8;
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int BINS_PER_THREAD = BINS / THREADS;
constexpr int BINS_PER_RANK = BINS / CLUSTER;
constexpr int TAIL = BINS - 1;               // the last bin: everything from z = -20.47 down
constexpr float BINS_PER_UNIT = 100.f;
constexpr float TAIL_Z = 20.47f;
constexpr int CAP = 1024;                    // members sorted at once
constexpr float RACE_Z = 19.6f;              // reach of the race (see above)
constexpr float NEAR = 1e-4f;
constexpr int kMaxResident = 22016;          // logits of a slice in shared memory: 2 CTAs per SM
constexpr float LOG2E = 1.4426950408889634f;
static_assert(BINS_PER_RANK <= THREADS && 2 * THREADS >= CAP, "one element per thread in the reductions and the sort");

struct Shared {
    uint32_t hist[BINS];         // this CTA's counts
    uint32_t tot[BINS];          // the cluster's counts
    uint64_t list[CAP];          // first CTA: members, as composites
    double slot[2][CLUSTER];     // cluster-wide sums, alternating
    uint64_t lo[CLUSTER], hi[CLUSTER];
    uint64_t threshold;
    double list_sum;
    double wred[WARPS];
    uint64_t wlo[WARPS], whi[WARPS];
    float2 wscan[WARPS];
    float2 win[CLUSTER];         // race: best and second best key of each CTA
    int win_col[CLUSTER];
    float wbest[WARPS], wsecond[WARPS];
    int wcol[WARPS];
    float min_x;                 // smallest logit that min-p keeps
    int first[2];
    uint32_t list_n;
};

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

__device__ __forceinline__ int bin_of(float d) {   // d = max z - z; non-decreasing in d
    return d < TAIL_Z ? min(static_cast<int>(d * BINS_PER_UNIT), TAIL - 1) : TAIL;
}
__device__ __forceinline__ float weight_of(float d) { return ex2_ftz(-d * LOG2E); }

struct Args {
    SampleFilteredArgs a;
    int vec_ok;
    int* err;
};

template <bool kResident>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS, 2) sample_filtered_kernel(const Args args) {
    const SampleFilteredArgs& a = args.a;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    float* slice = reinterpret_cast<float*>(smem_raw + (sizeof(Shared) + 15) / 16 * 16);
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const float T = __ldg(a.temperatures + row);
    int k = a.top_k ? __ldg(a.top_k + row) : 0;
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
    const float inv_t = fminf(1.0f / T, 3.4028235e38f);

    // ---- this CTA's slice: whole quads [q0, q1) of the row; absent columns read as NaN
    const float* lrow = a.logits + static_cast<int64_t>(row) * a.row_stride;
    const int nquads = (a.vocab + 3) >> 2;
    const int per = (nquads + CLUSTER - 1) / CLUSTER;
    const int q0 = min(nquads, rank * per), q1 = min(nquads, q0 + per);
    auto load_quad = [&](int qd) -> float4 {
        const int col = qd * 4;
        if (args.vec_ok && col + 3 < a.vocab) return __ldg(reinterpret_cast<const float4*>(lrow + col));
        const float none = __uint_as_float(0x7fc00000u);
        float4 v;
        v.x = __ldg(lrow + col);
        v.y = col + 1 < a.vocab ? __ldg(lrow + col + 1) : none;
        v.z = col + 2 < a.vocab ? __ldg(lrow + col + 2) : none;
        v.w = col + 3 < a.vocab ? __ldg(lrow + col + 3) : none;
        return v;
    };
    // f(column, logit) for every logit of the slice that is above -inf (not NaN)
    auto sweep = [&](auto f) {
        for (int qd = q0 + tid; qd < q1; qd += THREADS) {
            const float4 v = kResident ? reinterpret_cast<const float4*>(slice)[qd - q0] : load_quad(qd);
            if (v.x > -INFINITY) f(4 * qd, v.x);
            if (v.y > -INFINITY) f(4 * qd + 1, v.y);
            if (v.z > -INFINITY) f(4 * qd + 2, v.z);
            if (v.w > -INFINITY) f(4 * qd + 3, v.w);
        }
    };
    for (int b = tid; b < BINS; b += THREADS) sh.hist[b] = 0u;
    if (tid == 0) sh.list_n = 0u;
    float mx = -INFINITY;
#pragma unroll 4
    for (int qd = q0 + tid; qd < q1; qd += THREADS) {
        const float4 v = load_quad(qd);
        if (kResident) reinterpret_cast<float4*>(slice)[qd - q0] = v;
        mx = fmaxf(fmax3(mx, v.x, v.y), fmaxf(v.z, v.w));     // NaN loses
    }

    // ---- cluster-wide reductions; every CTA ends with the same values
    int phase = 0;
    auto cluster_sum = [&](double v) -> double {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) sh.wred[warp] = v;
        __syncthreads();
        double* mine = &sh.slot[phase][rank];
        if (tid < CLUSTER) {
            double s = 0.0;
            for (int w = 0; w < WARPS; ++w) s += sh.wred[w];
            *cluster.map_shared_rank(mine, tid) = s;
        }
        cluster.sync();
        double s = 0.0;
        for (int r = 0; r < CLUSTER; ++r) s += sh.slot[phase][r];
        phase ^= 1;
        return s;
    };
    // smallest and largest of two 64-bit numbers
    auto cluster_range = [&](uint64_t& lo, uint64_t& hi) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            lo = min(lo, static_cast<uint64_t>(__shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(lo), off)));
            hi = max(hi, static_cast<uint64_t>(__shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(hi), off)));
        }
        if (lane == 0) { sh.wlo[warp] = lo; sh.whi[warp] = hi; }
        __syncthreads();
        if (tid < CLUSTER) {
            for (int w = 0; w < WARPS; ++w) { lo = min(lo, sh.wlo[w]); hi = max(hi, sh.whi[w]); }
            *cluster.map_shared_rank(&sh.lo[rank], tid) = lo;
            *cluster.map_shared_rank(&sh.hi[rank], tid) = hi;
        }
        cluster.sync();
        lo = sh.lo[0];
        hi = sh.hi[0];
        for (int r = 1; r < CLUSTER; ++r) { lo = min(lo, sh.lo[r]); hi = max(hi, sh.hi[r]); }
        cluster.sync();                                   // read before anyone writes them again
    };
    // the cluster's histogram from every CTA's, which is cleared for its next use
    auto cluster_hist = [&]() {
        cluster.sync();
        if (tid < BINS_PER_RANK) {
            const int b = rank * BINS_PER_RANK + tid;
            uint32_t s = 0;
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) s += *cluster.map_shared_rank(&sh.hist[b], r);
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) *cluster.map_shared_rank(&sh.tot[b], r) = s;
        }
        cluster.sync();
        for (int b = tid; b < BINS; b += THREADS) sh.hist[b] = 0u;
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

    uint64_t lo64 = 0, hi64 = (mx > -INFINITY) ? key_of(mx) : 0u;
    cluster_range(lo64, hi64);                            // its barriers also publish the slice and the cleared histogram
    if (hi64 == 0) {                                      // nothing above -inf
        if (rank == 0 && tid == 0) a.out_ids[row] = -1;
        return;
    }
    const float M = value_of(static_cast<uint32_t>(hi64));
    if (M == INFINITY) {                                  // infinite logits win; the lowest column among them
        uint64_t first = ~0ull, none = 0;
        sweep([&](int col, float x) { if (x == INFINITY) first = min(first, static_cast<uint64_t>(col)); });
        cluster_range(first, none);
        if (rank == 0 && tid == 0) a.out_ids[row] = static_cast<int64_t>(first);
        return;
    }
    if (tid == 0)
        sh.min_x = mp > 0.f ? __double2float_ru(static_cast<double>(M) + static_cast<double>(T) * log(static_cast<double>(mp)))
                            : -INFINITY;
    auto depth = [&](float x) { return (M - x) * inv_t; };

    // ---- thresholds
    uint64_t keep = 0;                                    // a token is kept if its composite is >= keep
    bool need_k = k > 0 && k < a.vocab;
    const bool need_p = p < 1.f;

    // From a range of members (bins [b_lo, b_hi] and composites >= keep, n of them) to the threshold.
    // By count: the goal-th member, in order.  By weight: the last member before which the weights,
    // those above the range in front, sum to less than the goal.  Sets `keep`; returns the weight of
    // every kept token (weigh: also when selecting by count).
    auto select = [&](bool by_weight, bool weigh, int b_lo, int b_hi, uint32_t n, double goal) -> double {
        float ws = 0.f;
        uint64_t cmin = ~0ull, cmax = 0ull;
        uint64_t* list0 = cluster.map_shared_rank(sh.list, 0);
        uint32_t* n0 = cluster.map_shared_rank(&sh.list_n, 0);
        auto collect = [&](uint64_t c) {
            const uint32_t at = atomicAdd(n0, 1u);
            if (at < CAP) list0[at] = c;
        };
        const bool fits = n <= CAP;
        sweep([&](int col, float x) {
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
        double above = cluster_sum(static_cast<double>(ws));
        if (!fits) {
            cluster_range(cmin, cmax);
            for (int half = 0; half < 64 && n > CAP; ++half) {       // composites differ: 64 halvings leave one
                const uint64_t mid = cmin + ((cmax - cmin) >> 1);       // upper half: (mid, cmax]
                ws = 0.f;
                uint32_t cnt = 0;
                sweep([&](int col, float x) {
                    const uint64_t c = composite(x, col);
                    if (c <= mid || c > cmax) return;
                    ++cnt;
                    if (weigh) ws += weight_of(depth(x));
                });
                const uint32_t upper = static_cast<uint32_t>(cluster_sum(static_cast<double>(cnt)));
                const double w_upper = weigh ? cluster_sum(static_cast<double>(ws)) : 0.0;
                if (by_weight ? above + w_upper >= goal : static_cast<double>(upper) >= goal) {
                    cmin = mid + 1;
                    n = upper;
                } else {
                    above += w_upper;
                    if (!by_weight) goal -= static_cast<double>(upper);
                    cmax = mid;
                    n -= upper;
                }
            }
            sweep([&](int col, float x) {
                const uint64_t c = composite(x, col);
                if (c >= cmin && c <= cmax) collect(c);
            });
            n = min(n, static_cast<uint32_t>(CAP));
            cluster.sync();
        }
        // the first CTA sorts the members, earliest first, and finds the threshold
        if (rank == 0) {
            int n2 = 32;
            while (n2 < static_cast<int>(n)) n2 <<= 1;
            for (int i = static_cast<int>(n) + tid; i < n2; i += THREADS) sh.list[i] = 0ull;
            __syncthreads();
            for (int size = 2; size <= n2; size <<= 1)
                for (int half = size >> 1; half >= 1; half >>= 1) {
                    for (int i = tid; i < (n2 >> 1); i += THREADS) {
                        const int x = (i / half) * 2 * half + (i % half), y = x + half;
                        const uint64_t cx = sh.list[x], cy = sh.list[y];
                        const bool down = (x & size) == 0;
                        if (down ? cx < cy : cx > cy) {
                            sh.list[x] = cy;
                            sh.list[y] = cx;
                        }
                    }
                    __syncthreads();
                }
            // weights of members 2 tid, 2 tid + 1 and the sum before them
            const int i0 = 2 * tid, i1 = i0 + 1;
            double w0 = 0.0, w1 = 0.0;
            if (weigh) {
                if (i0 < static_cast<int>(n)) w0 = weight_of(depth(value_of(static_cast<uint32_t>(sh.list[i0] >> 32))));
                if (i1 < static_cast<int>(n)) w1 = weight_of(depth(value_of(static_cast<uint32_t>(sh.list[i1] >> 32))));
            }
            double s = w0 + w1;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double x = __shfl_up_sync(0xffffffffu, s, off);
                if (lane >= off) s += x;
            }
            if (lane == 31) sh.wred[warp] = s;
            __syncthreads();
            double before = above;
            for (int w = 0; w < warp; ++w) before += sh.wred[w];
            before += s - w0 - w1;
            const bool in0 = i0 < static_cast<int>(n) && (by_weight ? before < goal : i0 < goal);
            const bool in1 = i1 < static_cast<int>(n) && (by_weight ? before + w0 < goal : i1 < goal);
            const int kept = __syncthreads_count(in0) + __syncthreads_count(in1);
            double part = (in0 ? w0 : 0.0) + (in1 ? w1 : 0.0);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
            if (lane == 0) sh.wred[warp] = part;
            __syncthreads();
            if (tid < CLUSTER) {
                double sum = above;
                for (int w = 0; w < WARPS; ++w) sum += sh.wred[w];
                // none kept: just above the range
                *cluster.map_shared_rank(&sh.threshold, tid) = kept > 0 ? sh.list[kept - 1] : n > 0 ? sh.list[0] + 1 : cmax + 1;
                *cluster.map_shared_rank(&sh.list_sum, tid) = sum;
            }
            if (tid == 0) sh.list_n = 0u;
        }
        cluster.sync();
        keep = sh.threshold;
        return sh.list_sum;
    };

    if (need_k || need_p) {
        float ws = 0.f;
        uint32_t tail = 0;
        sweep([&](int, float x) {
            const float d = depth(x);
            const int b = bin_of(d);
            if (b == TAIL) ++tail; else atomicAdd(&sh.hist[b], 1u);
            if (need_p) ws += weight_of(d);
        });
        tail = __reduce_add_sync(0xffffffffu, tail);
        if (lane == 0 && tail) atomicAdd(&sh.hist[TAIL], tail);
        double Z = cluster_sum(static_cast<double>(ws));
        cluster_hist();
        int k_bin = BINS;                                 // the bin of the last token top-k keeps
        uint32_t k_left = 0;                              // tokens it keeps in that bin
        if (need_k) {
            // counts are below 2^24 in fp32 where it matters: the vocabulary is limited to that
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
                Z = select(false, need_p, k_bin, k_bin, sh.tot[k_bin], static_cast<double>(k_left));
        }
        if (need_p) {
            const double goal = static_cast<double>(p) * Z;
            auto kept_in = [&](int b) { return b < k_bin ? sh.tot[b] : b == k_bin ? k_left : 0u; };   // after top-k
            // bounds of the running sum at the end of each bin
            float up[BINS_PER_THREAD], dn[BINS_PER_THREAD];
            float2 mine = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < BINS_PER_THREAD; ++i) {
                const int b = tid * BINS_PER_THREAD + i;
                const float cnt = static_cast<float>(kept_in(b));
                up[i] = cnt * weight_of(b / BINS_PER_UNIT);
                dn[i] = b == TAIL ? 0.f : cnt * weight_of((b + 1) / BINS_PER_UNIT);
                mine.x += up[i];
                mine.y += dn[i];
            }
            float2 run = scan2(mine);
            if (tid == 0) sh.first[0] = sh.first[1] = TAIL;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < BINS_PER_THREAD; ++i) {
                run.x += up[i];
                run.y += dn[i];
                if (run.x >= static_cast<float>(goal) * (1.f - 1e-4f)) atomicMin(&sh.first[0], tid * BINS_PER_THREAD + i);
                if (run.y >= static_cast<float>(goal) * (1.f + 1e-4f)) atomicMin(&sh.first[1], tid * BINS_PER_THREAD + i);
            }
            __syncthreads();
            const int b_lo = sh.first[0], b_hi = sh.first[1];
            __syncthreads();
            if (b_lo < TAIL) {
                uint32_t n = 0;
                for (int b = b_lo + lane; b <= b_hi; b += 32) n += kept_in(b);
                n = __reduce_add_sync(0xffffffffu, n);
                select(true, true, b_lo, b_hi, n, goal);
            }
        }
    }

    // ---- the race
    __syncthreads();                                      // min_x
    const float min_x = fmaxf(sh.min_x, M - RACE_Z * T);
    uint64_t seed = a.seed, offset = a.offset;
    if (a.seed_offset) {
        seed = __ldg(a.seed_offset);
        offset = __ldg(a.seed_offset + 1);
    }
    const uint64_t rr = static_cast<uint64_t>(row) + offset;
    const PhiloxRow prow = philox_row(static_cast<uint32_t>(rr), static_cast<uint32_t>(rr >> 32), static_cast<uint32_t>(seed),
                                      static_cast<uint32_t>(seed >> 32));
    const RoundKeys unused = {};
    auto in_race = [&](float x, int col) { return x >= min_x && composite(x, col) >= keep; };
    auto race = [&](auto f) {                             // f(column, logit, noise word) for every token in the race
        for (int qd = q0 + tid; qd < q1; qd += THREADS) {
            const float4 v = kResident ? reinterpret_cast<const float4*>(slice)[qd - q0] : load_quad(qd);
            const float l[4] = {v.x, v.y, v.z, v.w};
            bool in[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) in[e] = in_race(l[e], 4 * qd + e);
            if (!(in[0] || in[1] || in[2] || in[3])) continue;
            const uint4 w = philox_row_at<false>(static_cast<uint32_t>(qd), prow, unused);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (in[e]) f(4 * qd + e, l[e], ws[e]);
        }
    };
    auto key32 = [&](float x, uint32_t noise) {
        // e = -ln u from the exact w = 1 - u where u is near 1, from the hardware logarithm elsewhere
        const float w = one_minus_u_of(noise);
        const float e = w < 0.015625f ? w * fmaf(w, fmaf(w, fmaf(w, 0.25f, 0.333333343f), 0.5f), 1.0f)
                                      : -__logf(__uint2float_rn(2u * (noise >> 9) + 1u) * 5.9604644775390625e-08f);
        return -depth(x) - __logf(e);
    };
    float best = -INFINITY, second = -INFINITY;
    int col_of = -1;
    auto take = [&](float kb, int cb, float k2) {         // merge another (best, column, second best)
        if (cb < 0) return;
        if (col_of < 0 || kb > best || (kb == best && cb < col_of)) {
            second = fmaxf(fmaxf(best, k2), second);
            best = kb;
            col_of = cb;
        } else {
            second = fmaxf(second, kb);
        }
    };
    race([&](int col, float x, uint32_t noise) { take(key32(x, noise), col, -INFINITY); });
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float ob = __shfl_xor_sync(0xffffffffu, best, off), os = __shfl_xor_sync(0xffffffffu, second, off);
        const int oc = __shfl_xor_sync(0xffffffffu, col_of, off);
        take(ob, oc, os);
    }
    if (lane == 0) { sh.wbest[warp] = best; sh.wsecond[warp] = second; sh.wcol[warp] = col_of; }
    __syncthreads();
    if (tid < CLUSTER) {
        best = second = -INFINITY;
        col_of = -1;
        for (int w = 0; w < WARPS; ++w) take(sh.wbest[w], sh.wcol[w], sh.wsecond[w]);
        *cluster.map_shared_rank(&sh.win[rank], tid) = make_float2(best, second);
        *cluster.map_shared_rank(&sh.win_col[rank], tid) = col_of;
    }
    cluster.sync();
    best = second = -INFINITY;
    col_of = -1;
    for (int r = 0; r < CLUSTER; ++r) take(sh.win[r].x, sh.win_col[r], sh.win[r].y);
    if (best - second > NEAR) {
        if (rank == 0 && tid == 0) a.out_ids[row] = static_cast<int64_t>(col_of);
        return;
    }
    // ---- too near in fp32: the same keys in fp64, as an order-preserving integer and the column
    double kd = 0.0;
    int cd = -1;
    const float bar = best - NEAR;
    race([&](int col, float x, uint32_t noise) {
        if (key32(x, noise) < bar) return;
        const double e = -log1p(-static_cast<double>(one_minus_u_of(noise)));
        const double key = (static_cast<double>(x) - static_cast<double>(M)) / static_cast<double>(T) - log(e);
        if (cd < 0 || key > kd) { kd = key; cd = col; }   // columns come in rising order
    });
    uint64_t none = ~0ull, top = 0ull;
    if (cd >= 0) {
        const uint64_t b = static_cast<uint64_t>(__double_as_longlong(kd));
        top = (b >> 63) ? ~b : b | 0x8000000000000000ull;
    }
    const uint64_t mine = top;
    cluster_range(none, top);
    uint64_t col_min = (cd >= 0 && mine == top) ? static_cast<uint64_t>(cd) : ~0ull, zero = 0ull;
    cluster_range(col_min, zero);
    if (rank == 0 && tid == 0) a.out_ids[row] = static_cast<int64_t>(col_min);
}

size_t smem_bytes(int slice) { return (sizeof(Shared) + 15) / 16 * 16 + static_cast<size_t>(slice) * 4; }

}  // namespace

pkv_status launch_sample_filtered(const SampleFilteredArgs& a, int* err, cudaStream_t stream) {
    if (a.batch == 0) return PKV_OK;
    if (!setup_once(kSetupSampleFiltered, [] {
            return cudaFuncSetAttribute(sample_filtered_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(smem_bytes(kMaxResident))) == cudaSuccess;
        }))
        return PKV_ERR_CUDA;
    Args args;
    args.a = a;
    args.vec_ok = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.row_stride % 4 == 0;
    args.err = err;
    const int slice = ((a.vocab + 3) / 4 + CLUSTER - 1) / CLUSTER * 4;
    const dim3 grid(CLUSTER, a.batch);
    if (slice <= kMaxResident)
        sample_filtered_kernel<true><<<grid, THREADS, smem_bytes(slice), stream>>>(args);
    else
        sample_filtered_kernel<false><<<grid, THREADS, smem_bytes(0), stream>>>(args);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
