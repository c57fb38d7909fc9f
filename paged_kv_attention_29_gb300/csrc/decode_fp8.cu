// Decode attention over an 8-bit KV cache: one query token per sequence.
//
//   out[b, h] = sum_j p_j 2^ev_j v_j,   p = softmax_j(scale * 2^ek_j * (q[b, h] . k_j)),  j < L_b
//
// with e4m3 rows k_j, v_j of KV head h / G and their scale exponents ek_j, ev_j.  The step reads
// 258 bytes per (key, KV head) and is bound by HBM for every group size, provided the arithmetic
// stays out of the way: at 258 bytes for 512 G flops, fp32 arithmetic on the CUDA cores would
// already be the bound at G = 4.  So both products run on tensor cores, transposed so that the
// key or value tile is the 16-row operand and the query heads (G of 8 columns) the narrow one:
//
//   S^T [16 keys x 8 heads]  += K [16 x 16 dims] Q^T          mma.m16n8k16, f16 in, fp32 sums
//   O^T [16 dims x 8 heads]  += V^T [16 x 16 keys] P^T
//
// e4m3 values are exact in f16, so the tiles are converted without a multiplication (two values
// per instruction) and the scales enter in fp32: ek on the scores, ev in the exponent of the
// weight.  The order of the 16 dims (keys) of a step is free as long as both operands agree, so a
// lane takes whole 16-byte pieces of a row.
//
// * q is bf16; a head's row times a power of two that puts its largest element in [2^14, 2^15)
//   is exact in f16 down to 2^-28 of that element (and to within 2^-39 of it below).
// * With s_j the scores in the log2 domain and m a running maximum of them, the softmax sum is
//   l = sum 2^(s_j - m) in fp32, and the weight of key j in the second product is 2^(t_j - T),
//   t_j = s_j - m + ev_j, T a reference that follows the largest t: the largest weight seen is held
//   in [2^kTopT, 2^kMarginT], near the top of f16 (65504), whatever the scales are.  Rounding to f16
//   costs 2^-11 of each term, an eighth of the output's bf16 rounding, so long as a weight is at least
//   2^-14; below, an absolute 2^-25, which is 2^-(25 + kTopT) = 2^-38 of the largest: what thousands
//   of light keys behind a heavy one add to a channel in which that one holds 0 is kept.  (With
//   the largest weight at 1, keys below 2^-25 of it were lost, though l counted them.)  A piece is
//   written as o * 2^T; where values or l's terms (up to 2^64) are so large that this may leave
//   fp32's range, relative to m + lg l + 12, which makes it an average of values and leaves the merge
//   room for its sum.  (t is taken relative to m, not s + ev, which would lose ev's bits beside a large
//   score.)
// * Both references move only when a score exceeds them by a margin (weights stay below 2^15,
//   l's terms below 2^64), found by one vote per chunk; the rescale is a rare branch.
//
// Work split: the batch's tokens in 32-token chunks, sequence after sequence, are cut into equal
// contiguous runs, one for each group of num_kv_heads warps of a persistent grid; warp h of the
// group walks its run for KV head h.  A token's rows of all heads are contiguous in the pool, so
// the warps of a group, which advance together, read whole DRAM pages between them: a head's row
// alone is 128 bytes at a stride of a token.  A run that crosses a sequence border writes a piece
// (m, l, o) for each side, and a second kernel merges each head's pieces in run order, so results
// do not depend on timing.
// Measured (8 KV heads, groups of 2): batch 64 with 512 to 4096 tokens, 320 MB, 56 us = 5.7 TB/s; 8
// contexts of 16k to 40k tokens, 461 MB, 76.5 us = 6.0 TB/s; DRAM reads 1.006 of the bytes.  Taking one
// head after the other instead of side by side: 64 and 89 us; with 256-byte L2 promotion on top: 77 and
// 109.  12 warps x 2 stages: 57 and 78.  535 instructions per chunk, 35% of issue slots.  Where the largest
// weight is held costs nothing there and, in a graph, 0.5 of 20.5 us with groups of 8 and 14 chunks to a
// run (37 sequences of 0 to 2999 tokens: 20.0 us at 2^0 with a margin of 2^8, 20.2 at 2^7, 20.3 at 2^11).
//
// Each warp owns a ring of shared-memory stages, each holding a chunk's K and V codes (TMA tiles
// with 128-byte swizzle: conflict-free 16-byte loads below) and its 2 x 32 scale bytes, all
// landing on one mbarrier.
#include <cuda_fp16.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int D = kHeadDim;
constexpr int CHUNK = 32;                    // tokens per stage
constexpr int WARPS = 8;
constexpr int STAGES = 3;                    // per warp
constexpr int THREADS = WARPS * 32;
constexpr int TILE_BYTES = CHUNK * D;        // one e4m3 tile
constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K, V
constexpr int SCALE_BYTES = 2 * CHUNK;       // a stage's K scales, V scales
constexpr int MAX_BATCH = 4096;
constexpr int KMIN = 2;                      // chunks a warp takes at least, where the batch allows it
constexpr float kTopT = 13.f;                // log2 of the largest weight, when its reference moves
constexpr float kMarginT = 15.f;             // and what moves it
constexpr float kMarginM = 64.f;             // the same of the softmax terms, which move to 0
static_assert(TILE_BYTES % 1024 == 0, "swizzled tiles start on 1 KiB");

struct Params {
    const uint16_t* q;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int max_blocks;
    int batch;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    float scale_log2;      // softmax scale * log2(e)
    int groups;            // groups of num_kv_heads warps in the grid
    int32_t* plan;         // [batch + 1] chunks before each sequence
    float* part_ml;        // [pieces][G][2]  (m, l); piece = (sequence + run) * num_kv_heads + KV head
    float* part_o;         // [pieces][G][D]
    int* err;
};

// Runs the `total` chunks are cut into: one for each group, unless that left fewer than KMIN chunks to a run.
__device__ __forceinline__ int runs_of(int groups, int total) {
    return max(1, min(groups, (total + KMIN - 1) / KMIN));
}

// First chunk of run r.
__device__ __forceinline__ int run_begin(int r, int total, int runs) {
    return static_cast<int>(static_cast<uint64_t>(r) * static_cast<uint32_t>(total) / static_cast<uint32_t>(runs));
}

struct Cursor {
    int b, c, n;      // sequence, chunk within it, chunks of the sequence
};

__device__ __forceinline__ Cursor cursor_at(const int32_t* prefix, int batch, int i) {
    int lo = 0, hi = batch;          // prefix[lo] <= i < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= i) lo = mid; else hi = mid;
    }
    return Cursor{lo, i - prefix[lo], prefix[lo + 1] - prefix[lo]};
}

__device__ __forceinline__ void cursor_next(Cursor& cu, const int32_t* prefix, int batch) {
    if (++cu.c < cu.n) return;
    cu.c = 0;
    do { ++cu.b; } while (cu.b < batch && prefix[cu.b + 1] == prefix[cu.b]);
    cu.n = cu.b < batch ? prefix[cu.b + 1] - prefix[cu.b] : 0;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// The raw query words of this lane: head g = lane / 4 of the group, dims 32 (lane % 4) ... + 31.
template <int G>
__device__ __forceinline__ void load_q(const Params& p, int b, int kv_head, int lane, uint4 (&w)[4]) {
    const int h = lane >> 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
    if (h < G) {
        const uint16_t* row = p.q + (static_cast<int64_t>(b) * p.num_kv_heads + kv_head) * (G * D) + h * D + 32 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(row) + i);
    }
}

// The query operand in f16 and, for the two heads 2t, 2t + 1 of this lane's columns, the factor
// that turns a raw product into log2-domain scores.
__device__ __forceinline__ void make_q(const uint4 (&w)[4], float scale_log2, int lane, uint32_t (&qb)[16], float (&qf)[2]) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max(amax, max((x[e] << 16) & 0x7fffffffu, x[e] & 0x7fff0000u));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // E: biased exponent of the row's largest magnitude, held where the factors stay normal (a row
    // that is smaller than 2^-111 gives scores of 0 against any cache)
    const int E = max(static_cast<int>(amax >> 23), 16);
    const float mul = E == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(268 - min(E, 254)) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) qb[4 * i + e] = pack_f16x2(bf16_lo(x[e]) * mul, bf16_hi(x[e]) * mul);
    }
    const float f = E == 255 ? mul : __uint_as_float(static_cast<uint32_t>(E - 14) << 23) * scale_log2;
    qf[0] = __shfl_sync(0xffffffffu, f, (lane & 3) * 8);        // head 2t sits in lanes 8t .. 8t + 3
    qf[1] = __shfl_sync(0xffffffffu, f, (lane & 3) * 8 + 4);
}

template <int G>
__global__ void __launch_bounds__(THREADS, 1)
decode_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* scales = smem + WARPS * STAGES * STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(scales + WARPS * STAGES * SCALE_BYTES);
    int32_t* tsum = reinterpret_cast<int32_t*>(bars + WARPS * STAGES);
    int32_t* prefix = tsum + THREADS;

    const int tid = threadIdx.x;
    const int lane = tid & 31;
    const int warp = tid >> 5;
    const int hkv = p.num_kv_heads;
    const int cap = p.max_blocks * p.block_size;
    auto length_of = [&](int b) { return min(max(__ldg(p.context_lens + b), 0), cap); };

    // ---- chunks of each sequence and their running sum (every CTA computes the same)
    const int per = (p.batch + THREADS - 1) / THREADS;
    const int b0 = tid * per, b1 = min(p.batch, b0 + per);
    int local = 0;
    for (int b = b0; b < b1; ++b) {
        const int L = __ldg(p.context_lens + b);
        if ((L < 0 || L > cap) && blockIdx.x == 0) record_error(p.err, PKV_DEVERR_SEQLENS, b);
        local += (length_of(b) + CHUNK - 1) / CHUNK;
    }
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) tsum[warp] = incl;
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += tsum[w];
    for (int b = b0; b < b1; ++b) {
        prefix[b] = run;
        run += (length_of(b) + CHUNK - 1) / CHUNK;
    }
    if (tid == THREADS - 1) prefix[p.batch] = run;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = tid; b <= p.batch; b += THREADS) p.plan[b] = prefix[b];

    // ---- this warp's run of chunks and KV head
    const int gw = blockIdx.x * WARPS + warp;
    const int run_id = gw / hkv, head = gw - run_id * hkv;
    const int total = prefix[p.batch];
    const int W = runs_of(p.groups, total);
    if (run_id >= W) return;
    const int begin = run_begin(run_id, total, W);
    const int n_mine = run_begin(run_id + 1, total, W) - begin;
    if (n_mine <= 0) return;

    const uint32_t stage0 = smem_u32(smem) + warp * STAGES * STAGE_BYTES;
    const uint32_t scale0 = smem_u32(scales) + warp * STAGES * SCALE_BYTES;
    const uint32_t bar0 = smem_u32(bars + warp * STAGES);
    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
    const uint64_t policy = l2_policy_evict_first();

    // ---- copies: a cursor of their own, the block it is in, and a window of 32 block-table entries
    Cursor pc = cursor_at(prefix, p.batch, begin);
    Cursor cc = pc;
    int blk = pc.c * CHUNK / p.block_size, off = pc.c * CHUNK - blk * p.block_size;
    int bt_b = -1, bt_base = 0, bt_lane = -1;
    int issued = 0, put = 0;         // chunks issued; the stage the next one goes to
    auto issue_next = [&]() {
        if (pc.b != bt_b || blk < bt_base || blk >= bt_base + 32) {
            bt_b = pc.b;
            bt_base = blk;
            const int at = bt_base + lane;
            bt_lane = at < p.max_blocks ? __ldg(p.block_tables + static_cast<int64_t>(pc.b) * p.max_blocks + at) : -1;
        }
        const int phys = __shfl_sync(0xffffffffu, bt_lane, blk - bt_base);
        if (lane == 0) {
            const bool known = phys >= 0 && phys < p.num_blocks;
            if (!known) record_error(p.err, PKV_DEVERR_BLOCK_ID, pc.b);
            const uint32_t bar = bar0 + 8 * put;
            const uint32_t dst = stage0 + put * STAGE_BYTES, sdst = scale0 + put * SCALE_BYTES;
            // the tensor copies fill a block outside the pool with zeros; its scales come from block 0
            const int64_t srow = (static_cast<int64_t>(known ? phys : 0) * hkv + head) * p.block_size + off;
            mbar_arrive_expect_tx(bar, STAGE_BYTES + SCALE_BYTES);
            tma_load_4d_hint(dst, &tm_k, bar, 0, head, off, phys, policy);
            tma_load_4d_hint(dst + TILE_BYTES, &tm_v, bar, 0, head, off, phys, policy);
            bulk_load(sdst, p.k_scale + srow, CHUNK, bar);
            bulk_load(sdst + CHUNK, p.v_scale + srow, CHUNK, bar);
        }
        ++issued;
        put = put + 1 == STAGES ? 0 : put + 1;
        off += CHUNK;
        if (off == p.block_size) { off = 0; ++blk; }
        cursor_next(pc, prefix, p.batch);
        if (pc.c == 0) blk = off = 0;
    };
    for (int i = 0; i < min(n_mine, STAGES); ++i) issue_next();

    const int g = lane >> 2, t = lane & 3;
    // swizzled 16-byte pieces: K row r (r % 8 = g): pieces 2t, 2t + 1; V row r: piece g
    const uint32_t k_piece0 = static_cast<uint32_t>(((2 * t) ^ g) << 4), k_piece1 = static_cast<uint32_t>(((2 * t + 1) ^ g) << 4);
    uint32_t qb[16];
    float qf[2];
    uint4 qw[4];
    load_q<G>(p, cc.b, head, lane, qw);
    make_q(qw, p.scale_log2, lane, qb, qf);
    int L = length_of(cc.b);
    // the next segment's query rows and length, loaded while this one streams
    int L_next = 0;
    auto prefetch_next = [&](int done) {
        if (n_mine - done <= cc.n - cc.c) return;
        Cursor nx = cc;
        nx.c = nx.n - 1;
        cursor_next(nx, prefix, p.batch);
        load_q<G>(p, nx.b, head, lane, qw);
        L_next = length_of(nx.b);
    };
    prefetch_next(0);

    float o[8][4];
    float m[2], T[2], l[2];
    bool fresh = true;               // no chunk of this segment seen yet
    auto reset = [&]() {
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[u][e] = 0.f;
        m[0] = m[1] = T[0] = T[1] = l[0] = l[1] = 0.f;
        fresh = true;
    };
    reset();

    int k = 0, st = 0;               // chunk of the run; its stage
    uint32_t parity = 0;
    bool failed = false;
    for (; k < n_mine; ++k) {
        const bool ok = mbar_wait(bar0 + 8 * st, parity, p.err, gw);
        if (__any_sync(0xffffffffu, !ok)) { failed = true; break; }
        const uint32_t kb = stage0 + st * STAGE_BYTES, vb = kb + TILE_BYTES;
        const uint32_t sb = scale0 + st * SCALE_BYTES;
        if (++st == STAGES) { st = 0; parity ^= 1u; }
        const int valid = min(CHUNK, L - cc.c * CHUNK);
        if (valid < CHUNK) {
            // slots past the sequence's end may hold anything (a freed block is not cleared); their
            // weight is 0 but 0 * NaN is NaN, so their V codes are cleared
            for (int i = lane; i < (CHUNK - valid) * 8; i += 32)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + valid * D + i * 16), "r"(0) : "memory");
            __syncwarp();
        }
        // this lane's key's scales (key = lane), as a factor and an exponent
        const float kf_lane = e8m0_value(ld_shared_u8(sb + lane)), ev_lane = e8m0_exponent(ld_shared_u8(sb + CHUNK + lane));
        // ---- scores: S^T = K Q^T, 16 keys per tile; step e takes dims 32t + 4e .. + 3 of this lane's piece
        float c[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
            const uint32_t row0 = kb + (16 * i + g) * D, row1 = row0 + 8 * D;
            const uint4 x0 = ld_shared_v4(row0 + k_piece0), x1 = ld_shared_v4(row0 + k_piece1);
            const uint4 y0 = ld_shared_v4(row1 + k_piece0), y1 = ld_shared_v4(row1 + k_piece1);
            const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            const uint32_t y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t a0, a1, a2, a3;
                f16_of_codes(x[e], a0, a2);
                f16_of_codes(y[e], a1, a3);
                mma_f16(c[i], a0, a1, a2, a3, qb[2 * e], qb[2 * e + 1]);
            }
        }
        // ---- log2-domain scores relative to m; this lane: keys g + 8 r, heads 2t, 2t + 1
        float d[4][2], w[4][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float kf = __shfl_sync(0xffffffffu, kf_lane, g + 8 * r);
#pragma unroll
            for (int h = 0; h < 2; ++h) d[r][h] = fmaf(c[r >> 1][(r & 1) * 2 + h] * qf[h], kf, -m[h]);
        }
        if (valid < CHUNK) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (g + 8 * r >= valid) d[r][0] = d[r][1] = -INFINITY;
        }
        const float d_max = fmax3(fmax3(d[0][0], d[0][1], d[1][0]), fmax3(d[1][1], d[2][0], d[2][1]), fmaxf(d[3][0], d[3][1]));
        if (__any_sync(0xffffffffu, fresh || d_max > kMarginM)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float up = fmaxf(fmaxf(d[0][h], d[1][h]), fmaxf(d[2][h], d[3][h]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, x));
                if (!fresh) up = fmaxf(up, 0.f);
                if (!(fabsf(up) < INFINITY)) up = 0.f;   // no finite score: any reference does
                m[h] += up;
                l[h] *= fresh ? 1.f : ex2_ftz(-up);      // a fresh l is 0, and up may be any score
                // o keeps its units; below 2^-256 it is nothing beside the new maximum's weight (>= 2^-126), and a
                // larger T would cost the next weights their low bits
                T[h] = fresh ? 0.f : fmaxf(T[h] - up, -256.f);
#pragma unroll
                for (int r = 0; r < 4; ++r) d[r][h] -= up;
            }
        }
        // ---- exponents of the weights over their reference: s - m + ev - T
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float ev = __shfl_sync(0xffffffffu, ev_lane, g + 8 * r);
#pragma unroll
            for (int h = 0; h < 2; ++h) w[r][h] = (d[r][h] + ev) - T[h];
        }
        if (valid < CHUNK) {                             // whatever scale a slot past the end has
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (g + 8 * r >= valid) w[r][0] = w[r][1] = -INFINITY;
        }
        const float w_max = fmax3(fmax3(w[0][0], w[0][1], w[1][0]), fmax3(w[1][1], w[2][0], w[2][1]), fmaxf(w[3][0], w[3][1]));
        if (__any_sync(0xffffffffu, fresh || w_max > kMarginT)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float up = fmaxf(fmaxf(w[0][h], w[1][h]), fmaxf(w[2][h], w[3][h]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, x));
                up -= kTopT;
                if (!fresh) up = fmaxf(up, 0.f);
                if (!(fabsf(up) < INFINITY)) up = 0.f;
                T[h] += up;
                const float f = fresh ? 1.f : ex2_ftz(-up);          // a fresh o is 0
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r][h] -= up;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    o[u][h] *= f;
                    o[u][2 + h] *= f;
                }
            }
        }
        fresh = false;
        uint32_t pb[4];               // P^T operand: key pairs of this lane's head g
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            l[0] += ex2_ftz(d[r][0]);
            l[1] += ex2_ftz(d[r][1]);
            pb[r] = transposed_8x8(pack_f16x2(ex2_ftz(w[r][0]), ex2_ftz(w[r][1])));
        }
        // ---- O^T += V^T P^T, 16 keys per step; row g of tile u: dim 16g + 2u, row g + 8: dim 16g + 2u + 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ka = 16 * i + 2 * t;            // keys ka, ka + 1, ka + 8, ka + 9
            const uint32_t ra = vb + ka * D, sa = static_cast<uint32_t>((g ^ (2 * t)) << 4), sd = static_cast<uint32_t>((g ^ (2 * t + 1)) << 4);
            const uint4 va = ld_shared_v4(ra + sa), vd = ld_shared_v4(ra + D + sd);
            const uint4 ve = ld_shared_v4(ra + 8 * D + sa), vf = ld_shared_v4(ra + 9 * D + sd);
            const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wd[4] = {vd.x, vd.y, vd.z, vd.w};
            const uint32_t we[4] = {ve.x, ve.y, ve.z, ve.w}, wf[4] = {vf.x, vf.y, vf.z, vf.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3;
                f16_of_codes(__byte_perm(wa[w], wd[w], 0x5140), a0, a1);
                f16_of_codes(__byte_perm(we[w], wf[w], 0x5140), a2, a3);
                mma_f16(o[2 * w], a0, a1, a2, a3, pb[2 * i], pb[2 * i + 1]);
                f16_of_codes(__byte_perm(wa[w], wd[w], 0x7362), a0, a1);
                f16_of_codes(__byte_perm(we[w], wf[w], 0x7362), a2, a3);
                mma_f16(o[2 * w + 1], a0, a1, a2, a3, pb[2 * i], pb[2 * i + 1]);
            }
        }
        if (valid < CHUNK) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the cleared rows, before the stage's next copy
        __syncwarp();
        if (issued < n_mine) issue_next();

        // ---- end of the sequence or of the run: write the piece
        if (cc.c == cc.n - 1 || k == n_mine - 1) {
            const int64_t piece = static_cast<int64_t>(cc.b + run_id) * hkv + head;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
                const int hq = 2 * t + h;                      // query head of the group
                if (hq < G) {
                    // |o| is below 2^48 (weights, codes, keys); 2^(T - e) may be out of range where its product with o is not
                    const float e = T[h] > 64.f && l[h] < INFINITY ? static_cast<float>(static_cast<int>(__float_as_uint(l[h]) >> 23) - 115) : 0.f;
                    const float f = ex2_ftz(0.5f * (T[h] - e));
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (piece * G + hq) * D + 16 * g);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        dst[u] = make_float4(o[2 * u][h] * f * f, o[2 * u][2 + h] * f * f, o[2 * u + 1][h] * f * f,
                                             o[2 * u + 1][2 + h] * f * f);
                    if (g == 0) {
                        p.part_ml[(piece * G + hq) * 2] = m[h] + e;
                        p.part_ml[(piece * G + hq) * 2 + 1] = l[h] * ex2_ftz(-e);
                    }
                }
            }
            if (k != n_mine - 1) {
                cursor_next(cc, prefix, p.batch);
                make_q(qw, p.scale_log2, lane, qb, qf);
                L = L_next;
                prefetch_next(k + 1);
                reset();
            }
        } else {
            ++cc.c;
        }
    }
    if (failed)       // copies in flight land before the CTA's shared memory goes away
        for (; k < issued; ++k) {
            const bool ok = mbar_wait(bar0 + 8 * st, parity, p.err, gw);
            if (++st == STAGES) { st = 0; parity ^= 1u; }
            if (__any_sync(0xffffffffu, !ok)) break;
        }
}

// Merge the pieces of each (sequence, query head): SPLIT warps take every SPLIT-th piece in run order
// each, and their sums are added in warp order.
template <int G, int SPLIT>
__global__ void __launch_bounds__(128) decode_fp8_combine_kernel(const Params p, int num_heads, uint16_t* __restrict__ out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float4 part[4][32];
    __shared__ float2 part_ml[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int idx = blockIdx.x * (4 / SPLIT) + warp / SPLIT, sub = warp % SPLIT;
    if (idx >= p.batch * num_heads) return;               // whole CTAs only if SPLIT > 1
    const int b = idx / num_heads;
    const int h = idx - b * num_heads;
    const int g = h / G, hh = h - g * G;
    const int hkv = p.num_kv_heads;
    const int first = p.plan[b], n = p.plan[b + 1] - first, all = p.plan[p.batch];
    uint2* dst = reinterpret_cast<uint2*>(out + static_cast<int64_t>(idx) * D + 4 * lane);
    if (n == 0) {
        if (sub == 0) *dst = make_uint2(0u, 0u);
        return;
    }
    const int W = runs_of(p.groups, all);
    // the run that holds chunk i is floor(((i + 1) W - 1) / all); W <= all, so every run holds a chunk
    auto run_of = [&](int i) {
        return static_cast<int>((static_cast<uint64_t>(i + 1) * static_cast<uint32_t>(W) - 1) / static_cast<uint32_t>(all));
    };
    const int wf = run_of(first), wl = run_of(first + n - 1);
    constexpr int BATCH = 4;        // pieces whose loads are issued together
    float M = -INFINITY, L = 0.f;   // sums relative to the running maximum
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w0 = wf + sub; w0 <= wl; w0 += BATCH * SPLIT) {
        float2 ml[BATCH];
        float4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (w0 + i * SPLIT <= wl) {
                const int64_t at = (static_cast<int64_t>(b + w0 + i * SPLIT) * hkv + g) * G + hh;
                ml[i] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
                v[i] = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * lane);
            } else {
                ml[i] = make_float2(-INFINITY, 0.f);
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        const float m_new = fmax3(M, fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));   // finite: a piece's m is
        const float keep = ex2_ftz(M - m_new);
        L *= keep;
        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
        M = m_new;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const float f = exp2f(ml[i].x - M);
            L = fmaf(f, ml[i].y, L);
            acc.x = fmaf(f, v[i].x, acc.x);
            acc.y = fmaf(f, v[i].y, acc.y);
            acc.z = fmaf(f, v[i].z, acc.z);
            acc.w = fmaf(f, v[i].w, acc.w);
        }
    }
    if (SPLIT > 1) {
        part[warp][lane] = acc;
        if (lane == 0) part_ml[warp] = make_float2(M, L);
        __syncthreads();
        if (sub != 0) return;
        float m_all = M;
#pragma unroll
        for (int i = 1; i < SPLIT; ++i) m_all = fmaxf(m_all, part_ml[warp + i].x);
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < SPLIT; ++i) {
            const float2 ml = part_ml[warp + i];
            const float4 v = part[warp + i][lane];
            const float f = exp2f(ml.x - m_all);          // 0 for a warp without a piece
            L = fmaf(f, ml.y, L);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
    }
    const float inv = 1.f / L;
    *dst = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

size_t dynamic_smem_bytes(int batch) {
    return 1024 + WARPS * STAGES * (STAGE_BYTES + SCALE_BYTES + 8) + THREADS * 4 + static_cast<size_t>(batch + 1) * 4;
}

constexpr size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int G>
bool set_smem_attr(int bytes) {
    return cudaFuncSetAttribute(decode_fp8_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

template <int G>
pkv_status launch_pair(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p, int num_heads, uint16_t* out,
                       int sms, cudaStream_t stream) {
    // both launches are programmatic dependents of what precedes them in the stream; each kernel waits
    // for its predecessor's completion before touching global memory
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = dynamic_smem_bytes(p.batch);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, decode_fp8_kernel<G>, tm_k, tm_v, p) != cudaSuccess) return PKV_ERR_CUDA;
    // a sequence is cut into about groups / batch pieces: with four or more, four warps share a head's merge
    const bool split = p.groups >= 4 * p.batch;
    cfg.gridDim = dim3(split ? p.batch * num_heads : (p.batch * num_heads + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    const cudaError_t e = split ? cudaLaunchKernelEx(&cfg, decode_fp8_combine_kernel<G, 4>, p, num_heads, out)
                                : cudaLaunchKernelEx(&cfg, decode_fp8_combine_kernel<G, 1>, p, num_heads, out);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

size_t decode_fp8_workspace_bytes(int batch, int num_kv_heads, int log_group) {
    const size_t G = static_cast<size_t>(1) << log_group;
    const size_t pieces = static_cast<size_t>(batch) * num_kv_heads + static_cast<size_t>(sm_count()) * WARPS;
    return align256(static_cast<size_t>(batch + 1) * 4) + align256(pieces * G * 2 * 4) + align256(pieces * G * D * 4);
}

pkv_status launch_decode_fp8(const DecodeFp8Args& a, int* err, cudaStream_t stream) {
    if (a.batch > MAX_BATCH) return PKV_ERR_UNSUPPORTED;
    const int lg = group_log2(a.num_heads, a.num_kv_heads);
    if (lg < 0) return PKV_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    if (a.workspace == nullptr || a.workspace_bytes < decode_fp8_workspace_bytes(a.batch, a.num_kv_heads, lg))
        return PKV_ERR_WORKSPACE;
    if (a.batch == 0) return PKV_OK;
    // the chunks of a batch are counted in 32 bits
    if (static_cast<int64_t>(a.batch) * ((static_cast<int64_t>(a.max_blocks) * a.block_size + CHUNK - 1) / CHUNK) > 0x7fffffffLL)
        return PKV_ERR_UNSUPPORTED;

    CUtensorMap tm_k, tm_v;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.num_kv_heads),
                              static_cast<uint64_t>(a.block_size), static_cast<uint64_t>(a.num_blocks)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.num_kv_heads) * D,
                                 static_cast<uint64_t>(a.block_size) * a.num_kv_heads * D};
    const uint32_t box[4] = {static_cast<uint32_t>(D), 1u, static_cast<uint32_t>(CHUNK), 1u};
    if (encode_tiled(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(a.k_cache), dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) != CUDA_SUCCESS ||
        encode_tiled(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(a.v_cache), dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) != CUDA_SUCCESS)
        return PKV_ERR_INVALID_ARG;

    if (!setup_once(kSetupDecodeFp8, [] {
            const int bytes = static_cast<int>(dynamic_smem_bytes(MAX_BATCH));
            return set_smem_attr<1>(bytes) && set_smem_attr<2>(bytes) && set_smem_attr<4>(bytes) && set_smem_attr<8>(bytes);
        }))
        return PKV_ERR_CUDA;

    const size_t G = static_cast<size_t>(1) << lg;
    Params p;
    p.q = a.q;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.max_blocks = a.max_blocks;
    p.batch = a.batch;
    p.num_kv_heads = a.num_kv_heads;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
    p.groups = sms * WARPS / a.num_kv_heads;
    if (p.groups < 1) return PKV_ERR_UNSUPPORTED;
    const size_t pieces = static_cast<size_t>(a.batch + p.groups) * a.num_kv_heads;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.plan = reinterpret_cast<int32_t*>(ws);
    ws += align256(static_cast<size_t>(a.batch + 1) * 4);
    p.part_ml = reinterpret_cast<float*>(ws);
    ws += align256(pieces * G * 2 * 4);
    p.part_o = reinterpret_cast<float*>(ws);
    p.err = err;
    switch (lg) {
        case 0: return launch_pair<1>(tm_k, tm_v, p, a.num_heads, a.out, sms, stream);
        case 1: return launch_pair<2>(tm_k, tm_v, p, a.num_heads, a.out, sms, stream);
        case 2: return launch_pair<4>(tm_k, tm_v, p, a.num_heads, a.out, sms, stream);
        default: return launch_pair<8>(tm_k, tm_v, p, a.num_heads, a.out, sms, stream);
    }
}

}  // namespace pkv
