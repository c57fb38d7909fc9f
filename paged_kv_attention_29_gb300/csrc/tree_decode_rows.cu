// Attention of small trees of drafted tokens over an 8-bit KV cache: no more than 16
// rows (nodes x query heads of a KV head) to a sequence.
//
// For sequence b with n_b nodes, the last of its L_b keys, and KV head g, row r (node r / G,
// query head G g + r % G):
//
//   out_r = sum_j p_j 2^ev_j v_j,   p = softmax_j(scale 2^ek_j q_r . k_j)
//
// over the keys before the tree and the nodes that the node's mask names.  A key costs 258
// bytes and 512 flops a row, so the step is bound by HBM if the codes are turned into
// operands cheaply.  Both products run transposed on mma.m16n8k16 with the key or value tile
// as the 16-row operand,
//
//   S^T [16 keys x 8 rows] += K [16 x 16 dims] Q^T
//   O^T [16 dims x 8 rows] += V^T [16 x 16 keys] P^T
//
// so that codes become f16 (exactly, two to an instruction) once for all NT = 1 or 2 groups
// of 8 rows, in the registers of the warp that uses them.
//
// Why 16 rows, measured at batch 64 with 512 to 4096 keys (8 KV heads): 8 rows 57 us, 16 rows
// 73, against 101 on tcgen05 (tree_decode.cu) whatever the rows up to 32; 32 rows took 132 here, as
// one warp with 255 registers or as two that share a stage: two or three warps a scheduler
// do not hide the latencies of some 700 to 1100 instructions a chunk.
//
// Numbers as in the single-token kernel: a query row times a power of two is exact in f16
// down to 2^-28 of its largest element; scores, their maximum m and the sum l are fp32; the
// weight of a key in the second product is f16 of 2^(s - m + ev - T), T following the largest
// of these exponents so that it is held between 2^kTopT and 2^kMarginT; both references move
// only past a margin, each row's by what that row sees (the warp votes to look, no more).  A
// row's references are set by the first key it sees.
//
// Work split: the sequences' 32-key chunks, one after the other, are cut into equal runs, one
// for each group of num_kv_heads warps; warp h of a group walks its run for KV head h (a
// token's rows of all heads lie side by side).  A sequence that a run holds whole is written
// at once; of others each run leaves (m, l, O), and a second kernel joins them in the order of
// the runs.  Results do not depend on timing.
//
// Each warp owns a ring of stages in shared memory: a chunk's K and V codes (TMA, 128-byte
// swizzle) and scale bytes, all landing on one mbarrier.
#include <algorithm>

#include "fp8_rows.cuh"

namespace pkv {
namespace {

using namespace fp8_rows;

// shared memory: stages, then scales, a barrier for each stage, the running sums
constexpr int SM_SCALES = WARPS * STAGES * STAGE_BYTES, SM_BARS = SM_SCALES + WARPS * STAGES * SCALE_BYTES, SM_SUMS = SM_BARS + WARPS * STAGES * 8;
constexpr size_t smem_bytes(int batch) { return SM_SUMS + WARPS * 4 + static_cast<size_t>(batch + 1) * 4; }

struct Params {
    const uint16_t* q;
    const uint8_t* v_codes;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_nodes;
    const unsigned long long* mask;
    uint16_t* out;
    float2* part_ml;       // [run][KV head][2][rows]  (m, l): of the sequence a run goes on with, and of the one it leaves open
    float* part_o;         // [run][KV head][2][rows][D]
    int4* meta;            // [run][KV head]: last run of the sequence left open or -1, its first node's row, its rows
    int max_blocks, batch, num_heads, num_kv_heads, lg, block_size, num_blocks;
    int max_nodes, max_context, mask_words, total_nodes;
    int groups;            // groups of num_kv_heads warps in the grid
    float scale_log2;
    int* err;
};

struct Seq {
    int q0, n, len;
};
__device__ __forceinline__ bool sequence(const Params& p, int b, Seq& s) {
    s.q0 = __ldg(p.cu_nodes + b);
    const int q1 = __ldg(p.cu_nodes + b + 1);
    s.len = __ldg(p.context_lens + b);
    const long long n = static_cast<long long>(q1) - s.q0;
    const bool fits = s.q0 >= 0 && n > 0 && q1 <= p.total_nodes && n <= p.max_nodes && n <= s.len && s.len <= p.max_context &&
                      s.len <= static_cast<long long>(p.max_blocks) * p.block_size;
    s.n = fits ? static_cast<int>(n) : 0;
    return n == 0 || fits;
}
__device__ __forceinline__ int chunks_of(const Seq& s) { return s.n ? (s.len + CHUNK - 1) / CHUNK : 0; }

__device__ __forceinline__ int runs_of(int groups, int total) { return max(1, min(groups, total / KMIN)); }
// Which of a chunk's 32 keys a row sees: w, its node's mask (no tree here has more than 16 nodes; all ones for a row that is
// nobody's); `first` is the node of the chunk's first key (negative before the tree, above -32), `keys` the sequence's
// keys in the chunk.
__device__ __forceinline__ uint32_t visible(uint32_t w, int first, int keys) {
    const uint32_t m = first < 0 ? (w << -first) | ((1u << -first) - 1u) : w >> first;
    return keys >= CHUNK ? m : m & ((1u << keys) - 1u);
}

__device__ __forceinline__ bool nan_codes(uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u; }

// NT groups of 8 rows
template <int NT>
__global__ void __launch_bounds__(THREADS, 1)
tree_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
    constexpr int ROWS = 8 * NT;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) uint8_t smem[];
    int32_t* tsum = reinterpret_cast<int32_t*>(smem + SM_SUMS);
    int32_t* prefix = tsum + WARPS;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hkv = p.num_kv_heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- chunks of each sequence and their running sum (every CTA computes the same)
    const int per = (p.batch + THREADS - 1) / THREADS;
    const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
    int local = 0;
    for (int b = b0; b < b1; ++b) {
        Seq s;
        if (!sequence(p, b, s) && blockIdx.x == 0) record_error(p.err, PKV_DEVERR_SEQLENS, b);
        local += chunks_of(s);
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
        Seq s;
        sequence(p, b, s);
        prefix[b] = run;
        run += chunks_of(s);
    }
    if (tid == THREADS - 1) prefix[p.batch] = run;
    __syncthreads();

    // ---- this warp's run of chunks and KV head
    const int gw = blockIdx.x * WARPS + warp;
    const int run_id = gw / hkv, head = gw - run_id * hkv;
    if (run_id >= p.groups) return;
    const int total = prefix[p.batch];
    const int W = runs_of(p.groups, total);
    const int begin = run_id < W ? run_begin(run_id, total, W) : 0;
    const int n_mine = run_id < W ? run_begin(run_id + 1, total, W) - begin : 0;
    int4 meta = make_int4(-1, 0, 0, 0);
    if (n_mine <= 0) {
        if (lane == 0) p.meta[gw] = meta;
        return;
    }
    const Ring ring{smem_u32(smem) + warp * STAGES * STAGE_BYTES, smem_u32(smem + SM_SCALES) + warp * STAGES * SCALE_BYTES,
                    smem_u32(smem + SM_BARS) + warp * STAGES * 8};
    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(ring.bar0 + 8 * s, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
    const uint64_t policy = l2_policy_evict_first();

    Cursor cc = cursor_at(prefix, p.batch, begin);
    Copies copies(cc, p.block_size);
    auto issue_next = [&]() { copies.next(tm_k, tm_v, p, ring, prefix, head, lane, policy); };
    for (int i = 0; i < min(n_mine, STAGES); ++i) issue_next();

    const int g = lane >> 2, t = lane & 3;
    // swizzled 16-byte pieces: K row r (r % 8 = g): pieces 2t, 2t + 1; V row r: piece g
    const uint32_t k_piece0 = static_cast<uint32_t>(((2 * t) ^ g) << 4), k_piece1 = static_cast<uint32_t>(((2 * t + 1) ^ g) << 4);
    uint32_t qb[NT][16];
    float qf[NT][2];
    uint32_t mask[NT][2];            // of the rows of this lane's columns
    Seq s;
    // The segment's query rows, f16, row 8 x + g of this lane's dims 32 t .. + 31, and for the rows 8 x + 2t and 8 x + 2t + 1
    // of its columns the mask and the factor that turns a raw product into log2-domain scores.
    auto enter = [&]() {
        sequence(p, cc.b, s);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int r = 8 * x + g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = 8 * x + 2 * t + h;
                mask[x][h] = col < s.n << p.lg ? static_cast<uint32_t>(__ldg(p.mask + static_cast<int64_t>(s.q0 + (col >> p.lg)) * p.mask_words)) : 0xffffffffu;
            }
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
            if (r < s.n << p.lg) {
                const uint16_t* row = p.q + (static_cast<int64_t>(s.q0 + (r >> p.lg)) * p.num_heads + (head << p.lg) + (r & ((1 << p.lg) - 1))) * D + 32 * t;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(row) + i);
            }
            make_q(w, p.scale_log2, lane, qb[x], qf[x]);
        }
    };
    enter();
    int seg_begin = cc.c;            // the segment's first chunk

    float o[NT][8][4];
    float m[NT][2], T[NT][2], l[NT][2];
    uint32_t seen = 0u;              // bit 2 x + h: row 8 x + 2t + h has seen a key
    auto reset = [&]() {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][u][e] = 0.f;
            m[x][0] = m[x][1] = T[x][0] = T[x][1] = l[x][0] = l[x][1] = 0.f;
        }
        seen = 0u;
    };
    reset();

    int k = 0, st = 0;               // chunk of the run; its stage
    uint32_t parity = 0;
    bool failed = false;
    for (; k < n_mine; ++k) {
        const bool ok = mbar_wait(ring.bar0 + 8 * st, parity, p.err, gw);
        if (__any_sync(0xffffffffu, !ok)) { failed = true; break; }
        const uint32_t kb = ring.stage0 + st * STAGE_BYTES, vb = kb + TILE_BYTES;
        const uint32_t sb = ring.scale0 + st * SCALE_BYTES;
        if (++st == STAGES) { st = 0; parity ^= 1u; }
        const int valid = min(CHUNK, s.len - cc.c * CHUNK), first = cc.c * CHUNK - (s.len - s.n);
        const bool tree = first + CHUNK > 0;               // nodes among the keys, in the last chunks
        uint32_t hurt = 0u;                                // nodes' rows with NaN codes among V's
        if (tree) {
            // Slots past the sequence's end may hold anything (a freed block is not cleared), and a NaN code of a node's
            // row would reach the rows that do not see it through a weight of 0: both leave the tile.
            for (int r = max(0, -first) + (lane >> 3); r - (lane >> 3) < CHUNK; r += 4) {
                bool bad = false;
                if (r < CHUNK) {
                    const uint32_t at = vb + r * D + (lane & 7) * 16;
                    const uint4 c = ld_shared_v4(at);
                    bad = r < valid && (nan_codes(c.x) || nan_codes(c.y) || nan_codes(c.z) || nan_codes(c.w));
                    if (bad || r >= valid) {
                        uint32_t y[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (r >= valid || (y[e] >> (8 * i) & 0x7fu) == 0x7fu) y[e] &= ~(0xffu << (8 * i));
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
                    }
                }
                hurt |= __reduce_or_sync(0xffffffffu, bad ? 1u << r : 0u);
            }
            __syncwarp();
        }
        // this lane's key's scales (key = lane), as a factor and an exponent
        const float kf_lane = e8m0_value(ld_shared_u8(sb + lane)), ev_lane = e8m0_exponent(ld_shared_u8(sb + CHUNK + lane));
        // ---- scores: S^T = K Q^T, 16 keys per tile; step e takes dims 32t + 4e .. + 3 of this lane's piece
        float c[NT][2][4];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 2; ++i) c[x][i][0] = c[x][i][1] = c[x][i][2] = c[x][i][3] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {             // pieces 2t and 2t + 1
            uint4 a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = ld_shared_v4(kb + (8 * i + g) * D + (half ? k_piece1 : k_piece0));
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2)                 // 8 dims: q words 4 (2 half + e2) ..
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 &u = a[2 * i], &v = a[2 * i + 1];
                        const uint32_t wu = e2 ? (e ? u.w : u.z) : (e ? u.y : u.x), wv = e2 ? (e ? v.w : v.z) : (e ? v.y : v.x);
                        uint32_t a0, a1, a2, a3;
                        f16_of_codes(wu, a0, a2);
                        f16_of_codes(wv, a1, a3);
#pragma unroll
                        for (int x = 0; x < NT; ++x) mma_f16(c[x][i], a0, a1, a2, a3, qb[x][8 * half + 4 * e2 + 2 * e], qb[x][8 * half + 4 * e2 + 2 * e + 1]);
                    }
        }
        // ---- weights, 8 rows at a time; this lane: keys g + 8 r, rows 8 x + 2t, 8 x + 2t + 1
        float kf[4], ev[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            kf[r] = __shfl_sync(0xffffffffu, kf_lane, g + 8 * r);
            ev[r] = __shfl_sync(0xffffffffu, ev_lane, g + 8 * r);
        }
        uint32_t pb[NT][4];               // P^T operand: key pairs of row 8 x + g
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float d[4][2], w[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) d[r][h] = fmaf(c[x][r >> 1][(r & 1) * 2 + h] * qf[x][h], kf[r], -m[x][h]);
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if (tree) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    see[h] = visible(mask[x][h], first, valid) >> g;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!((see[h] >> (8 * r)) & 1u)) d[r][h] = -INFINITY;
                }
            }
            const uint32_t before = seen >> (2 * x);       // bits 0 and 1: the two rows
            const float d_max = fmax3(fmax3(d[0][0], d[0][1], d[1][0]), fmax3(d[1][1], d[2][0], d[2][1]), fmaxf(d[3][0], d[3][1]));
            if (__any_sync(0xffffffffu, (before & 3u) != 3u || d_max > kMarginM)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool fresh = !((before >> h) & 1u);
                    float up = fmaxf(fmaxf(d[0][h], d[1][h]), fmaxf(d[2][h], d[3][h]));
                    bool none = see[h] == 0u || !((see[h] | see[h] >> 8 | see[h] >> 16 | see[h] >> 24) & 1u);
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) {
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, y));
                        none &= __shfl_xor_sync(0xffffffffu, static_cast<int>(none), y) != 0;
                    }
                    if (!none) seen |= 1u << (2 * x + h);
                    if (!fresh && !(up > kMarginM)) up = 0.f;   // another row's reference moves, not this one's
                    if (!(fabsf(up) < INFINITY)) up = 0.f;   // no finite score: any reference does
                    m[x][h] += up;
                    l[x][h] *= fresh ? 1.f : ex2_ftz(-up);   // a fresh l is 0, and up may be any score
                    // o keeps its units; below 2^-256 it is nothing beside the new maximum's weight (>= 2^-126), and a
                    // larger T would cost the next weights their low bits
                    T[x][h] = fresh ? 0.f : fmaxf(T[x][h] - up, -256.f);
#pragma unroll
                    for (int r = 0; r < 4; ++r) d[r][h] -= up;
                }
            }
            // exponents of the weights over their reference: s - m + ev - T
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[r][h] = (d[r][h] + ev[r]) - T[x][h];
            if (tree) {                                    // whatever scale a key that is not seen has
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!((see[h] >> (8 * r)) & 1u)) w[r][h] = -INFINITY;
            }
            const float w_max = fmax3(fmax3(w[0][0], w[0][1], w[1][0]), fmax3(w[1][1], w[2][0], w[2][1]), fmaxf(w[3][0], w[3][1]));
            if (__any_sync(0xffffffffu, (before & 3u) != 3u || w_max > kMarginT)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool fresh = !((before >> h) & 1u);
                    float up = fmaxf(fmaxf(w[0][h], w[1][h]), fmaxf(w[2][h], w[3][h]));
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, y));
                    up = fresh || up > kMarginT ? up - kTopT : 0.f;
                    if (!(fabsf(up) < INFINITY)) up = 0.f;
                    T[x][h] += up;
                    const float f = fresh ? 1.f : ex2_ftz(-up);          // a fresh o is 0
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[r][h] -= up;
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        o[x][u][h] *= f;
                        o[x][u][2 + h] *= f;
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                l[x][0] += ex2_ftz(d[r][0]);
                l[x][1] += ex2_ftz(d[r][1]);
                pb[x][r] = transposed_8x8(pack_f16x2(ex2_ftz(w[r][0]), ex2_ftz(w[r][1])));
            }
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
#pragma unroll
                for (int x = 0; x < NT; ++x) mma_f16(o[x][2 * w], a0, a1, a2, a3, pb[x][2 * i], pb[x][2 * i + 1]);
                f16_of_codes(__byte_perm(wa[w], wd[w], 0x7362), a0, a1);
                f16_of_codes(__byte_perm(we[w], wf[w], 0x7362), a2, a3);
#pragma unroll
                for (int x = 0; x < NT; ++x) mma_f16(o[x][2 * w + 1], a0, a1, a2, a3, pb[x][2 * i], pb[x][2 * i + 1]);
            }
        }
        if (hurt != 0u) {
            // NaN, for the rows that see a node with NaN codes, in the codes' dims (this lane's are 16 g .. 16 g + 15)
            for (int r = 0; r < CHUNK; ++r) {
                if (!((hurt >> r) & 1u)) continue;
                const int pos = cc.c * CHUNK + r, lb = pos / p.block_size;
                const int phys = __ldg(p.block_tables + static_cast<int64_t>(cc.b) * p.max_blocks + lb);
                if (phys < 0 || phys >= p.num_blocks) continue;
                const uint8_t* code = p.v_codes + ((static_cast<int64_t>(phys) * p.block_size + (pos - lb * p.block_size)) * hkv + head) * D + 16 * g;
                uint32_t which = 0u;
                for (int d = 0; d < 16; ++d) which |= (__ldg(code + d) & 0x7fu) == 0x7fu ? 1u << d : 0u;
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t see = 8 * x + 2 * t + h < s.n << p.lg ? visible(mask[x][h], first, valid) : 0u;
                        if (!((see >> r) & 1u)) continue;
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            if ((which >> (2 * u)) & 1u) o[x][u][h] = __uint_as_float(0x7fc00000u);
                            if ((which >> (2 * u + 1)) & 1u) o[x][u][2 + h] = __uint_as_float(0x7fc00000u);
                        }
                    }
            }
        }
        if (tree) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // what was cleared, before the stage's next copy
        __syncwarp();
        if (copies.issued < n_mine) issue_next();

        // ---- end of the sequence or of the run: its rows, or what this run knows of them
        if (cc.c == cc.n - 1 || k == n_mine - 1) {
            const bool whole = seg_begin == 0 && cc.c == cc.n - 1;
            const int part = seg_begin > 0 ? 0 : 1;
            if (!whole && part == 1)                       // the run that holds chunk i is floor(((i + 1) W - 1) / total)
                meta = make_int4(static_cast<int>((static_cast<uint64_t>(begin + k + cc.n - cc.c) * static_cast<uint32_t>(W) - 1) / static_cast<uint32_t>(total)),
                                 s.q0, s.n << p.lg, 0);
            const int64_t slot = static_cast<int64_t>(gw) * 2 + part;
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float sum = l[x][h];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    const int row = 8 * x + 2 * t + h;
                    if (row >= s.n << p.lg) continue;
                    // |o| is below 2^48 (weights, codes, keys); 2^(T - e) may be out of range where its product with o is not
                    const float e = T[x][h] > 64.f && sum < INFINITY ? static_cast<float>(static_cast<int>(__float_as_uint(sum) >> 23) - 115) : 0.f;
                    float f = ex2_ftz(0.5f * (T[x][h] - e));
                    sum *= ex2_ftz(-e);
                    if (whole) {
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        uint32_t y[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) y[u] = pack_bf16x2(o[x][u][h] * f * f * inv, o[x][u][2 + h] * f * f * inv);
                        uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(s.q0 + (row >> p.lg)) * p.num_heads + (head << p.lg) +
                                                                       (row & ((1 << p.lg) - 1))) * D + 16 * g);
                        dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                        dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * ROWS + row) * D + 16 * g);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            dst[u] = make_float4(o[x][2 * u][h] * f * f, o[x][2 * u][2 + h] * f * f, o[x][2 * u + 1][h] * f * f, o[x][2 * u + 1][2 + h] * f * f);
                        if (g == 0) p.part_ml[slot * ROWS + row] = make_float2((seen >> (2 * x + h)) & 1u ? m[x][h] + e : -INFINITY, sum);
                    }
                }
            if (k != n_mine - 1) {
                cursor_next(cc, prefix, p.batch);
                seg_begin = 0;
                enter();
                reset();
            }
        } else {
            ++cc.c;
        }
    }
    if (failed)       // copies in flight land before the CTA's shared memory goes away
        for (; k < copies.issued; ++k) {
            const bool ok = mbar_wait(ring.bar0 + 8 * st, parity, p.err, gw);
            if (++st == STAGES) { st = 0; parity ^= 1u; }
            if (__any_sync(0xffffffffu, !ok)) break;
        }
    if (lane == 0) p.meta[gw] = failed ? make_int4(-1, 0, 0, 0) : meta;
}

// The sequences that several runs share: CTA (run, head) joins the one that its run leaves open, a warp each row.
template <int ROWS>
__global__ void __launch_bounds__(256) tree_rows_join_kernel(const Params p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int gw = blockIdx.x, hkv = p.num_kv_heads;
    const int4 u = p.meta[gw];
    if (u.x < 0) return;
    const int run = gw / hkv, head = gw - run * hkv, lane = threadIdx.x & 31;
    for (int row = threadIdx.x >> 5; row < u.z; row += 8) {
        auto at = [&](int i) { return ((static_cast<int64_t>(i) * hkv + head) * 2 + (i == run ? 1 : 0)) * ROWS + row; };
        constexpr int BATCH = 4;        // parts whose loads are issued together
        float M = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = run; i0 <= u.x; i0 += BATCH) {
            float2 ml[BATCH];
            float4 v[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + i <= u.x) {
                    ml[i] = p.part_ml[at(i0 + i)];
                    v[i] = *reinterpret_cast<const float4*>(p.part_o + at(i0 + i) * D + 4 * lane);
                }
            }
            const float now = fmax3(M, fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
            const float keep = M == now ? 1.f : ex2_ftz(M - now);
            l *= keep;
            acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
            M = now;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const float f = ml[i].x == M ? 1.f : ex2_ftz(ml[i].x - M);
                l = fmaf(f, ml[i].y, l);
                acc.x = fmaf(f, v[i].x, acc.x);
                acc.y = fmaf(f, v[i].y, acc.y);
                acc.z = fmaf(f, v[i].z, acc.z);
                acc.w = fmaf(f, v[i].w, acc.w);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* dst = p.out + (static_cast<int64_t>(u.y + (row >> p.lg)) * p.num_heads + (head << p.lg) + (row & ((1 << p.lg) - 1))) * D + 4 * lane;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
}

constexpr size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int max_groups(int num_kv_heads) { return sm_count() * WARPS / num_kv_heads; }

template <int NT>
bool allow_smem() {
    return cudaFuncSetAttribute(tree_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_bytes(kMaxTreeBatch))) == cudaSuccess;
}

template <int NT>
cudaError_t launch_pair(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p, cudaStream_t stream) {
    const int warps = p.groups * p.num_kv_heads;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = programmatic(dim3((warps + WARPS - 1) / WARPS), THREADS, smem_bytes(p.batch), stream, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_rows_kernel<NT>, tm_k, tm_v, p);
    if (e != cudaSuccess) return e;
    cfg = programmatic(dim3(warps), 256, 0, stream, attr);
    return cudaLaunchKernelEx(&cfg, tree_rows_join_kernel<8 * NT>, p);
}

size_t part_slots(int num_kv_heads) { return static_cast<size_t>(2) * max_groups(num_kv_heads) * num_kv_heads; }

}  // namespace

size_t tree_rows_workspace_bytes(int num_kv_heads) {
    const size_t slots = part_slots(num_kv_heads);
    return align256(slots * kTreeRows * D * 4) + align256(slots * kTreeRows * 8) + align256(slots * 8);
}

bool tree_rows_fits(const TreeDecodeArgs& a, int lg) {
    // what the tables can hold, not max_context: a batch's chunks are counted in 32 bits, and which kernel takes it does not
    // depend on how tight that bound is
    const int64_t chunks = (static_cast<int64_t>(a.max_blocks) * a.block_size + CHUNK - 1) / CHUNK;
    return a.k_scale != nullptr && (a.max_nodes << lg) <= kTreeRows && max_groups(a.num_kv_heads) >= 1 && a.batch * chunks <= 0x7fffffffLL;
}

pkv_status launch_tree_rows(const TreeDecodeArgs& a, int lg, int* err, cudaStream_t stream) {
    if (!setup_once(kSetupTreeRows, [] { return allow_smem<1>() && allow_smem<2>(); })) return PKV_ERR_CUDA;
    CUtensorMap tm_k, tm_v;
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.num_kv_heads), static_cast<uint64_t>(a.block_size),
                              static_cast<uint64_t>(a.num_blocks)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.num_kv_heads) * D,
                                 static_cast<uint64_t>(a.block_size) * a.num_kv_heads * D};
    const uint32_t box[4] = {static_cast<uint32_t>(D), 1u, static_cast<uint32_t>(CHUNK), 1u};
    if (encode_tiled(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(a.k_cache), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B) != CUDA_SUCCESS ||
        encode_tiled(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(a.v_cache), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B) != CUDA_SUCCESS)
        return PKV_ERR_INVALID_ARG;
    const size_t slots = part_slots(a.num_kv_heads);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    Params p{};
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + align256(slots * kTreeRows * D * 4));
    p.meta = reinterpret_cast<int4*>(ws + align256(slots * kTreeRows * D * 4) + align256(slots * kTreeRows * 8));
    p.q = a.q;
    p.v_codes = static_cast<const uint8_t*>(a.v_cache);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.cu_nodes = a.cu_nodes;
    p.mask = reinterpret_cast<const unsigned long long*>(a.tree_mask);
    p.out = a.out;
    p.max_blocks = a.max_blocks;
    p.batch = a.batch;
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
    // as many groups as the bounds allow runs, and no fewer than the lengths themselves ask for: how a batch is cut, and
    // with it every rounding, does not depend on how tight the bounds are
    const int64_t chunks = static_cast<int64_t>(a.batch) * ((static_cast<int64_t>(a.max_context) + CHUNK - 1) / CHUNK);
    p.groups = static_cast<int>(std::min<int64_t>(max_groups(a.num_kv_heads), std::max<int64_t>(1, chunks / KMIN)));
    const cudaError_t e = a.max_nodes << lg <= 8 ? launch_pair<1>(tm_k, tm_v, p, stream) : launch_pair<2>(tm_k, tm_v, p, stream);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
