// What the attentions of few query rows over the 8-bit cache share (one token: decode_fp8.cu, small trees:
// tree_decode_rows.cu): 32-key chunks that go by in a ring of stages of each warp, products on mma.sync with the codes
// turned into f16 in registers, and a query row's f16 form.
#pragma once

#include <cuda_fp16.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp8_rows {

constexpr int D = kHeadDim;
constexpr int CHUNK = 32;                    // keys per stage
constexpr int WARPS = 8;
constexpr int STAGES = 3;                    // per warp
constexpr int THREADS = WARPS * 32;
constexpr int TILE_BYTES = CHUNK * D;        // one e4m3 tile
constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K, V
constexpr int SCALE_BYTES = 2 * CHUNK;       // a stage's K scales, V scales
constexpr int KMIN = 2;                      // chunks a run takes at least, where the batch allows it
constexpr float kTopT = 13.f;                // log2 of the largest weight, when its reference moves
constexpr float kMarginT = 15.f;             // and what moves it
constexpr float kMarginM = 64.f;             // the same of the softmax terms, which move to 0
static_assert(TILE_BYTES % 1024 == 0, "swizzled tiles start on 1 KiB");

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

// A warp's ring in shared memory.
struct Ring {
    uint32_t stage0, scale0, bar0;
};

// A warp's copies of its chunks into its ring: a cursor of their own, the block it is in, and a window of 32 block-table entries.
struct Copies {
    Cursor at;
    int blk, off;
    int bt_b = -1, bt_base = 0, bt_lane = -1;
    int issued = 0, put = 0;         // chunks issued; the stage the next one goes to

    __device__ __forceinline__ Copies(const Cursor& start, int block_size) : at(start) {
        blk = at.c * CHUNK / block_size;
        off = at.c * CHUNK - blk * block_size;
    }

    template <typename Params>
    __device__ __forceinline__ void next(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p, const Ring& ring, const int32_t* prefix,
                                         int head, int lane, uint64_t policy) {
        if (at.b != bt_b || blk < bt_base || blk >= bt_base + 32) {
            bt_b = at.b;
            bt_base = blk;
            const int i = bt_base + lane;
            bt_lane = i < p.max_blocks ? __ldg(p.block_tables + static_cast<int64_t>(at.b) * p.max_blocks + i) : -1;
        }
        const int phys = __shfl_sync(0xffffffffu, bt_lane, blk - bt_base);
        if (lane == 0) {
            const bool known = phys >= 0 && phys < p.num_blocks;
            if (!known) record_error(p.err, PKV_DEVERR_BLOCK_ID, at.b);
            const uint32_t bar = ring.bar0 + 8 * put;
            const uint32_t dst = ring.stage0 + put * STAGE_BYTES, sdst = ring.scale0 + put * SCALE_BYTES;
            // the tensor copies fill a block outside the pool with zeros; its scales come from block 0
            const int64_t srow = (static_cast<int64_t>(known ? phys : 0) * p.num_kv_heads + head) * p.block_size + off;
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
        cursor_next(at, prefix, p.batch);
        if (at.c == 0) blk = off = 0;
    }
};

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

// The query operand in f16: w, the raw words of row lane / 4, dims 32 (lane % 4) ... + 31, times a power of two; and, for the
// rows 2t, 2t + 1 (t = lane % 4) of this lane's columns, the factor that turns a raw product into log2-domain scores.
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
    qf[0] = __shfl_sync(0xffffffffu, f, (lane & 3) * 8);        // row 2t sits in lanes 8t .. 8t + 3
    qf[1] = __shfl_sync(0xffffffffu, f, (lane & 3) * 8 + 4);
}

}  // namespace fp8_rows
}  // namespace pkv
