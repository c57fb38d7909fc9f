// Varlen prefill attention over an 8-bit KV cache.
//
// The keys and values a batch attends to are first decoded, once per call, into bf16 tiles of 128
// tokens in the workspace, and the tcgen05 prefill kernel then runs over those tiles.  A row's
// scale is a power of two, so code * 2^e is exact in bf16 (down to its subnormals): the result
// is bit for bit that of the bf16 prefill over a cache holding the decoded values.
//
// Decoding once costs 387 bytes of traffic per K or V row (129 in, 256 out, mostly into L2, where
// the attention reads it back), linear in the keys; the attention reads each tile once per
// 256 / G query tokens and its work is quadratic, so what decoding inside the attention kernel
// would save in traffic it would pay back in conversions repeated for every query tile, on the
// softmax warps' issue slots, which already bound that kernel.
//
// Tile j of sequence s lives at tile floor((cu_k[s] - cu_k[0] + 127 s) / 128) + j: consecutive
// sequences' ranges cannot overlap (ceil(k / 128) <= (k + 127) / 128), so no scan is needed.
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int D = kHeadDim;
constexpr int TILE = 128;         // tokens per workspace tile (a prefill KV tile)
constexpr int PART = 32;          // tokens one CTA decodes at a time
constexpr int THREADS = 256;

struct DecodeTilesParams {
    const uint8_t* codes[2];      // K, V
    const uint8_t* scale[2];
    uint16_t* tiles[2];           // [num_tiles][TILE][num_kv_heads][D] bf16
    const int32_t* cu_k;
    const int32_t* block_tables;
    int32_t* tile_tables;         // [num_seqs][max_tiles]
    int max_blocks, num_seqs, num_kv_heads, block_size, num_blocks, max_tiles;
    int64_t num_tiles, total_k;
    int* err;
};

__device__ __forceinline__ int64_t first_tile(const int32_t* cu_k, int s) {
    return (static_cast<int64_t>(__ldg(cu_k + s)) - __ldg(cu_k) + static_cast<int64_t>(TILE - 1) * s) / TILE;
}

// Keys of sequence s, or -1 where its tiles do not fit (the lengths break the call's bounds).
__device__ __forceinline__ int keys_of(const DecodeTilesParams& p, int s) {
    const int64_t kl = static_cast<int64_t>(__ldg(p.cu_k + s + 1)) - __ldg(p.cu_k + s);
    const int64_t first = first_tile(p.cu_k, s);
    if (kl < 0 || kl > static_cast<int64_t>(p.max_blocks) * p.block_size || first < 0) return -1;
    const int64_t need = (kl + TILE - 1) / TILE;
    const bool within = static_cast<int64_t>(__ldg(p.cu_k + s + 1)) - __ldg(p.cu_k) <= p.total_k;
    return within && need <= p.max_tiles && first + need <= p.num_tiles ? static_cast<int>(kl) : -1;
}

// Four e4m3 codes times f (a power of two), as four bf16.
__device__ __forceinline__ uint2 bf16_of_codes(uint32_t w, float f) {
    uint32_t a, b;
    f16_of_codes(w, a, b);
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return make_uint2(pack_bf16x2(lo.x * f, lo.y * f), pack_bf16x2(hi.x * f, hi.y * f));
}

__global__ void __launch_bounds__(THREADS) decode_tiles_kernel(const DecodeTilesParams p) {
    const int tid = threadIdx.x;
    // the tables the attention kernel walks: tile j of sequence s
    const int64_t entries = static_cast<int64_t>(p.num_seqs) * p.max_tiles;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + tid; i < entries; i += static_cast<int64_t>(gridDim.x) * THREADS) {
        const int s = static_cast<int>(i / p.max_tiles), j = static_cast<int>(i - static_cast<int64_t>(s) * p.max_tiles);
        const int kl = keys_of(p, s);
        if (kl < 0 && j == 0) record_error(p.err, PKV_DEVERR_SEQLENS, s);
        p.tile_tables[i] = j * TILE < kl ? static_cast<int32_t>(first_tile(p.cu_k, s) + j) : -1;
    }
    const int64_t items = p.num_tiles * (TILE / PART) * 2;
    const int vecs = PART * p.num_kv_heads * (D / 16);        // 16 codes each
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int which = static_cast<int>(it & 1);
        const int64_t tile = (it >> 1) / (TILE / PART);
        const int part = static_cast<int>((it >> 1) - tile * (TILE / PART));
        int lo = 0, hi = p.num_seqs;                          // the last sequence whose first tile is not behind
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_tile(p.cu_k, mid) <= tile) lo = mid; else hi = mid;
        }
        const int kl = keys_of(p, lo);
        const int64_t tok0 = (tile - first_tile(p.cu_k, lo)) * TILE + part * PART;
        if (tok0 < 0 || tok0 >= kl) continue;
        const int n = min(PART, static_cast<int>(kl - tok0));
        const int blk = static_cast<int>(tok0 / p.block_size);
        const int off0 = static_cast<int>(tok0 - static_cast<int64_t>(blk) * p.block_size);
        const int phys = __ldg(p.block_tables + static_cast<int64_t>(lo) * p.max_blocks + blk);
        const bool known = phys >= 0 && phys < p.num_blocks;
        if (!known && tid == 0) record_error(p.err, PKV_DEVERR_BLOCK_ID, lo);
        const int64_t src_row = (static_cast<int64_t>(known ? phys : 0) * p.block_size + off0) * p.num_kv_heads;
        const uint4* src = reinterpret_cast<const uint4*>(p.codes[which] + src_row * D);
        uint4* dst = reinterpret_cast<uint4*>(p.tiles[which] + (tile * TILE + part * PART) * p.num_kv_heads * D);
        const uint8_t* scale = p.scale[which] + static_cast<int64_t>(known ? phys : 0) * p.num_kv_heads * p.block_size + off0;
        for (int v = tid; v < vecs; v += THREADS) {
            const int row = v / (D / 16);
            const int tok = row / p.num_kv_heads, h = row - tok * p.num_kv_heads;
            if (tok >= n) break;
            const uint32_t byte = __ldg(scale + static_cast<int64_t>(h) * p.block_size + tok);
            const float f = !known ? 0.f : e8m0_value(byte);
            const uint4 w = known ? __ldcs(src + v) : make_uint4(0, 0, 0, 0);
            const uint2 a = bf16_of_codes(w.x, f), b = bf16_of_codes(w.y, f), c = bf16_of_codes(w.z, f), d = bf16_of_codes(w.w, f);
            dst[2 * v] = make_uint4(a.x, a.y, b.x, b.y);
            dst[2 * v + 1] = make_uint4(c.x, c.y, d.x, d.y);
        }
    }
}

constexpr size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int64_t tiles_of(int num_seqs, int64_t total_k) { return (total_k + static_cast<int64_t>(TILE - 1) * num_seqs) / TILE + 1; }

}  // namespace

size_t prefill_fp8_workspace_bytes(int num_seqs, int num_kv_heads, int max_seqlen_q, int max_seqlen_k, int64_t total_k,
                                   int log_group) {
    const size_t pool = static_cast<size_t>(tiles_of(num_seqs, total_k)) * TILE * num_kv_heads * D * 2;
    const size_t tables = static_cast<size_t>(num_seqs) * ((max_seqlen_k + TILE - 1) / TILE) * 4;
    return align256(prefill_workspace_bytes(num_seqs, max_seqlen_q, log_group)) + align256(tables) + 2 * align256(pool);
}

pkv_status launch_prefill_fp8(const PrefillFp8Args& a, int* err, cudaStream_t stream) {
    const int lg = group_log2(a.num_heads, a.num_kv_heads);
    if (lg < 0) return PKV_ERR_UNSUPPORTED;
    const int64_t num_tiles = tiles_of(a.num_seqs, a.total_k);
    const int max_tiles = (a.max_seqlen_k + TILE - 1) / TILE;
    if (num_tiles > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    if (a.workspace == nullptr || a.workspace_bytes < prefill_fp8_workspace_bytes(a.num_seqs, a.num_kv_heads, a.max_seqlen_q,
                                                                                  a.max_seqlen_k, a.total_k, lg))
        return PKV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const size_t plan_bytes = prefill_workspace_bytes(a.num_seqs, a.max_seqlen_q, lg);
    const size_t pool = static_cast<size_t>(num_tiles) * TILE * a.num_kv_heads * D * 2;
    int32_t* tables = reinterpret_cast<int32_t*>(ws + align256(plan_bytes));
    uint8_t* k_tiles = ws + align256(plan_bytes) + align256(static_cast<size_t>(a.num_seqs) * max_tiles * 4);

    DecodeTilesParams p;
    p.codes[0] = a.k_cache;
    p.codes[1] = a.v_cache;
    p.scale[0] = a.k_scale;
    p.scale[1] = a.v_scale;
    p.tiles[0] = reinterpret_cast<uint16_t*>(k_tiles);
    p.tiles[1] = reinterpret_cast<uint16_t*>(k_tiles + align256(pool));
    p.cu_k = a.cu_k;
    p.block_tables = a.block_tables;
    p.tile_tables = tables;
    p.max_blocks = a.max_blocks;
    p.num_seqs = a.num_seqs;
    p.num_kv_heads = a.num_kv_heads;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.max_tiles = max_tiles;
    p.num_tiles = num_tiles;
    p.total_k = a.total_k;
    p.err = err;
    const int64_t items = num_tiles * (TILE / PART) * 2;
    decode_tiles_kernel<<<static_cast<unsigned>(std::min<int64_t>(items, 8LL * sm_count())), THREADS, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;

    PrefillArgs f;
    f.q = a.q;
    f.k_cache = p.tiles[0];
    f.v_cache = p.tiles[1];
    f.cu_q = a.cu_q;
    f.cu_k = a.cu_k;
    f.block_tables = tables;
    f.out = a.out;
    f.max_blocks = max_tiles;
    f.num_seqs = a.num_seqs;
    f.total_q = a.total_q;
    f.max_seqlen_q = a.max_seqlen_q;
    f.max_seqlen_k = a.max_seqlen_k;
    f.num_heads = a.num_heads;
    f.num_kv_heads = a.num_kv_heads;
    f.block_size = TILE;
    f.num_blocks = static_cast<int>(num_tiles);
    f.softmax_scale = a.softmax_scale;
    f.workspace = a.workspace;
    f.workspace_bytes = plan_bytes;
    return launch_prefill(f, err, stream, kPrefillPlanAndRun);
}

}  // namespace pkv
