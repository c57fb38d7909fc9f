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
// Measured: 32 prompts, 18,000 keys of 8 KV heads, 25 us for the tiles (37 MB in, 74 MB out) beside 54 us of
// attention; a prompt of 8192 tokens 11 us beside 160.  Eight codes per lane, so that a warp stores
// whole lines: sixteen took 31 us.
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
constexpr int PART = 16;          // tokens one CTA decodes at a time
constexpr int THREADS = 256;
constexpr int BATCH = 4;
constexpr int CTAS_PER_SM = 4;
constexpr int MAX_NEAR = 1023;

struct DecodeTilesParams {
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    uint16_t* k_tiles;            // [num_tiles][TILE][num_kv_heads][D] bf16
    uint16_t* v_tiles;
    const int32_t* cu_k;
    const int32_t* block_tables;
    int32_t* tile_tables;         // [num_seqs][max_tiles]
    int max_blocks, num_seqs, num_kv_heads, block_size, num_blocks, max_tiles;
    uint32_t heads_magic;         // ceil(2^32 / num_kv_heads), which divides a part's rows by umulhi; 0 for one head
    int64_t num_tiles, total_k;
    int* err;
};

__device__ __forceinline__ int64_t first_tile(const int32_t* cu_k, int s) {
    return (static_cast<int64_t>(cu_k[s]) - cu_k[0] + static_cast<int64_t>(TILE - 1) * s) / TILE;
}

// Keys of sequence s, or -1 where its tiles do not fit (the lengths break the call's bounds).
__device__ __forceinline__ int keys_of(const DecodeTilesParams& p, const int32_t* cu_k, int s) {
    const int64_t kl = static_cast<int64_t>(cu_k[s + 1]) - cu_k[s];
    const int64_t first = first_tile(cu_k, s);
    if (kl < 0 || kl > static_cast<int64_t>(p.max_blocks) * p.block_size || first < 0) return -1;
    const int64_t need = (kl + TILE - 1) / TILE;
    const bool within = static_cast<int64_t>(cu_k[s + 1]) - cu_k[0] <= p.total_k;
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

// Started beside the plan (which it does not read) by programmatic launch; it ends after the plan has, so
// the attention kernel, which waits for this one, finds both done.
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) decode_tiles_kernel(const DecodeTilesParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    // the running key counts, searched for every item: in shared memory where they fit
    __shared__ int32_t cu_near[MAX_NEAR + 1];
    const bool near = p.num_seqs <= MAX_NEAR;
    if (near)
        for (int i = tid; i <= p.num_seqs; i += THREADS) cu_near[i] = __ldg(p.cu_k + i);
    __syncthreads();
    const int32_t* cu_k = near ? cu_near : p.cu_k;
    // the tables the attention kernel walks: tile j of sequence s
    const int64_t entries = static_cast<int64_t>(p.num_seqs) * p.max_tiles;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + tid; i < entries; i += static_cast<int64_t>(gridDim.x) * THREADS) {
        const int s = static_cast<int>(i / p.max_tiles), j = static_cast<int>(i - static_cast<int64_t>(s) * p.max_tiles);
        const int kl = keys_of(p, cu_k, s);
        if (kl < 0 && j == 0) record_error(p.err, PKV_DEVERR_SEQLENS, s);
        p.tile_tables[i] = j * TILE < kl ? static_cast<int32_t>(first_tile(cu_k, s) + j) : -1;
    }
    const int64_t items = p.num_tiles * (TILE / PART);
    const int row_vecs = p.num_kv_heads * (D / 8);            // 8 codes each (a warp stores 512 bytes in a row): a token's
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t tile = it / (TILE / PART);
        const int part = static_cast<int>(it - tile * (TILE / PART));
        int lo = 0, hi = p.num_seqs;                          // the last sequence whose first tile is not behind
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_tile(cu_k, mid) <= tile) lo = mid; else hi = mid;
        }
        const int kl = keys_of(p, cu_k, lo);
        const int64_t tok0 = (tile - first_tile(cu_k, lo)) * TILE + part * PART;
        if (tok0 < 0 || tok0 >= kl) continue;
        const int n = min(PART, static_cast<int>(kl - tok0));
        const int blk = static_cast<int>(tok0 / p.block_size);
        const int off0 = static_cast<int>(tok0 - static_cast<int64_t>(blk) * p.block_size);
        const int phys = __ldg(p.block_tables + static_cast<int64_t>(lo) * p.max_blocks + blk);
        const bool known = phys >= 0 && phys < p.num_blocks;
        if (!known && tid == 0) record_error(p.err, PKV_DEVERR_BLOCK_ID, lo);
        const int64_t block = known ? phys : 0;
        const int64_t src0 = (block * p.block_size + off0) * row_vecs;
        const int64_t dst0 = (tile * TILE + part * PART) * row_vecs;
        const int64_t scale0 = block * p.num_kv_heads * p.block_size + off0;
        const int vecs = n * row_vecs;
        // K and V of BATCH vectors at a time, loads first
        for (int v0 = tid; v0 < vecs; v0 += BATCH * THREADS) {
            uint2 w[2][BATCH];
            float f[2][BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int v = min(v0 + i * THREADS, vecs - 1);
                const int row = v / (D / 8), tok = p.heads_magic ? static_cast<int>(__umulhi(row, p.heads_magic)) : row;
                const int h = row - tok * p.num_kv_heads;
                const int64_t at = scale0 + static_cast<int64_t>(h) * p.block_size + tok;
                w[0][i] = __ldcs(reinterpret_cast<const uint2*>(p.k_codes) + src0 + v);
                w[1][i] = __ldcs(reinterpret_cast<const uint2*>(p.v_codes) + src0 + v);
                f[0][i] = e8m0_value(__ldg(p.k_scale + at));
                f[1][i] = e8m0_value(__ldg(p.v_scale + at));
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int v = v0 + i * THREADS;
                if (v >= vecs) break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint2 c = known ? w[x][i] : make_uint2(0, 0);
                    const float g = known ? f[x][i] : 0.f;
                    const uint2 a = bf16_of_codes(c.x, g), b = bf16_of_codes(c.y, g);
                    (reinterpret_cast<uint4*>(x ? p.v_tiles : p.k_tiles) + dst0)[v] = make_uint4(a.x, a.y, b.x, b.y);
                }
            }
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int64_t tiles_of(int num_seqs, int64_t total_k) { return (total_k + static_cast<int64_t>(TILE - 1) * num_seqs) / TILE + 1; }

}  // namespace

size_t prefill_fp8_workspace_bytes(int num_seqs, int num_kv_heads, int max_seqlen_q, int max_seqlen_k, int64_t total_k,
                                   int log_group) {
    const size_t pool = static_cast<size_t>(tiles_of(num_seqs, total_k)) * TILE * num_kv_heads * D * 2;
    const size_t tables = static_cast<size_t>(num_seqs) * ((static_cast<int64_t>(max_seqlen_k) + TILE - 1) / TILE) * 4;
    return align256(prefill_workspace_bytes(num_seqs, max_seqlen_q, log_group)) + align256(tables) + 2 * align256(pool);
}

pkv_status launch_prefill_fp8(const PrefillFp8Args& a, int* err, cudaStream_t stream) {
    const int lg = group_log2(a.num_heads, a.num_kv_heads);
    if (lg < 0) return PKV_ERR_UNSUPPORTED;
    if (a.max_seqlen_k > (1 << 24)) return PKV_ERR_UNSUPPORTED;     // (the plan's own limit is lower)
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
    p.k_codes = a.k_cache;
    p.v_codes = a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.k_tiles = reinterpret_cast<uint16_t*>(k_tiles);
    p.v_tiles = reinterpret_cast<uint16_t*>(k_tiles + align256(pool));
    p.cu_k = a.cu_k;
    p.block_tables = a.block_tables;
    p.tile_tables = tables;
    p.max_blocks = a.max_blocks;
    p.num_seqs = a.num_seqs;
    p.num_kv_heads = a.num_kv_heads;
    p.heads_magic = a.num_kv_heads > 1 ? static_cast<uint32_t>(((1ull << 32) + a.num_kv_heads - 1) / a.num_kv_heads) : 0u;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.max_tiles = max_tiles;
    p.num_tiles = num_tiles;
    p.total_k = a.total_k;
    p.err = err;
    PrefillArgs f;
    f.q = a.q;
    f.k_cache = p.k_tiles;
    f.v_cache = p.v_tiles;
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
    // the plan; the tiles beside it; the attention after both
    pkv_status st = launch_prefill(f, err, stream, kPrefillPlanOnly);
    if (st != PKV_OK) return st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(num_tiles * (TILE / PART), static_cast<int64_t>(CTAS_PER_SM) * sm_count())));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, decode_tiles_kernel, p) != cudaSuccess) return PKV_ERR_CUDA;
    return launch_prefill(f, err, stream, kPrefillRunOnly);
}

}  // namespace pkv
