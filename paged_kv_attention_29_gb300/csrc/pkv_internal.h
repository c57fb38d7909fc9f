// Host-side declarations shared by the libpkv translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pkv.h"

namespace pkv {

constexpr int kHeadDim = 128;
constexpr int kMaxLogGroup = 3;      // query heads per KV head: 1, 2, 4 or 8
constexpr int kBlockQuantum = 256;   // block_size must be a multiple of this

// log2(num_heads / num_kv_heads) when that ratio is 1, 2, 4 or 8; otherwise -1.
int group_log2(int num_heads, int num_kv_heads);

// Device address of the current device's error word (int[2]); nullptr on failure.
int* device_error_word();

// Streaming multiprocessors of the current device (cached per device).
int sm_count();

// One-time set-up of kernel attributes, per device.  Runs `setup` with the
// current device once (thread-safe; a failed set-up is retried on the next
// call) and returns whether the set-up for `key` has succeeded on this device.
enum SetupKey { kSetupDecode = 0, kSetupPrefill, kSetupRopeStore, kSetupDecodeFp8, kSetupSampleFiltered, kSetupStoreFp8,
                kSetupStoreFp8Rope, kSetupTreeDecode, kSetupTreeRows, kNumSetupKeys };
bool setup_once(SetupKey key, bool (*setup)());

// cuTensorMapEncodeTiled through the runtime's driver entry point.
CUresult encode_tiled(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t rank, void* base,
                      const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                      CUtensorMapSwizzle swizzle,
                      CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);

// ---- a1 / a2 --------------------------------------------------------------
cudaError_t launch_slot_mapping(const int32_t* cu_q, const int32_t* cu_k, const int32_t* ctx,
                                const int32_t* block_tables, int max_blocks, int num_seqs,
                                int total_q, int block_size, int num_blocks, int32_t* slots,
                                int* err, cudaStream_t stream);

cudaError_t launch_store_kvcache(const uint16_t* k, const uint16_t* v, int64_t n_tokens,
                                 int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                 uint16_t* k_cache, uint16_t* v_cache, int64_t num_slots,
                                 int row_elems, int* err, cudaStream_t stream);

// ---- f2: RoPE fused into the KV write -------------------------------------------
constexpr int kMaxRopePairs = 128;   // head_dim <= 256

struct RopeStoreArgs {
    const uint16_t* q;        // nullptr: rotate and store K only
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* positions;
    const int32_t* slots;
    uint16_t* k_cache;
    uint16_t* v_cache;
    int64_t q_stride, q_out_stride, k_stride, v_stride;   // elements between tokens
    int64_t num_slots;
    int64_t kv_row;            // num_kv_heads * head_dim
    int num_heads, num_kv_heads, head_dim;
    uint64_t turns[kMaxRopePairs];    // 2^64 * frac(base^(-2i/d) / (2 pi)), i < d/2
};

// Threads one CTA needs (one per work item of a token); 0 if above 1024.
int rope_store_threads(const RopeStoreArgs& a);
cudaError_t launch_rope_store(const RopeStoreArgs& a, int64_t n_tokens, int* err, cudaStream_t stream);

// ---- 8-bit KV cache: append ---------------------------------------------------
struct StoreFp8Args {
    const uint16_t* q;            // nullptr: no query rows (num_heads is then 0)
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* positions;     // nullptr: no rotation (and no query rows)
    const int32_t* slots;
    uint8_t* k_cache;             // e4m3 codes [num_blocks, block_size, num_kv_heads, 128]
    uint8_t* v_cache;
    uint8_t* k_scale;             // E8M0 bytes [num_blocks, num_kv_heads, block_size]
    uint8_t* v_scale;
    int64_t q_stride, q_out_stride, k_stride, v_stride;
    int64_t num_slots;
    int num_heads, num_kv_heads, block_size;
    uint64_t turns[kHeadDim / 2]; // as RopeStoreArgs
};
cudaError_t launch_store_fp8(const StoreFp8Args& a, int64_t n_tokens, int* err, cudaStream_t stream);

// ---- a4 ---------------------------------------------------------------------
struct DecodeArgs {
    const uint16_t* q;
    const uint16_t* k_cache;
    const uint16_t* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    uint16_t* out;
    int max_blocks;
    int batch;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    float softmax_scale;
    void* workspace;
    size_t workspace_bytes;
    const uint16_t* k_new = nullptr;   // fused KV write (pkv_decode_append); nullptr: none
    const uint16_t* v_new = nullptr;
    int32_t* slot_out = nullptr;
};

int decode_total_warps();                                  // warps the decode grid runs
size_t decode_workspace_bytes(int batch, int num_kv_heads, int log_group, int total_warps);
pkv_status launch_decode(const DecodeArgs& a, int* err, cudaStream_t stream);

// ---- a3 ---------------------------------------------------------------------
struct PrefillArgs {
    const uint16_t* q;
    const uint16_t* k_cache;
    const uint16_t* v_cache;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* block_tables;
    uint16_t* out;
    int max_blocks;
    int num_seqs;
    int total_q;
    int max_seqlen_q;
    int max_seqlen_k;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    float softmax_scale;
    void* workspace;
    size_t workspace_bytes;
};

// log_group = log2(num_heads / num_kv_heads)
size_t prefill_workspace_bytes(int num_seqs, int max_seqlen_q, int log_group);
// kPrefillPlanAndRun: plan the work list into the workspace, then attend;
// kPrefillPlanOnly: the plan alone; kPrefillRunOnly: attend on the plan already
// in the workspace (made for the same lengths, bounds and group size).
enum PrefillMode { kPrefillPlanAndRun, kPrefillPlanOnly, kPrefillRunOnly };
pkv_status launch_prefill(const PrefillArgs& a, int* err, cudaStream_t stream, PrefillMode mode);

// ---- 8-bit KV cache: attention ---------------------------------------------------
struct DecodeFp8Args {
    const uint16_t* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    uint16_t* out;
    int max_blocks;
    int batch;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    float softmax_scale;
    void* workspace;
    size_t workspace_bytes;
};
size_t decode_fp8_workspace_bytes(int batch, int num_kv_heads, int log_group);
pkv_status launch_decode_fp8(const DecodeFp8Args& a, int* err, cudaStream_t stream);

struct PrefillFp8Args {
    const uint16_t* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* block_tables;
    uint16_t* out;
    int max_blocks;
    int num_seqs;
    int total_q;
    int64_t total_k;
    int max_seqlen_q;
    int max_seqlen_k;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    float softmax_scale;
    void* workspace;
    size_t workspace_bytes;
};
size_t prefill_fp8_workspace_bytes(int num_seqs, int num_kv_heads, int max_seqlen_q, int max_seqlen_k, int64_t total_k,
                                   int log_group);
pkv_status launch_prefill_fp8(const PrefillFp8Args& a, int* err, cudaStream_t stream);

// ---- a5 ---------------------------------------------------------------------
cudaError_t launch_sample(const float* logits, int batch, int vocab, int64_t row_stride,
                          const float* temperatures, uint64_t seed, uint64_t offset,
                          const uint64_t* seed_offset, int64_t* out_ids, int* err, cudaStream_t stream);


// Sampling with filters; seed_offset: device {seed, offset}, or nullptr to use the host values.
struct SampleFilteredArgs {
    const float* logits;
    const float* temperatures;
    const int32_t* top_k;      // nullptr: off for every row
    const float* top_p;
    const float* min_p;
    const uint64_t* seed_offset;
    int64_t* out_ids;
    int64_t row_stride;
    uint64_t seed, offset;
    int batch, vocab;
};
pkv_status launch_sample_filtered(const SampleFilteredArgs& a, int* err, cudaStream_t stream);

// ---- trees of drafted tokens ------------------------------------------------------
// A launch that may start before the kernel in front of it has ended (the kernel waits with griddepcontrol.wait before it
// touches global memory); attr has to live until the launch.
inline cudaLaunchConfig_t programmatic(dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

constexpr int kMaxTreeNodes = 256;
constexpr int kMaxTreeBatch = 4096;
constexpr int kTreeRows = 16;         // nodes x group of the trees that tree_decode_rows.cu takes
constexpr int kMaxLayers = PKV_MAX_LAYERS;

struct TreeDecodeArgs {
    const uint16_t* q;
    const void* k_cache;
    const void* v_cache;
    const uint8_t* k_scale;       // nullptr: bf16 cache
    const uint8_t* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_nodes;
    const uint64_t* tree_mask;
    uint16_t* out;
    int max_blocks;
    int batch;
    int total_nodes;
    int max_nodes;
    int mask_words;
    int max_context;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    float softmax_scale;
    void* workspace;
    size_t workspace_bytes;
};
size_t tree_decode_workspace_bytes(int num_kv_heads);
pkv_status launch_tree_decode(const TreeDecodeArgs& a, int* err, cudaStream_t stream);
// Small trees on the 8-bit cache, to which launch_tree_decode hands over; lg = log2(num_heads / num_kv_heads).
bool tree_rows_fits(const TreeDecodeArgs& a, int lg);
size_t tree_rows_workspace_bytes(int num_kv_heads);
pkv_status launch_tree_rows(const TreeDecodeArgs& a, int lg, int* err, cudaStream_t stream);

struct TreeAcceptArgs {
    const int64_t* target;
    const int64_t* draft;
    const uint64_t* tree_mask;
    const int32_t* cu_nodes;
    const int32_t* context_lens;
    int32_t* path;
    int32_t* path_lens;
    int64_t* next_tokens;
    int32_t* new_context_lens;
    int batch, total_nodes, max_nodes, mask_words, max_path;
};
cudaError_t launch_tree_accept(const TreeAcceptArgs& a, int* err, cudaStream_t stream);

// Every layer's pools, as a kernel argument.
struct PoolTable {
    void* k[kMaxLayers];
    void* v[kMaxLayers];
    uint8_t* k_scale[kMaxLayers];
    uint8_t* v_scale[kMaxLayers];
    int layers;
};

struct TreeCompactArgs {
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_nodes;
    const int32_t* path;
    const int32_t* path_lens;
    int max_blocks, batch, max_path, block_size, num_blocks, num_kv_heads;
    int row_bytes;                // K or V of one token, all KV heads
};
cudaError_t launch_tree_compact(const PoolTable& pools, const TreeCompactArgs& a, int* err, cudaStream_t stream);

struct CopyBlocksArgs {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* rows;          // nullptr: whole blocks
    int pairs, block_size, num_blocks, num_kv_heads;
    int row_bytes;
};
cudaError_t launch_copy_blocks(const PoolTable& pools, const CopyBlocksArgs& a, int* err, cudaStream_t stream);

}  // namespace pkv
