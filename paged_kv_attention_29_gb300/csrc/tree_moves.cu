// What follows the attention of a tree of drafted tokens: the accepted path, its rows
// moved together in every layer's pools, and the rows of blocks copied for a fork.
#include <algorithm>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// ---------------------------------------------------------------------------
// accepted path
// ---------------------------------------------------------------------------
// One warp per tree.  A node's parent is the highest bit of its mask below its own.  The walk starts at node 0 and
// goes to the first child whose draft is the token sampled at the node, as long as there is one.  Lane i holds nodes
// i, i + 32, ... in registers, so a step of the walk is a read of one target and a ballot per 32 nodes; what a tree
// costs is the latency of its loads and of the walk's steps: 2.0 us a call in a graph for one tree of 26 nodes.
constexpr int ACCEPT_WARPS = 4, NODE_REGS = kMaxTreeNodes / 32;

__global__ void __launch_bounds__(32 * ACCEPT_WARPS) tree_accept_kernel(const TreeAcceptArgs a, int* err) {
    __shared__ long long targets[ACCEPT_WARPS][kMaxTreeNodes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x * ACCEPT_WARPS + warp;
    if (b >= a.batch) return;
    const int q0 = __ldg(a.cu_nodes + b), q1 = __ldg(a.cu_nodes + b + 1), len = __ldg(a.context_lens + b);
    const long long nodes = static_cast<long long>(q1) - q0;
    int32_t* path = a.path + static_cast<int64_t>(b) * a.max_path;
    const bool fits = q0 >= 0 && nodes >= 0 && q1 <= a.total_nodes && nodes <= a.max_nodes && nodes <= len;
    const int n = fits ? static_cast<int>(nodes) : 0;
    if (!fits && nodes != 0 && lane == 0) record_error(err, PKV_DEVERR_SEQLENS, b);
    int parent[NODE_REGS];
    long long draft[NODE_REGS];
#pragma unroll
    for (int k = 0; k < NODE_REGS; ++k) {
        parent[k] = -1;
        draft[k] = 0;
        if (32 * k >= n) continue;
        const int i = 32 * k + lane;
        if (i < n) {
            const int64_t at = static_cast<int64_t>(q0) + i;
            draft[k] = __ldg(reinterpret_cast<const long long*>(a.draft) + at);
            targets[warp][i] = __ldg(reinterpret_cast<const long long*>(a.target) + at);
            for (int w = i >> 6; w >= 0; --w) {
                unsigned long long m = __ldg(reinterpret_cast<const unsigned long long*>(a.tree_mask) + at * a.mask_words + w);
                if (w == i >> 6) m &= (1ull << (i & 63)) - 1ull;
                if (m) {
                    parent[k] = 64 * w + 63 - __clzll(static_cast<long long>(m));
                    break;
                }
            }
        }
    }
    __syncwarp();
    int count = 0, cur = n > 0 ? 0 : -1;
    long long next = -1;
    while (cur >= 0) {
        if (lane == 0) path[count] = cur;
        ++count;
        next = targets[warp][cur];
        if (count == a.max_path) break;
        int child = -1;
#pragma unroll
        for (int k = 0; k < NODE_REGS; ++k) {
            if (32 * k >= n || child >= 0) continue;
            const unsigned hit = __ballot_sync(0xffffffffu, parent[k] == cur && draft[k] == next);
            if (hit) child = 32 * k + __ffs(static_cast<int>(hit)) - 1;
        }
        cur = child;
    }
    for (int d = count + lane; d < a.max_path; d += 32) path[d] = -1;
    if (lane == 0) {
        a.path_lens[b] = count;
        a.next_tokens[b] = next;
        a.new_context_lens[b] = len - n + count;
    }
}

// ---------------------------------------------------------------------------
// compaction of the accepted rows
// ---------------------------------------------------------------------------
// CTA (x, b): some pools (a layer's K or V each) of sequence b.  The accepted node of depth d moves to the d-th row
// behind the context.  A path's nodes ascend and node path[d] >= d, so a row that is written has been read before by
// the same thread: each thread takes columns of all rows in order, BATCH rows at a time, loads first.  What a call costs
// beside its bytes is the chain of path, block table and rows, so the GPU is filled once: a CTA walks the chain for as
// many pools as that takes, one warp lists the rows that move (and where their scales lie: a division by the block size
// costs more than a move), and the 8-bit rows' scales have a warp of their own.
// Measured in a graph: one sequence, 28 layers 2.4 us; 128 sequences on the 8-bit cache, 52 MB in rows of 1 KB and
// single scale bytes, 15.9 us (3.3 TB/s); 128 on bf16, 103 MB, 24.1 us.
constexpr int ROW_THREADS = 256, COMPACT_THREADS = ROW_THREADS + 32, COMPACT_CTAS = 5, BATCH = 4;

__global__ void __launch_bounds__(COMPACT_THREADS, COMPACT_CTAS)
tree_compact_kernel(const __grid_constant__ PoolTable pools, const TreeCompactArgs a, int pools_per_cta, int* err) {
    __shared__ int64_t src[kMaxTreeNodes], dst[kMaxTreeNodes];     // rows that move, block * block_size + offset
    __shared__ int64_t src_scale[kMaxTreeNodes], dst_scale[kMaxTreeNodes];   // and the places of their first head's scales
    __shared__ int moves;
    const int b = blockIdx.y, tid = threadIdx.x;
    if (tid < 32) {
        const bool say = blockIdx.x == 0;
        const int32_t* path = a.path + static_cast<int64_t>(b) * a.max_path;
        int node = tid < a.max_path ? __ldg(path + tid) : -1;      // asked for before the lengths are known
        const int q0 = __ldg(a.cu_nodes + b), q1 = __ldg(a.cu_nodes + b + 1), len = __ldg(a.context_lens + b), count = __ldg(a.path_lens + b);
        const long long n = static_cast<long long>(q1) - q0;
        const bool fits = n >= 0 && n <= kMaxTreeNodes && n <= len && len <= static_cast<long long>(a.max_blocks) * a.block_size;
        bool good = fits && count >= 0 && count <= a.max_path && count <= n;
        if (!good && count != 0 && say && tid == 0) record_error(err, fits ? PKV_DEVERR_TREE : PKV_DEVERR_SEQLENS, b);
        int listed = 0, before = -1;                               // the last node of the 32 before
        for (int d0 = 0; good && d0 < count; d0 += 32) {
            const int d = d0 + tid;
            if (d0) node = d < count ? __ldg(path + d) : -1;
            int prev = __shfl_up_sync(0xffffffffu, node, 1);
            if (tid == 0) prev = before;
            before = __shfl_sync(0xffffffffu, node, 31);
            // a path that does not ascend could be read after it is written
            good = __all_sync(0xffffffffu, d >= count || (node > prev && node < n));
            if (!good && say && tid == 0) record_error(err, PKV_DEVERR_TREE, b);
            int64_t row[2] = {-1, -1}, scale[2];
            if (good && d < count && node != d) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int pos = len - static_cast<int>(n) + (k ? d : node), lb = pos / a.block_size;
                    const int phys = __ldg(a.block_tables + static_cast<int64_t>(b) * a.max_blocks + lb);
                    const int off = pos - lb * a.block_size;
                    scale[k] = static_cast<int64_t>(phys) * a.num_kv_heads * a.block_size + off;
                    if (phys >= 0 && phys < a.num_blocks)
                        row[k] = static_cast<int64_t>(phys) * a.block_size + off;
                    else if (say)
                        record_error(err, PKV_DEVERR_BLOCK_ID, b);
                }
            }
            const bool moving = row[0] >= 0 && row[1] >= 0;
            const unsigned who = __ballot_sync(0xffffffffu, moving);
            if (moving) {
                const int at = listed + __popc(who & ((1u << tid) - 1u));
                src[at] = row[0];
                dst[at] = row[1];
                src_scale[at] = scale[0];
                dst_scale[at] = scale[1];
            }
            listed += __popc(who);
        }
        if (tid == 0) moves = good ? listed : 0;
    }
    __syncthreads();
    const int count = moves;
    if (count == 0) return;
    const int pool0 = blockIdx.x * pools_per_cta, here = min(pools_per_cta, 2 * pools.layers - pool0);
    // one column; from[d] * stride and to[d] * stride: its places in the listed rows
    auto move = [&](auto* column, const int64_t* from, const int64_t* to, int64_t stride) {
        for (int d0 = 0; d0 < count; d0 += BATCH) {
            std::remove_reference_t<decltype(*column)> x[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (d0 + i < count) x[i] = column[from[d0 + i] * stride];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (d0 + i < count) column[to[d0 + i] * stride] = x[i];
        }
    };
    if (tid < ROW_THREADS) {
        const int vecs = a.row_bytes / 16;
        for (int c = tid; c < here * vecs; c += ROW_THREADS) {
            const int i = c / vecs, x = pool0 + i;
            move(static_cast<uint4*>(x & 1 ? pools.v[x >> 1] : pools.k[x >> 1]) + (c - i * vecs), src, dst, vecs);
        }
    } else if (pools.k_scale[0] != nullptr) {
        for (int c = tid - ROW_THREADS; c < here * a.num_kv_heads; c += 32) {
            const int i = c / a.num_kv_heads, x = pool0 + i;
            move((x & 1 ? pools.v_scale[x >> 1] : pools.k_scale[x >> 1]) + static_cast<int64_t>(c - i * a.num_kv_heads) * a.block_size, src_scale,
                 dst_scale, 1);
        }
    }
}

// ---------------------------------------------------------------------------
// block copies
// ---------------------------------------------------------------------------
// CTA (chunk, pool, pair).  The first rows of a block are one run of bytes in the source and in the destination; each
// CTA moves CHUNK bytes of it, all of a thread's loads before its stores.
// Measured: 64 blocks filled to any row, 28 layers, 1.07 GB read and written: 164 us, 97% of a plain copy's rate; one block of
// 137 rows, 31 MB: 5.1 us in a graph.
constexpr int COPY_THREADS = 256, COPY_VECS = 8, CHUNK = COPY_THREADS * COPY_VECS * 16;

__global__ void __launch_bounds__(COPY_THREADS) copy_blocks_kernel(const __grid_constant__ PoolTable pools, const CopyBlocksArgs a, int* err) {
    const int pair = blockIdx.z, pool = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    const int s = __ldg(a.src + pair), d = __ldg(a.dst + pair), n = a.rows ? __ldg(a.rows + pair) : a.block_size;
    const bool say = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    if (s < 0 || n == 0) return;
    if (s >= a.num_blocks || d < 0 || d >= a.num_blocks) {
        if (say) record_error(err, PKV_DEVERR_BLOCK_ID, pair);
        return;
    }
    if (n < 0 || n > a.block_size) {
        if (say) record_error(err, PKV_DEVERR_SEQLENS, pair);
        return;
    }
    if (s == d) return;
    const int64_t block_bytes = static_cast<int64_t>(a.block_size) * a.row_bytes, bytes = static_cast<int64_t>(n) * a.row_bytes;
    uint8_t* rows = static_cast<uint8_t*>(is_v ? pools.v[pool] : pools.k[pool]);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * CHUNK;
    const uint4* from = reinterpret_cast<const uint4*>(rows + s * block_bytes + at);
    uint4* to = reinterpret_cast<uint4*>(rows + d * block_bytes + at);
    const int vecs = static_cast<int>(min(static_cast<int64_t>(CHUNK), bytes - at) / 16);
    uint4 x[COPY_VECS];
#pragma unroll
    for (int i = 0; i < COPY_VECS; ++i)
        if (static_cast<int>(threadIdx.x) + i * COPY_THREADS < vecs) x[i] = __ldcs(from + threadIdx.x + i * COPY_THREADS);
#pragma unroll
    for (int i = 0; i < COPY_VECS; ++i)
        if (static_cast<int>(threadIdx.x) + i * COPY_THREADS < vecs) to[threadIdx.x + i * COPY_THREADS] = x[i];
    uint8_t* scales = is_v ? pools.v_scale[pool] : pools.k_scale[pool];
    if (scales == nullptr || blockIdx.x != 0) return;
    // scales [KV head][row]: the first n bytes of each head, 16 at a time and the rest singly
    const int full = n / 16, per_head = full + (n & 15);
    const int64_t s0 = static_cast<int64_t>(s) * a.num_kv_heads * a.block_size, d0 = static_cast<int64_t>(d) * a.num_kv_heads * a.block_size;
    for (int i = threadIdx.x; i < per_head * a.num_kv_heads; i += COPY_THREADS) {
        const int h = i / per_head, v = i - h * per_head;
        const int64_t head = static_cast<int64_t>(h) * a.block_size;
        if (v < full)
            *reinterpret_cast<uint4*>(scales + d0 + head + 16 * v) = *reinterpret_cast<const uint4*>(scales + s0 + head + 16 * v);
        else
            scales[d0 + head + 15 * full + v] = scales[s0 + head + 15 * full + v];
    }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, int* err, cudaStream_t stream) {
    tree_accept_kernel<<<(a.batch + ACCEPT_WARPS - 1) / ACCEPT_WARPS, 32 * ACCEPT_WARPS, 0, stream>>>(a, err);
    return cudaGetLastError();
}

cudaError_t launch_tree_compact(const PoolTable& pools, const TreeCompactArgs& a, int* err, cudaStream_t stream) {
    // as many pools to a CTA as let all CTAs run at once
    const int64_t all = 2ll * pools.layers * a.batch, room = static_cast<int64_t>(COMPACT_CTAS) * std::max(1, sm_count());
    const int per = static_cast<int>(std::min<int64_t>(2 * pools.layers, (all + room - 1) / room));
    tree_compact_kernel<<<dim3((2 * pools.layers + per - 1) / per, a.batch), COMPACT_THREADS, 0, stream>>>(pools, a, per, err);
    return cudaGetLastError();
}

cudaError_t launch_copy_blocks(const PoolTable& pools, const CopyBlocksArgs& a, int* err, cudaStream_t stream) {
    const int64_t bytes = static_cast<int64_t>(a.block_size) * a.row_bytes;
    copy_blocks_kernel<<<dim3(static_cast<unsigned>((bytes + CHUNK - 1) / CHUNK), 2 * pools.layers, a.pairs), COPY_THREADS, 0, stream>>>(pools, a, err);
    return cudaGetLastError();
}

}  // namespace pkv
