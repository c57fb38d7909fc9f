// Append to an 8-bit KV cache: rotary embedding (optional), rounding to e4m3 with one
// power-of-two scale per row, and the scatter to the pool slots, in one pass.
//
// A row is one token of one KV head, 128 numbers x.  Its scale exponent is
//   e = min { e >= -126 : max|x| <= 448 * 2^e }
// and its codes are e4m3(x * 2^-e), rounded to nearest even (one rounding; K is rounded from the
// fp32 rotated value).  e4m3 is a floating-point format, so a finer scale would buy no relative
// precision, while a power of two makes every decoded value code * 2^e exact in bf16 and lets a
// reader apply the scale by exponent arithmetic.  The byte stored is e + 127 (E8M0); a row that
// holds an infinity or a NaN gets byte 255, E8M0's NaN, and codes 0: it reads as NaN.
//
// The step is bound by HBM: 256 bytes in and 129 out per K or V row, 512 per Q row.  Eight lanes
// hold a row, lane j elements [8j, 8j+8) and [64+8j, 64+8j+8): both halves of its rotary pairs,
// 16-byte loads, a row maximum by three shuffles.  A warp takes 4 rows at a time and U such
// groups of one token, so its (cos, sin) of the lane's 8 pairs are computed once for 4U rows.
#include <cuda_fp8.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 256;
constexpr int ROW_LANES = 8;
constexpr int GROUP = 32 / ROW_LANES;    // rows a warp holds at a time

// The E8M0 byte of a row whose largest |x| has these fp32 bits (largest as an integer, so an
// infinity or a NaN in the row shows as an exponent of 255).  448 = 1.75 * 2^8: with
// amax = (1 + m) 2^(E - 127), the exponent is E - 127 - 8, one more if 1 + m > 1.75.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
    const int E = static_cast<int>(amax_bits >> 23);
    if (E == 255) return 255;
    const int b = E - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(b, 1);
}

// Eight fp32 values times `inv`, as eight e4m3 codes.
__device__ __forceinline__ uint2 to_codes(const float (&x)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <bool kRope, int U>
__global__ void __launch_bounds__(THREADS) store_fp8_kernel(const StoreFp8Args a, int64_t n_tokens, int chunks, int* err) {
    const int lane = threadIdx.x & 31;
    const int j = lane & (ROW_LANES - 1);
    const int sub = lane / ROW_LANES;
    const int rows = a.num_heads + 2 * a.num_kv_heads;      // num_heads is 0 without q
    const int64_t items = n_tokens * chunks;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5); it < items; it += stride) {
        const int64_t t = it / chunks;
        const int chunk = static_cast<int>(it - t * chunks);
        const int slot = __ldg(a.slots + t);
        const bool in_pool = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && chunk == 0 && lane == 0) record_error(err, PKV_DEVERR_SLOT, static_cast<int>(t));
        uint4 lo[U], hi[U];
        const int r0 = chunk * (GROUP * U) + sub;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * GROUP;
            lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
            if (r < rows && (r < a.num_heads || in_pool)) {
                const uint16_t* src;
                if (kRope && r < a.num_heads)
                    src = a.q + t * a.q_stride + static_cast<int64_t>(r) * kHeadDim;
                else if (r < a.num_heads + a.num_kv_heads)
                    src = a.k + t * a.k_stride + static_cast<int64_t>(r - a.num_heads) * kHeadDim;
                else
                    src = a.v + t * a.v_stride + static_cast<int64_t>(r - a.num_heads - a.num_kv_heads) * kHeadDim;
                lo[u] = __ldcs(reinterpret_cast<const uint4*>(src) + j);
                hi[u] = __ldcs(reinterpret_cast<const uint4*>(src) + ROW_LANES + j);
            }
        }
        float cs[8], sn[8];
        if (kRope) {
            const int pos = __ldg(a.positions + t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t f = a.turns[8 * j + e];
                __sincosf(reduced_angle(pos, static_cast<uint32_t>(f), static_cast<uint32_t>(f >> 32)), &sn[e], &cs[e]);
            }
        }
        const int64_t blk = in_pool ? slot / a.block_size : 0;
        const int off = in_pool ? slot - static_cast<int>(blk) * a.block_size : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * GROUP;
            const bool is_q = r < a.num_heads;
            const bool is_k = !is_q && r < a.num_heads + a.num_kv_heads;
            const uint32_t wl[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w};
            const uint32_t wh[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
            float x[8], y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = bf16_lo(wl[e]);
                x[2 * e + 1] = bf16_hi(wl[e]);
                y[2 * e] = bf16_lo(wh[e]);
                y[2 * e + 1] = bf16_hi(wh[e]);
            }
            if (kRope && (is_q || is_k)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = x[e], q = y[e];
                    x[e] = fmaf(p, cs[e], -q * sn[e]);
                    y[e] = fmaf(q, cs[e], p * sn[e]);
                }
            }
            uint32_t amax = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
                amax = max(amax, __float_as_uint(y[e]) & 0x7fffffffu);
            }
#pragma unroll
            for (int d = 1; d < ROW_LANES; d <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            if (kRope && is_q) {
                uint4* dst = reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + static_cast<int64_t>(r) * kHeadDim);
                dst[j] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                    pack_bf16x2(x[6], x[7]));
                dst[ROW_LANES + j] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            } else if (r < rows && in_pool) {
                const int h = r - a.num_heads - (is_k ? 0 : a.num_kv_heads);
                const int byte = scale_byte(amax);
                uint2 c0 = make_uint2(0, 0), c1 = c0;
                if (byte != 255) {
                    // 2^-(byte - 127), a normal number: the byte is at most 248
                    const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
                    c0 = to_codes(x, inv);
                    c1 = to_codes(y, inv);
                }
                uint8_t* dst = (is_k ? a.k_cache : a.v_cache) +
                               (static_cast<int64_t>(slot) * a.num_kv_heads + h) * kHeadDim;
                *reinterpret_cast<uint2*>(dst + 8 * j) = c0;
                *reinterpret_cast<uint2*>(dst + 64 + 8 * j) = c1;
                if (j == 0)
                    (is_k ? a.k_scale : a.v_scale)[(blk * a.num_kv_heads + h) * a.block_size + off] =
                        static_cast<uint8_t>(byte);
            }
        }
    }
}

template <bool kRope, int U>
cudaError_t launch(const StoreFp8Args& a, int64_t n_tokens, int* err, cudaStream_t stream) {
    const int rows = a.num_heads + 2 * a.num_kv_heads;
    const int chunks = (rows + GROUP * U - 1) / (GROUP * U);
    const int64_t ctas = (n_tokens * chunks + THREADS / 32 - 1) / (THREADS / 32);
    store_fp8_kernel<kRope, U><<<static_cast<unsigned>(std::min<int64_t>(ctas, 1 << 20)), THREADS, 0, stream>>>(
        a, n_tokens, chunks, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_store_fp8(const StoreFp8Args& a, int64_t n_tokens, int* err, cudaStream_t stream) {
    if (n_tokens == 0) return cudaSuccess;
    return a.positions ? launch<true, 2>(a, n_tokens, err, stream) : launch<false, 2>(a, n_tokens, err, stream);
}

}  // namespace pkv
