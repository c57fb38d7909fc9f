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
// 16-byte loads, a row maximum by three shuffles.  A warp takes 4 rows at a time and several such
// groups of one token, so the (cos, sin) of its pairs are computed once for all of them.
//
// Measured on 10,814 tokens of 16 Q and 8 KV heads, 155 MB: 31.3 us = 4.97 TB/s through the ring of
// bulk copies, 38 us with the next item's loads in registers, 50 us without (one item per warp).
// 3 stages 33.2 us, 3 CTAs per SM 33.0, items of 8 rows 39.8, of 32 rows 37.0.  Issue slots are 53% busy, so
// they are not the bound.  With two items to a token and an even stride a warp's items are all Q rows or all K
// and V rows, which do not take equally long: the likely rest.
#include <cuda_fp8.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 256;
constexpr int ROW_LANES = 8;
constexpr int GROUP = 32 / ROW_LANES;    // rows a warp holds at a time
constexpr int CTAS_PER_SM = 2;

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
    for (int i = 0; i < 4; ++i) {
        float2 v;
        fmul2(v.x, v.y, x[2 * i], x[2 * i + 1], inv, inv);
        w[i] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// (cos, sin) of the angle that is turns / 2^32 of a turn.  The quadrant is taken off in integers, so
// what reaches the functions is at most an eighth of a turn, rounded to 2^-25 of itself, and the
// result is within a few 2^-24 -- which decides fewer roundings to e4m3 otherwise than exact values
// would than the hardware's approximation over a whole turn (4e-7) does.
__device__ __forceinline__ float2 cos_sin_of(uint32_t turns) {
    const uint32_t quadrant = (turns + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(turns - (quadrant << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);      // 2 / 2^32
    const float x = (quadrant & 1u) ? s : c, y = (quadrant & 1u) ? c : s;
    return make_float2(((quadrant + 1u) & 2u) ? -x : x, (quadrant & 2u) ? -y : y);
}

// Eight lanes' share of row r0 + sub of a token: its loads' bits, rotated (q, k), rounded and written.  The
// warp calls it together for rows r0 .. r0 + 3; what none of the four needs is skipped by all.
template <bool kRope>
__device__ __forceinline__ void put_row(const StoreFp8Args& a, int64_t t, int slot, int blk, int off, int r0, int sub, int j,
                                        const uint4& lo, const uint4& hi, const float (&cs)[8], const float (&sn)[8]) {
    const int hq = kRope ? a.num_heads : 0;                 // 0 without q
    const int r = r0 + sub;
    const bool is_q = r < hq;
    const bool is_k = !is_q && r < hq + a.num_kv_heads;
    const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w};
    const uint32_t wh[4] = {hi.x, hi.y, hi.z, hi.w};
    float y[8], z[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        y[2 * e] = bf16_lo(wl[e]);
        y[2 * e + 1] = bf16_hi(wl[e]);
        z[2 * e] = bf16_lo(wh[e]);
        z[2 * e + 1] = bf16_hi(wh[e]);
    }
    if (kRope && r0 < hq + a.num_kv_heads && (is_q || is_k)) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float u0, u1, v0, v1;
            fmul2(u0, u1, z[e], z[e + 1], -sn[e], -sn[e + 1]);
            fmul2(v0, v1, y[e], y[e + 1], sn[e], sn[e + 1]);
            ffma2(y[e], y[e + 1], y[e], y[e + 1], cs[e], cs[e + 1], u0, u1);
            ffma2(z[e], z[e + 1], z[e], z[e + 1], cs[e], cs[e + 1], v0, v1);
        }
    }
    if (kRope && is_q) {
        uint4* dst = reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + static_cast<int64_t>(r) * kHeadDim);
        dst[j] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        dst[ROW_LANES + j] = make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]),
                                        pack_bf16x2(z[6], z[7]));
    }
    if (r0 + GROUP <= hq) return;
    // the largest magnitude; a NaN anywhere shows as one, which is an exponent of 255 like an infinity's
    float m = amax3_nan(amax3_nan(amax3_nan(y[0], y[1], y[2]), y[3], y[4]), amax3_nan(y[5], y[6], y[7]),
                        amax3_nan(amax3_nan(z[0], z[1], z[2]), amax3_nan(z[3], z[4], z[5]), amax3_nan(z[6], z[7], 0.f)));
#pragma unroll
    for (int d = 1; d < ROW_LANES; d <<= 1) m = amax3_nan(m, __shfl_xor_sync(0xffffffffu, m, d), 0.f);
    if (!is_q && r < hq + 2 * a.num_kv_heads && slot >= 0 && slot < a.num_slots) {
        const int h = r - hq - (is_k ? 0 : a.num_kv_heads);
        const int byte = scale_byte(__float_as_uint(m) & 0x7fffffffu);
        uint2 c0 = make_uint2(0, 0), c1 = c0;
        if (byte != 255) {
            // 2^-(byte - 127), a normal number: the byte is at most 247
            const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
            c0 = to_codes(y, inv);
            c1 = to_codes(z, inv);
        }
        uint8_t* dst = (is_k ? a.k_cache : a.v_cache) + (static_cast<int64_t>(slot) * a.num_kv_heads + h) * kHeadDim;
        *reinterpret_cast<uint2*>(dst + 8 * j) = c0;
        *reinterpret_cast<uint2*>(dst + 64 + 8 * j) = c1;
        if (j == 0)
            (is_k ? a.k_scale : a.v_scale)[(static_cast<int64_t>(blk) * a.num_kv_heads + h) * a.block_size + off] =
                static_cast<uint8_t>(byte);
    }
}

// (cos, sin) of this lane's eight pairs 8j .. 8j + 7 at a position: two pairs per lane, the lane's own
// fractions of a turn f0 and f1 (pairs 2 lane, 2 lane + 1), handed on by shuffles.
__device__ __forceinline__ void pairs_of(int pos, uint64_t f0, uint64_t f1, int j, float (&cs)[8], float (&sn)[8]) {
    const float2 p0 = cos_sin_of(turns_of(pos, static_cast<uint32_t>(f0), static_cast<uint32_t>(f0 >> 32)));
    const float2 p1 = cos_sin_of(turns_of(pos, static_cast<uint32_t>(f1), static_cast<uint32_t>(f1 >> 32)));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cs[2 * e] = __shfl_sync(0xffffffffu, p0.x, 4 * j + e);
        sn[2 * e] = __shfl_sync(0xffffffffu, p0.y, 4 * j + e);
        cs[2 * e + 1] = __shfl_sync(0xffffffffu, p1.x, 4 * j + e);
        sn[2 * e + 1] = __shfl_sync(0xffffffffu, p1.y, 4 * j + e);
    }
}

// Few tokens: items are (token, 4U rows); a warp walks items with the grid's stride and issues the next
// item's loads before it works on the current one.
template <bool kRope, int U>
__global__ void __launch_bounds__(THREADS) store_fp8_kernel(const StoreFp8Args a, int64_t n_tokens, int chunks, int* err) {
    const int lane = threadIdx.x & 31;
    const int j = lane & (ROW_LANES - 1);
    const int sub = lane / ROW_LANES;
    const int hq = kRope ? a.num_heads : 0;
    const int rows = hq + 2 * a.num_kv_heads;
    const int64_t items = n_tokens * chunks;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
    int64_t it = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    if (it >= items) return;
    const uint64_t f0 = kRope ? a.turns[2 * lane] : 0, f1 = kRope ? a.turns[2 * lane + 1] : 0;
    struct Item {
        int64_t t;
        int chunk, slot, pos;
        uint4 lo[U], hi[U];
    };
    auto load = [&](int64_t i, Item& x) {
        x.t = i / chunks;
        x.chunk = static_cast<int>(i - x.t * chunks);
        x.slot = __ldg(a.slots + x.t);
        if (kRope) x.pos = __ldg(a.positions + x.t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = x.chunk * (GROUP * U) + u * GROUP + sub;
            x.lo[u] = x.hi[u] = make_uint4(0, 0, 0, 0);
            if (r < rows) {                                 // a skipped row is read too: its slot is not known yet
                const uint16_t* src;
                if (kRope && r < hq)
                    src = a.q + x.t * a.q_stride + static_cast<int64_t>(r) * kHeadDim;
                else if (r < hq + a.num_kv_heads)
                    src = a.k + x.t * a.k_stride + static_cast<int64_t>(r - hq) * kHeadDim;
                else
                    src = a.v + x.t * a.v_stride + static_cast<int64_t>(r - hq - a.num_kv_heads) * kHeadDim;
                x.lo[u] = __ldcs(reinterpret_cast<const uint4*>(src) + j);
                x.hi[u] = __ldcs(reinterpret_cast<const uint4*>(src) + ROW_LANES + j);
            }
        }
    };
    auto work = [&](const Item& x) {
        if (x.slot >= a.num_slots && x.chunk == 0 && lane == 0) record_error(err, PKV_DEVERR_SLOT, static_cast<int>(x.t));
        float cs[8], sn[8];
        if (kRope) pairs_of(x.pos, f0, f1, j, cs, sn);
        const int blk = max(x.slot, 0) / a.block_size, off = max(x.slot, 0) - blk * a.block_size;
#pragma unroll
        for (int u = 0; u < U; ++u)
            put_row<kRope>(a, x.t, x.slot, blk, off, x.chunk * (GROUP * U) + u * GROUP, sub, j, x.lo[u], x.hi[u], cs, sn);
    };
    Item cur, next;
    load(it, cur);
    for (; it + stride < items; it += stride) {
        load(it + stride, next);
        work(cur);
        cur = next;
    }
    work(cur);
}

// Many tokens: items are (token, RING_ROWS rows); each warp of a persistent grid keeps a ring of RING stages of
// shared memory filled by bulk copies (up to three an item: its q, k and v rows), which holds far more bytes in
// flight than registers do.
constexpr int RING = 2;
constexpr int RING_ROWS = 16;
constexpr int RING_STAGE = RING_ROWS * kHeadDim * 2;
constexpr int RING_CTAS_PER_SM = 2;
constexpr size_t kRingSmem = static_cast<size_t>(THREADS / 32) * RING * (RING_STAGE + 8);

template <bool kRope>
__global__ void __launch_bounds__(THREADS, RING_CTAS_PER_SM)
store_fp8_ring_kernel(const StoreFp8Args a, int64_t n_tokens, int chunks, int* err) {
    extern __shared__ __align__(128) uint8_t ring_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = lane & (ROW_LANES - 1);
    const int sub = lane / ROW_LANES;
    const int hq = kRope ? a.num_heads : 0;
    const int rows = hq + 2 * a.num_kv_heads;
    const int64_t items = n_tokens * chunks;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + warp;
    if (first >= items) return;
    const int64_t n_mine = (items - first + stride - 1) / stride;
    const uint32_t stage0 = smem_u32(ring_smem) + warp * RING * RING_STAGE;
    const uint32_t bar0 = smem_u32(ring_smem) + (THREADS / 32) * RING * RING_STAGE + warp * RING * 8;
    if (lane == 0) {
        for (int s = 0; s < RING; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    __syncwarp();
    const uint64_t f0 = kRope ? a.turns[2 * lane] : 0, f1 = kRope ? a.turns[2 * lane + 1] : 0;
    int slot[RING], pos[RING];
    int64_t issued = 0;
    auto issue = [&](int s) {                               // item `issued` into stage s
        const int64_t it = first + issued * stride;
        const int64_t t = it / chunks;
        const int r0 = static_cast<int>(it - t * chunks) * RING_ROWS, r1 = min(rows, r0 + RING_ROWS);
        slot[s] = __ldg(a.slots + t);
        pos[s] = kRope ? __ldg(a.positions + t) : 0;
        if (lane == 0) {
            const uint32_t bar = bar0 + 8 * s, dst = stage0 + s * RING_STAGE;
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(r1 - r0) * (kHeadDim * 2));
            auto part = [&](const uint16_t* src, int64_t token_stride, int begin, int end) {      // rows [begin, end) of the token
                const int x0 = max(r0, begin), x1 = min(r1, end);
                if (x0 < x1)
                    bulk_load(dst + (x0 - r0) * (kHeadDim * 2), src + t * token_stride + static_cast<int64_t>(x0 - begin) * kHeadDim,
                              static_cast<uint32_t>(x1 - x0) * (kHeadDim * 2), bar);
            };
            if (kRope) part(a.q, a.q_stride, 0, hq);
            part(a.k, a.k_stride, hq, hq + a.num_kv_heads);
            part(a.v, a.v_stride, hq + a.num_kv_heads, rows);
        }
        ++issued;
    };
#pragma unroll
    for (int s = 0; s < RING; ++s)
        if (issued < n_mine) issue(s);
    bool ok = true;
    int64_t done = 0;
    uint32_t parity = 0;
    while (done < n_mine && ok) {
#pragma unroll
        for (int s = 0; s < RING; ++s) {
            if (done >= n_mine || !ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * s, parity, err, 5));
            if (!ok) break;
            const int64_t it = first + done * stride;
            const int64_t t = it / chunks;
            const int chunk = static_cast<int>(it - t * chunks);
            const int sl = slot[s];
            if (sl >= a.num_slots && chunk == 0 && lane == 0) record_error(err, PKV_DEVERR_SLOT, static_cast<int>(t));
            float cs[8], sn[8];
            if (kRope) pairs_of(pos[s], f0, f1, j, cs, sn);
            const int blk = max(sl, 0) / a.block_size, off = max(sl, 0) - blk * a.block_size;
            const uint32_t at = stage0 + s * RING_STAGE + sub * (kHeadDim * 2) + 16 * j;
#pragma unroll
            for (int u = 0; u < RING_ROWS / GROUP; ++u) {
                const int r = chunk * RING_ROWS + u * GROUP;
                if (r >= rows) break;                       // whole groups past the token's rows (uniform)
                const uint4 lo = ld_shared_v4(at + u * GROUP * (kHeadDim * 2)), hi = ld_shared_v4(at + u * GROUP * (kHeadDim * 2) + 128);
                put_row<kRope>(a, t, sl, blk, off, r, sub, j, lo, hi, cs, sn);
            }
            ++done;
            __syncwarp();                                   // every lane has read the stage
            if (issued < n_mine) issue(s);
        }
        parity ^= 1u;
    }
    // copies still in flight (a wait above gave up) land before the CTA's shared memory goes away
    if (!ok)
        for (int64_t i = done; i < issued; ++i) mbar_wait(bar0 + 8 * static_cast<int>(i % RING), static_cast<uint32_t>((i / RING) & 1), err, 6);
}

template <bool kRope>
cudaError_t launch(const StoreFp8Args& a, int64_t n_tokens, int* err, cudaStream_t stream) {
    const int rows = a.num_heads + 2 * a.num_kv_heads;
    auto ctas_for = [&](int chunks) { return (n_tokens * chunks + THREADS / 32 - 1) / (THREADS / 32); };
    const int64_t sms = sm_count();
    // The ring pays once every warp of its grid walks a few items.
    const int ring_chunks = (rows + RING_ROWS - 1) / RING_ROWS;
    if (ctas_for(ring_chunks) >= 2 * RING_CTAS_PER_SM * sms) {
        if (!setup_once(kRope ? kSetupStoreFp8Rope : kSetupStoreFp8, [] {
                return cudaFuncSetAttribute(store_fp8_ring_kernel<kRope>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(kRingSmem)) == cudaSuccess;
            }))
            return cudaErrorUnknown;
        store_fp8_ring_kernel<kRope><<<static_cast<unsigned>(RING_CTAS_PER_SM * sms), THREADS, kRingSmem, stream>>>(a, n_tokens,
                                                                                                                     ring_chunks, err);
        return cudaGetLastError();
    }
    constexpr int U = 2;
    const int chunks = (rows + GROUP * U - 1) / (GROUP * U);
    const int64_t ctas = std::min<int64_t>(ctas_for(chunks), CTAS_PER_SM * sms);
    store_fp8_kernel<kRope, U><<<static_cast<unsigned>(ctas), THREADS, 0, stream>>>(a, n_tokens, chunks, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_store_fp8(const StoreFp8Args& a, int64_t n_tokens, int* err, cudaStream_t stream) {
    if (n_tokens == 0) return cudaSuccess;
    return a.positions ? launch<true>(a, n_tokens, err, stream) : launch<false>(a, n_tokens, err, stream);
}

}  // namespace pkv
