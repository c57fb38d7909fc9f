// The samplers' noise: Philox4x32-10 words and what is derived from them.
#pragma once

#include <stdint.h>

namespace pkv {

// Philox4x32 round constants from the SC'11 paper (multipliers and Weyl increments).
constexpr uint32_t kPhiloxM0 = 0xD2511F53u;
constexpr uint32_t kPhiloxM1 = 0xCD9E8D57u;
constexpr uint32_t kPhiloxW0 = 0x9E3779B9u;
constexpr uint32_t kPhiloxW1 = 0xBB67AE85u;

// Philox4x32-10 (ten rounds of two 32x32 -> 64 products, the high halves xored into the
// other words with the round key, which advances by the Weyl increments) for the counters
// (q, c1, c2, 0) of one row: the words that do not depend on q make round 0's second
// product and round 1's first product row constants, computed once.
struct PhiloxRow {
    uint32_t x0, y0, p_hi, p_lo, k0, k1;
};
__device__ __forceinline__ PhiloxRow philox_row(uint32_t c1, uint32_t c2, uint32_t k0, uint32_t k1) {
    PhiloxRow r;
    const uint64_t a = static_cast<uint64_t>(kPhiloxM1) * c2;
    r.x0 = static_cast<uint32_t>(a >> 32) ^ c1 ^ k0;
    r.y0 = static_cast<uint32_t>(a);
    const uint64_t p = static_cast<uint64_t>(kPhiloxM0) * r.x0;
    r.p_hi = static_cast<uint32_t>(p >> 32);
    r.p_lo = static_cast<uint32_t>(p);
    r.k0 = k0;
    r.k1 = k1;
    return r;
}
// The ten round keys of both words.  With a host seed they are computed on the host and
// read from the kernel's parameters, so the rounds spend no instruction on them.
struct RoundKeys {
    uint32_t k0[10], k1[10];
};
template <bool kParamKeys>
__device__ __forceinline__ uint32_t round_key(const RoundKeys& rk, uint32_t base, int word, int round) {
    if (kParamKeys) return word == 0 ? rk.k0[round] : rk.k1[round];
    return base + static_cast<uint32_t>(round) * (word == 0 ? kPhiloxW0 : kPhiloxW1);
}
template <bool kParamKeys>
__device__ __forceinline__ uint4 philox_row_at(uint32_t q, const PhiloxRow& r, const RoundKeys& rk) {
    const uint64_t b = static_cast<uint64_t>(kPhiloxM0) * q;            // round 0
    const uint32_t z0 = static_cast<uint32_t>(b >> 32) ^ round_key<kParamKeys>(rk, r.k1, 1, 0);
    const uint32_t w0 = static_cast<uint32_t>(b);
    const uint64_t d = static_cast<uint64_t>(kPhiloxM1) * z0;           // round 1
    uint4 c = make_uint4(static_cast<uint32_t>(d >> 32) ^ r.y0 ^ round_key<kParamKeys>(rk, r.k0, 0, 1),
                         static_cast<uint32_t>(d), r.p_hi ^ w0 ^ round_key<kParamKeys>(rk, r.k1, 1, 1), r.p_lo);
#pragma unroll
    for (int round = 2; round < 10; ++round) {
        const uint32_t k0 = round_key<kParamKeys>(rk, r.k0, 0, round);
        const uint32_t k1 = round_key<kParamKeys>(rk, r.k1, 1, round);
        const uint64_t e0 = static_cast<uint64_t>(kPhiloxM0) * c.x;
        const uint64_t e1 = static_cast<uint64_t>(kPhiloxM1) * c.z;
        c = make_uint4(static_cast<uint32_t>(e1 >> 32) ^ c.y ^ k0, static_cast<uint32_t>(e1),
                       static_cast<uint32_t>(e0 >> 32) ^ c.w ^ k1, static_cast<uint32_t>(e0));
    }
    return c;
}

// 1 - u of a noise word, exactly: with m = x >> 9, f = 1 + (2^23 - 1 - m) 2^-23 in [1, 2) has the
// complemented mantissa bits, and 1 - u = (2^24 - 2m - 1) 2^-24 = f - (1 - 2^-24), a difference
// of two floats within a factor of two of each other and therefore exact.
// ex2.approx, which the candidate bounds use, is within 2^-22 relatively, well inside their
// 1.001 margin; a bound flushed to zero only skips elements that cannot win (1 - u >= 2^-24).
__device__ __forceinline__ float one_minus_u_of(uint32_t x) {
    const float f = __uint_as_float(0x3F800000u | (~x >> 9));
    return f - 0.999999940395355224609375f;
}

}  // namespace pkv
