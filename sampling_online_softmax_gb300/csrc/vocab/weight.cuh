// weight.cuh -- softmax weights as whole numbers: 2^((l - m) c) in units of
// 2^-U, right to about 45 bits, in fp32 arithmetic alone.
//
// A draw picks the token at a border of a sum over the whole row, and top-p cuts
// the order at another, so a weight's error moves the choice wherever tokens are
// small: with 10^4 tokens in play, weights right to 2^-22 (one ex2.approx) would
// pick another token than the definition for about one row in a hundred.  GB300's
// FP64 pipe issues two FMAs a clock per SM, so an exp in double costs a row of
// 150 k logits over a millisecond; the same accuracy from pairs of floats takes
// about 50 fp32 operations.  Sums of whole numbers do not depend on their order.
//
// x = (l - m) c is kept as a pair (TwoSum of l and -m, products with their FMA
// remainders), x = n + t/32 + g with |g| <= 1/64, and
//   2^x = 2^n T[t] (1 + E),  E = e^y - 1,  y = g ln 2,  |y| < 0.0109,
// T from a table of float pairs, E by its Taylor series: y and y^2/2 as pairs,
// y^3/6 + y^4/24 + y^5/120 in fp32 (their sum is below 2^-22, so its rounding is
// below 2^-45; y^6/720 is below 2^-48).
#pragma once

#include <cstdint>
#include <cstring>

namespace spec {
namespace vocab {

#ifdef __CUDACC__
#define SPEC_HD __host__ __device__ __forceinline__
#else
#define SPEC_HD inline
#endif

constexpr int kPow2Steps = 32;
// 2^(t/32) as a float and the remainder.
#define SPEC_POW2_TABLE                                                                          \
    {                                                                                            \
        {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},    \
        {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, \
        {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, \
        {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, \
        {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, \
        {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, \
        {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, \
        {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, \
        {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, \
        {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, \
        {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, \
        {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, \
        {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, \
        {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, \
        {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, \
        {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f} \
    }

SPEC_HD float bits_float(int b) {
#ifdef __CUDA_ARCH__
    return __int_as_float(b);
#else
    float f;
    memcpy(&f, &b, 4);
    return f;
#endif
}

// What turns a row's logits into weights: the row maximum m, c = log2(e) / T as a pair, U.
struct Scale {
    float m;
    float ch, cl;
    int U;  // units of 2^-U; U + bits(V) <= 62, so that a row's sum stays below 2^63
};

SPEC_HD unsigned long long fixed_weight(float l, const Scale &s, const float2 *pow2) {
    const float dh = l - s.m;
    const float ph = dh * s.ch;
    if (!(ph > -60.f)) return 0ull;  // below half a unit for every U; also l = -inf
    const float bb = dh - l;
    const float dl = (l - (dh - bb)) + (-s.m - bb);
    float pl = fmaf(dh, s.ch, -ph);
    pl = fmaf(dh, s.cl, pl);
    pl = fmaf(dl, s.ch, pl);
    const float jf = rintf(ph * 32.f);
    const int j = static_cast<int>(jf);
    const float gx = fmaf(jf, -0.03125f, ph);  // exact: both are multiples of ph's last place
    const float g = gx + pl;                   // |pl| reaches 2^-18: left apart, y^3/6 would miss it
    const float gl = pl - (g - gx);
    constexpr float kLn2h = 0x1.62e430p-1f, kLn2l = -0x1.05c610p-29f;
    const float yh = g * kLn2h;
    float yl = fmaf(g, kLn2h, -yh);
    yl = fmaf(g, kLn2l, yl);
    yl = fmaf(gl, kLn2h, yl);
    const float sh = yh * yh;
    const float sl = fmaf(yh, yh, -sh);
    const float c3 = sh * yh * fmaf(yh, fmaf(yh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
    const float h = 0.5f * sh;
    const float eh = yh + h;
    const float el = (h - (eh - yh)) + (fmaf(0.5f, sl, yl) + fmaf(yh, yl, c3));
    const float2 T = pow2[j & (kPow2Steps - 1)];
    const float qh = T.x * eh;
    const float ql = fmaf(T.x, el, fmaf(T.x, eh, -qh)) + T.y * eh;
    const float wh = T.x + qh;
    const float wl = (qh - (wh - T.x)) + (T.y + ql);
    // wh + wl in units of 2^-U as (whole multiple of 2^22) + rest: scaled by a power of two, so exactly
    const int e = (j >> 5) + s.U - 22;                   // 2^e units of 2^(22 - U); e in [-41, 30]
    if (e < -24) return 0ull;                            // below half a unit
    const float up = bits_float((e + 127) << 23);
    const float t = wh * up;
    const uint32_t hi = static_cast<uint32_t>(t);
    const float rest = (t - static_cast<float>(hi)) + wl * up;  // exact, then one rounding
    const int lo = static_cast<int>(rintf(rest * 0x1p22f));
    return (static_cast<unsigned long long>(hi) << 22) + static_cast<long long>(lo);
}

// floor(W * f) for f in [0, 1), and whether f * W is no whole number, exactly.
SPEC_HD unsigned long long scaled_floor(unsigned long long W, float f, bool *rest) {
    int e = 0;
    const float fr = frexpf(f, &e);  // f = fr 2^e, fr in [0.5, 1), e <= 0
    const unsigned long long M = static_cast<unsigned long long>(fr * 16777216.f);
    const unsigned __int128 P = static_cast<unsigned __int128>(W) * M;
    const int s = 24 - e;  // >= 24
    if (s >= 128) {
        *rest = P != 0;
        return 0ull;
    }
    const unsigned __int128 q = P >> s;
    *rest = (q << s) != P;
    return static_cast<unsigned long long>(q);
}

}  // namespace vocab
}  // namespace spec
