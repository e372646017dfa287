// weight.cuh -- softmax weights as whole numbers: 2^((l - m) c) in units of
// 2^-U, each right to 2^-37 of itself and 0.8 units, in fp32 arithmetic alone.
//
// A draw picks the token at a border of a sum over the whole row, and top-p cuts
// the order at another, so a weight's error moves the choice wherever tokens are
// small: with 10^4 tokens in play, weights right to 2^-22 (one ex2.approx) would
// pick another token than the definition for about one row in a hundred.  GB300's
// FP64 pipe issues two FMAs a clock per SM, so an exp in double costs a row of
// 150 k logits over a millisecond; pairs of floats take about 75 instructions.  Sums of whole numbers do not
// depend on their order.  A row's sum stays below 2^63, so its length sets U: a sum over N tokens may be
// off by 0.8 N units (2^-24 of the largest weight for 524288 tokens, 2^-32 for 32000), all in one
// direction where the tokens are equal.
//
// x = (l - m) c is kept as a pair (TwoSum of l and -m, products with their FMA
// remainders), x = n + t/128 + g with |g| <= 1/256, and
//   2^x = 2^n T[t] (1 + E),  E = e^y - 1,  y = g ln 2,  |y| < 0.0028,
// T from a table of float pairs, E by its Taylor series: y as a pair, y^2/2 + y^3/6
// in fp32 (below 2^-18, so its rounding is below 2^-42; y^4/24 is below 2^-38).
#pragma once

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

namespace spec {
namespace vocab {

#ifdef __CUDACC__
#define SPEC_HD __host__ __device__ __forceinline__
#else
#define SPEC_HD inline
#endif

constexpr int kPow2Steps = 128, kPow2Bits = 7;
// 2^(t/128) as a float and the remainder.
#define SPEC_POW2_TABLE                                                                                        \
    {                                                                                                          \
        {0x1.0p+0f, 0x0.0p+0f}, {0x1.0163dap+0f, 0x1.3f6666p-25f}, {0x1.02c9a4p+0f, -0x1.887fap-28f},          \
        {0x1.04315ep+0f, 0x1.0dcffp-25f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0706b2p+0f, 0x1.3bbedcp-25f}, \
        {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.09e3ecp+0f, 0x1.58de7p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, \
        {0x1.0cc922p+0f, 0x1.6e48fep-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f}, {0x1.0fb66ap+0f, 0x1.ffda64p-25f}, \
        {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.12abdcp+0f, 0x1.b0c73p-30f}, {0x1.1429aap+0f, 0x1.d525bcp-25f}, \
        {0x1.15a98cp+0f, 0x1.14b1cap-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.18af94p+0f, -0x1.dcdc86p-26f}, \
        {0x1.1a35bep+0f, 0x1.6df96ep-25f}, {0x1.1bbe08p+0f, 0x1.011734p-26f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, \
        {0x1.1ed502p+0f, 0x1.7e6c8ep-27f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f}, {0x1.21f49ap+0f, -0x1.d0446ep-25f}, \
        {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.251ce4p+0f, 0x1.f654c8p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f}, \
        {0x1.284dfep+0f, 0x1.f5638p-28f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f}, {0x1.2b87fep+0f, -0x1.e4a4cep-25f}, \
        {0x1.2d285ap+0f, 0x1.b900c2p-26f}, {0x1.2ecafap+0f, 0x1.27c5eap-25f}, {0x1.306fep+0f, 0x1.4636e2p-25f}, \
        {0x1.32171p+0f, -0x1.d993e8p-27f}, {0x1.33c08cp+0f, -0x1.b37d2p-25f}, {0x1.356c56p+0f, -0x1.b5803cp-30f}, \
        {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.38cae6p+0f, 0x1.a0bb0cp-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f}, \
        {0x1.3c32dcp+0f, 0x1.89d472p-27f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.3fa45p+0f, 0x1.2b2006p-26f}, \
        {0x1.4160a2p+0f, 0x1.f72e2ap-28f}, {0x1.431f5ep+0f, -0x1.abd5dap-26f}, {0x1.44e086p+0f, 0x1.8624b4p-30f}, \
        {0x1.46a41ep+0f, 0x1.a3a00ap-25f}, {0x1.486a2cp+0f, -0x1.47d866p-25f}, {0x1.4a32bp+0f, -0x1.e50584p-25f}, \
        {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4dcb2ap+0f, -0x1.8088bcp-26f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f}, \
        {0x1.516daap+0f, 0x1.67b32p-27f}, {0x1.5342b6p+0f, -0x1.2c561p-25f}, {0x1.551a4cp+0f, 0x1.4bb242p-25f}, \
        {0x1.56f474p+0f, -0x1.295b04p-25f}, {0x1.58d12ep+0f, -0x1.6d07p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, \
        {0x1.5c9268p+0f, 0x1.4b28d6p-25f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f}, {0x1.605e1cp+0f, -0x1.a248fep-26f}, \
        {0x1.6247ecp+0f, -0x1.f8b55p-25f}, {0x1.643464p+0f, -0x1.66679cp-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f}, \
        {0x1.68155ep+0f, -0x1.766ad2p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.6c0128p+0f, -0x1.5e84a8p-25f}, \
        {0x1.6dfb24p+0f, -0x1.cd72e8p-27f}, {0x1.6ff7ep+0f, -0x1.ab9aep-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, \
        {0x1.73f9a4p+0f, 0x1.14b02ep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f}, {0x1.780694p+0f, 0x1.fbcba8p-25f}, \
        {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.7c1edp+0f, 0x1.30c132p-28f}, {0x1.7e2f34p+0f, -0x1.261634p-25f}, \
        {0x1.804276p+0f, -0x1.783cbep-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8471a4p+0f, 0x1.88f1ecp-26f}, \
        {0x1.868d9ap+0f, -0x1.2edb44p-26f}, {0x1.88ac7ep+0f, -0x1.9d665ap-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f}, \
        {0x1.8cf322p+0f, -0x1.29576ep-25f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f}, {0x1.9145bp+0f, 0x1.723ff8p-25f}, \
        {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.95a44cp+0f, 0x1.790a42p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f}, \
        {0x1.9a0f18p+0f, -0x1.e6bf08p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.9e8632p+0f, -0x1.873738p-26f}, \
        {0x1.a0c668p+0f, -0x1.2886a6p-26f}, {0x1.a309bep+0f, 0x1.8945a6p-25f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f}, \
        {0x1.a799e2p+0f, -0x1.99e994p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f}, {0x1.ac36bcp+0f, -0x1.606432p-31f}, \
        {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b0e072p+0f, 0x1.31b6ccp-25f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f}, \
        {0x1.b59728p+0f, 0x1.bcab28p-25f}, {0x1.b7f77p+0f, -0x1.a09438p-25f}, {0x1.ba5b04p+0f, -0x1.ebdf36p-25f}, \
        {0x1.bcc1eap+0f, -0x1.f687c6p-25f}, {0x1.bf2c26p+0f, -0x1.0a387ep-26f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, \
        {0x1.c40ab6p+0f, -0x1.7c2c98p-39f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f}, {0x1.c8f6dap+0f, -0x1.7f230ap-25f}, \
        {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.cdf0b6p+0f, -0x1.54478p-25f}, {0x1.d072d4p+0f, 0x1.40f13p-25f}, \
        {0x1.d2f87p+0f, 0x1.01b13ep-25f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.d80e32p+0f, -0x1.26cf8ep-25f}, \
        {0x1.da9e6p+0f, 0x1.ed9942p-27f}, {0x1.dd322p+0f, -0x1.9fc974p-25f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, \
        {0x1.e26462p+0f, -0x1.614bdap-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f}, {0x1.e7a52p+0f, -0x1.0e2cep-26f}, \
        {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.ecf482p+0f, 0x1.b1ccfep-25f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f}, \
        {0x1.f252b4p+0f, -0x1.1288aep-25f}, {0x1.f50766p+0f, -0x1.246ebp-26f}, {0x1.f7bfdap+0f, 0x1.b397c2p-25f}, \
        {0x1.fa7c18p+0f, 0x1.9e90d8p-28f}, {0x1.fd3c22p+0f, 0x1.71ee3ep-25f}                                   \
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

SPEC_HD int float_bits(float f) {
#ifdef __CUDA_ARCH__
    return __float_as_int(f);
#else
    int b;
    memcpy(&b, &f, 4);
    return b;
#endif
}

// What turns a row's logits into weights: the row maximum m, c = log2(e) / T as a pair, U.
struct Scale {
    float m;
    float ch, cl;
    int U;  // units of 2^-U; U + bits(V) <= 62, so that a row's sum stays below 2^63, and U <= 48 (fixed_weight)
};

// Branch-free, so that a vector's logits go through it side by side.  Weights below 2^least are 0 (-60: below
// half a unit for every U of a row); least + U > -100, so that the scale is a normal number.
SPEC_HD unsigned long long fixed_weight(float logit, const Scale &s, const float2 *pow2, float least = -60.f) {
    const bool some = (logit - s.m) * s.ch > least;  // not: logit = -inf
    const float l = some ? logit : s.m;
    const float dh = l - s.m;
    const float ph = dh * s.ch;
    const float bb = dh - l;
    const float dl = (l - (dh - bb)) + (-s.m - bb);
    float pl = fmaf(dh, s.ch, -ph);
    pl = fmaf(dh, s.cl, pl);
    pl = fmaf(dl, s.ch, pl);
    const float shifted = fmaf(ph, 128.f, 0x1.8p23f);  // its last bits are the nearest whole number to 128 ph
    const int j = float_bits(shifted) - 0x4b400000;
    const float gx = fmaf(shifted - 0x1.8p23f, -0x1p-7f, ph);  // exact: both are multiples of ph's last place
    const float g = gx + pl;                                   // |pl| reaches 2^-18: left apart, y^3/6 would miss it
    const float gl = pl - (g - gx);
    constexpr float kLn2h = 0x1.62e430p-1f, kLn2l = -0x1.05c610p-29f;
    const float yh = g * kLn2h;
    float yl = fmaf(g, kLn2h, -yh);
    yl = fmaf(g, kLn2l, yl);
    yl = fmaf(gl, kLn2h, yl);
    const float el = fmaf(yh * yh, fmaf(yh, 1.f / 6.f, 0.5f), yl);
    const float2 T = pow2[j & (kPow2Steps - 1)];
    const float qh = T.x * yh;
    const float ql = fmaf(T.x, el, fmaf(T.y, yh, fmaf(T.x, yh, -qh)));
    const float wh = T.x + qh;
    const float wl = (qh - (wh - T.x)) + (T.y + ql);
    // wh + wl in units of 2^-U as (whole multiple of 2^22) + rest: scaled by a power of two, so exactly
    const int e = (j >> kPow2Bits) + s.U - 22;                 // in [-41, 26]: |wl| < 2^-17 keeps lo below 2^31
    const float up = bits_float((e + 127) << 23);
    const float t = wh * up;
    const uint32_t hi = static_cast<uint32_t>(t);
    const float rest = (t - static_cast<float>(hi)) + wl * up;  // exact, then one rounding
    const int lo = static_cast<int>(rintf(rest * 0x1p22f));
    const unsigned long long v = (static_cast<unsigned long long>(hi) << 22) + static_cast<long long>(lo);
    return some ? v : 0ull;
}

// Whether a logit's weight is at least f, in (0, 1]: in units of 2^-40 of f's own size, so right to 2^-37 of f
// however small it is.
SPEC_HD bool weight_reaches(float l, const Scale &s, float f, const float2 *pow2) {
    int k = 0;
    const float fr = frexpf(f, &k);  // f = fr 2^k, fr in [0.5, 1)
    const float x = (l - s.m) * s.ch, size = static_cast<float>(k);
    if (!(x > size - 2.f)) return false;
    if (x > size + 1.f) return true;
    Scale near = s;
    near.U = 40 - k;
    return fixed_weight(l, near, pow2, size - 3.f) >= static_cast<unsigned long long>(fr * 16777216.f) << 16;
}

// A finite logit below every one that lies at most `depth` under the largest, m: below the difference's own
// error.  (Not -inf, which masked tokens and the padding of a row's vectors reach.)
SPEC_HD float logit_under(float m, float depth) { return fmaxf(m - depth - (fabsf(depth) + fabsf(m)) * 0x1p-18f, -FLT_MAX); }

// floor(W * f) for W < 2^63 and f in [0, 1), and whether f * W is no whole number, exactly.
SPEC_HD unsigned long long scaled_floor(unsigned long long W, float f, bool *rest) {
    int e = 0;
    const float fr = frexpf(f, &e);  // f = fr 2^e, fr in [0.5, 1), e <= 0
    const unsigned long long M = static_cast<unsigned long long>(fr * 16777216.f);
    const int s = 24 - e;  // >= 24; the product W M, above and below 2^32:
    const unsigned long long low = (W & 0xffffffffull) * M, A = (W >> 32) * M + (low >> 32);
    const uint32_t r = static_cast<uint32_t>(low);
    if (s < 32) {
        *rest = (r & ((1u << s) - 1)) != 0;
        return (A << (32 - s)) + (r >> s);
    }
    if (s >= 96) {
        *rest = W != 0 && M != 0;
        return 0ull;
    }
    const unsigned long long q = A >> (s - 32);
    *rest = r != 0 || (q << (s - 32)) != A;
    return q;
}

}  // namespace vocab
}  // namespace spec
