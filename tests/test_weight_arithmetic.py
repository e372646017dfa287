"""The whole-number softmax weights of the filtered sampler, on the CPU: the same source compiled for
the host, against 80-bit exponentials.

Bound: the dropped terms (y^4 / 24 below 2^-38, the pairs' second remainders) and the roundings below
2^-42 add up to less than 2^-37 relative, plus 0.8 units (fp32 keeps 24 bits of the last 22; then a rounding)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sampling_online_softmax_gb300", "csrc", "vocab")

PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include <random>
struct float2 { float x, y; };
#include "weight.cuh"
using namespace spec::vocab;
static const float2 table[kPow2Steps] = SPEC_POW2_TABLE;
int main() {
    std::mt19937 gen(1);
    std::normal_distribution<float> normal(0, 1);
    double worst = 0;
    for (int t = 0; t < kPow2Steps; ++t)
        worst = fmax(worst, fabsl(((long double)table[t].x + table[t].y) / exp2l((long double)t / kPow2Steps) - 1) * exp2(40));
    for (int i = 0; i < 3000000; ++i) {
        Scale s;
        s.m = fabsf(normal(gen)) * 5 + (i % 3) * 10;
        float l = i % 5 ? s.m - fabsf(normal(gen)) * (i % 7 + 1) * 3 : normal(gen) * exp2f(-(i % 40));
        if (i % 11 == 0) l = s.m;
        if (i % 13 == 0) { s.m = normal(gen) * 1e-3f - 40; l = s.m - fabsf(normal(gen)); }
        if (i % 17 == 0) { unsigned b; memcpy(&b, &l, 4); b &= 0xffff0000u; memcpy(&l, &b, 4); }
        if (l > s.m) l = s.m;
        const float T = i % 19 ? 0.3f + (i % 11) * 0.2f : exp2f(i % 30 - 15);
        constexpr float kH = 0x1.715476p+0f, kL = 0x1.4ae0c0p-26f;
        s.ch = kH / T;
        s.cl = (fmaf(-s.ch, T, kH) + kL) / T;
        s.U = 42 + i % 7;
        const long double e = expl(((long double)l - (long double)s.m) / (long double)T) * exp2l(s.U);
        const double far = fabsl((long double)fixed_weight(l, s, table) - e);
        worst = fmax(worst, (far - 0.8) / (double)e * exp2(40) * (e > 1));
        if (e < 0.25 && fixed_weight(l, s, table) != 0) worst = 1e9;
    }
    Scale s = {3.f, 1.f, 0.f, 48};
    if (fixed_weight(3.f, s, table) != 1ull << 48 || fixed_weight(-INFINITY, s, table) != 0 || fixed_weight(-3e38f, s, table) != 0) worst = 1e9;
    bool rest;
    if (scaled_floor(1000, 0.5f, &rest) != 500 || rest || scaled_floor(1001, 0.5f, &rest) != 500 || !rest || scaled_floor(7, 0.f, &rest) != 0 || rest) worst = 1e9;
    if (scaled_floor(1ull << 61, 1.f - 0x1p-24f, &rest) != (1ull << 61) - (1ull << 37) || rest || scaled_floor(1ull << 61, 0x1p-149f, &rest) != 0 || !rest) worst = 1e9;
    printf("%.3f\n", worst);
    return 0;
}
"""


def test_weights_against_long_doubles(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src = tmp_path / "w.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-ffp-contract=off", "-x", "c++", "-I", CSRC, "-o", str(tmp_path / "w"), str(src)], check=True, capture_output=True)
    worst = float(subprocess.run([str(tmp_path / "w")], capture_output=True, text=True, check=True).stdout)
    assert worst <= 8.0, "a weight is %.3f * 2^-40 off" % worst


UNDER = r"""
#include <cmath>
#include <cstdio>
#include <random>
struct float2 { float x, y; };
#include "weight.cuh"
using namespace spec::vocab;
int main() {
    std::mt19937 gen(2);
    std::uniform_real_distribution<float> draw(-1, 1);
    int wrong = 0;
    const float sizes[] = {0.f, 1e-38f, 1.f, 30.f, 1e9f, 3e37f, 3.3895314e38f, 3.4028e38f, FLT_MAX}, depths[] = {0.f, 1e-6f, 4.f, 150.f, 1e8f, 1e38f, INFINITY};
    for (float m : sizes)
        for (float d : depths)
            for (int i = 0; i < 1000; ++i) {
                const float top = i < 2 ? (i ? m : -m) : m * draw(gen), depth = i % 3 ? d : d * fabsf(draw(gen));
                const float low = logit_under(top, depth);
                // finite, and not above top - depth where that is a logit
                if (!(low >= -FLT_MAX) || (double)low > fmax((double)top - (double)depth, -(double)FLT_MAX)) ++wrong;
            }
    printf("%d\n", wrong);
    return 0;
}
"""


def test_the_bound_under_the_largest_logit_is_finite(tmp_path):
    """Also where the largest is the type's lowest value, as in a row masked by it: -inf would be reached by masked tokens
    and by the padding of a row's vectors, which lie outside the tensor."""
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src = tmp_path / "u.cpp"
    src.write_text(UNDER)
    subprocess.run(["g++", "-O2", "-ffp-contract=off", "-x", "c++", "-I", CSRC, "-o", str(tmp_path / "u"), str(src)], check=True, capture_output=True)
    assert int(subprocess.run([str(tmp_path / "u")], capture_output=True, text=True, check=True).stdout) == 0


REACHES = r"""
#include <cmath>
#include <cstdio>
#include <random>
struct float2 { float x, y; };
#include "weight.cuh"
using namespace spec::vocab;
static const float2 table[kPow2Steps] = SPEC_POW2_TABLE;
int main() {
    std::mt19937 gen(3);
    std::uniform_real_distribution<float> draw(0, 1);
    int wrong = 0, near = 0;
    for (int i = 0; i < 1000000; ++i) {
        Scale s;
        s.m = (draw(gen) - 0.5f) * (i % 3 ? 60.f : 1.f);
        const float T = i % 5 ? 0.3f + draw(gen) : exp2f(i % 30 - 15);
        constexpr float kH = 0x1.715476p+0f, kL = 0x1.4ae0c0p-26f;
        s.ch = kH / T;
        s.cl = (fmaf(-s.ch, T, kH) + kL) / T;
        s.U = 43;
        const float l = s.m - draw(gen) * 103.f * T;
        const long double w = expl(((long double)l - (long double)s.m) / (long double)T);
        float f = (float)w;  // within 2^-24 of the weight, or (below 2^-126) 2^-150; and some further off
        if (i % 7 == 0) f *= 1.f + (draw(gen) - 0.5f) * 0x1p-10f;
        if (i % 11 == 0) f *= 8.f * draw(gen);
        if (i % 13 == 0) f = draw(gen);
        if (!(f > 0.f && f <= 1.f)) continue;
        const long double off = fabsl((long double)f / w - 1);
        if (off <= exp2l(-37)) continue;
        near += off < exp2l(-24);
        wrong += weight_reaches(l, s, f, table) != (w >= (long double)f);
    }
    Scale s = {3.f, 1.f, 0.f, 48};
    if (!weight_reaches(3.f, s, 1.f, table) || weight_reaches(-INFINITY, s, 0x1p-149f, table) || !weight_reaches(-146.f, s, 0x1p-149f, table)) ++wrong;
    if (weight_reaches(-146.00002f, s, 0x1p-149f, table) || weight_reaches(-3e38f, s, 0x1p-149f, table)) ++wrong;
    printf("%d %d\n", wrong, near);
    return 0;
}
"""


def test_which_weights_reach_a_bound_of_any_size(tmp_path):
    """Against 80-bit exponentials, for every bound further than 2^-37 from the weight, down to fp32's smallest."""
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src = tmp_path / "r.cpp"
    src.write_text(REACHES)
    subprocess.run(["g++", "-O2", "-ffp-contract=off", "-x", "c++", "-I", CSRC, "-o", str(tmp_path / "r"), str(src)], check=True, capture_output=True)
    wrong, near = map(int, subprocess.run([str(tmp_path / "r")], capture_output=True, text=True, check=True).stdout.split())
    assert wrong == 0 and near > 100000
