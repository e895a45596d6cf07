"""The divisions of the 4-bit cache's write, which are formed from a rounded reciprocal and corrected by the exact
remainder, against IEEE division: every FP32 mantissa of the dividend with every BF16 mantissa of the divisor (host
arithmetic, compiled here; no GPU needed).  Exponents only shift all steps while nothing underflows, which the kernel sees to."""
import ctypes
import subprocess

import pytest

SOURCE = """
#include <cmath>
#include <cstdint>
#include <cstring>
#include <thread>
#include <vector>

static float from_bits(uint32_t b)
{
    float x;
    std::memcpy(&x, &b, 4);
    return x;
}

// q = d inv rounded, plus inv times what is left of d, once rounded
static float corrected(float d, float s, float inv)
{
    const float q = d * inv;
    return std::fmaf(std::fmaf(-q, s, d), inv, q);
}

static int64_t differ(float s)
{
    const float inv = 1.0f / s;
    int64_t n = 0;
    for (uint32_t m = 0; m < 1u << 23; ++m) {
        const float d = from_bits(0x3f800000u | m);
        n += corrected(d, s, inv) != d / s;
    }
    return n;
}

// of all 128 divisors 1, 1 + 2^-7, ... 2 - 2^-7
extern "C" int64_t by_scales()
{
    std::vector<int64_t> n(128);
    std::vector<std::thread> all;
    for (int t = 0; t < 16; ++t)
        all.emplace_back([&n, t] {
            for (uint32_t i = t; i < 128; i += 16)
                n[i] = differ(from_bits(0x3f800000u | i << 16));
        });
    for (auto &t : all)
        t.join();
    int64_t sum = 0;
    for (int64_t x : n)
        sum += x;
    return sum;
}

extern "C" int64_t by_fifteen()
{
    int64_t n = 0;
    for (uint32_t b = 0x3f800000u; b < 0x41800000u; ++b) {  // 1 to 16
        const float x = from_bits(b);
        n += corrected(x, 15.0f, 0.06666667014360428f) != x / 15.0f;
    }
    return n;
}
"""


@pytest.fixture(scope="module")
def so(tmp_path_factory):
    d = tmp_path_factory.mktemp("quotient")
    (d / "q.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-pthread", "-o",
                    str(d / "q.so"), str(d / "q.cpp")], check=True)
    so = ctypes.CDLL(str(d / "q.so"))
    so.by_scales.restype = so.by_fifteen.restype = ctypes.c_int64
    return so


def test_quotients_by_a_scale(so):
    assert so.by_scales() == 0


def test_quotients_by_fifteen(so):
    assert so.by_fifteen() == 0
