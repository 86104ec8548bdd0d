"""The quotient max / 6 that an NVFP4 block's scale is rounded from, on the host:
csrc/fp4_scale.h compiled by itself and compared with exact integers."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "fp4_scale.h"

// a float >= 0 to E4M3 as a count of its steps, ties to even: steps of 2^-9 up to 2^-6, then 8 a binade
static int steps_of(double v) {
    int e = 0;
    const double m = frexp(v, &e);                       // v = m 2^e, 0.5 <= m < 1
    const int k = e < -5 ? -9 : e - 4;                   // the step is 2^k
    const double r = nearbyint(ldexp(v, -k));
    return v == 0 || m == 0 ? 0 : (int)r + (k + 9) * 8;  // (a carry into the next binade is its first step)
}

// the same of t / 6 without forming it: the count n nearest to t / 6, by t against 6 middles (exact in doubles)
static int steps_of_sixth(float t) {
    int n = steps_of((double)t / 6.0);
    for (int c = n > 0 ? n - 1 : 0; c <= n + 1; ++c) {
        // value of count c
        double lo, hi;
        const int b = c / 8;
        lo = b == 0 ? ldexp(c, -9) : ldexp(8 + c % 8, b - 10);
        const int d = c + 1, bd = d / 8;
        hi = bd == 0 ? ldexp(d, -9) : ldexp(8 + d % 8, bd - 10);
        const double mid6 = 3.0 * (lo + hi);
        if ((double)t < mid6 || ((double)t == mid6 && c % 2 == 0)) return c;
    }
    return -1;
}

int main() {
    long bad = 0, bad_short = 0, off = 0;
    // every float whose sixth lies in the binades of E4M3 around 1, and those around every middle in all of them
    for (uint32_t u = 0; u < (1u << 23); ++u) {
        const uint32_t bits = (127u + 2u) << 23 | u;
        float t;
        memcpy(&t, &bits, 4);
        const float q = moe::fp4_sixth(t);
        bad += steps_of(q) != steps_of_sixth(t);
        // to nearest: 6 q is within 3 units in the last place of q of t (exact in doubles)
        off += fabs((double)q * 6 - (double)t) > 3 * ldexp(1.0, ilogb(q) - 23);
    }
    for (int c = 0; c < 127; ++c) {
        const int b = c / 8, d = c + 1, bd = d / 8;
        const double lo = b == 0 ? ldexp(c, -9) : ldexp(8 + c % 8, b - 10);
        const double hi = bd == 0 ? ldexp(d, -9) : ldexp(8 + d % 8, bd - 10);
        float t = (float)(3 * (lo + hi));
        for (int i = 0; i < 64; ++i) t = nextafterf(t, 0.f);
        for (int i = 0; i < 129; ++i, t = nextafterf(t, 1e9f)) bad += steps_of(moe::fp4_sixth(t)) != steps_of_sixth(t);
    }
    // values of up to 11 significant bits
    for (int m = 1024; m < 2048; ++m)
        for (int e = -24; e <= 1; ++e) {
            const float t = ldexpf((float)m, e);
            if (t <= 2688) bad_short += steps_of(moe::fp4_sixth_of_short(t)) != steps_of_sixth(t);
        }
    printf("%ld %ld %ld\n", bad, off, bad_short);
    return 0;
}
"""


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    d = tmp_path_factory.mktemp("fp4_scale")
    src, exe = d / "t.cpp", d / "t"
    src.write_text(PROGRAM)
    # (no contraction: a product and a sum stay two roundings, as written)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-I",
                    os.path.join(ROOT, "top_moe_expert_router_gb300", "csrc"), str(src), "-o", str(exe), "-lm"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, check=True)
    return [int(v) for v in r.stdout.split()]


def test_scales_of_any_float(counts):
    """silu(x) * up has 24 significant bits: no scale differs from that of the exact quotient, ties to even."""
    assert counts[0] == 0


def test_quotients_are_the_nearest(counts):
    assert counts[1] == 0


def test_scales_of_short_values(counts):
    """Elements of 16 bits have 11 significant bits or fewer."""
    assert counts[2] == 0
