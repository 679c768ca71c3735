"""The quotient of the e4m3 outputs on the host: the product with a rounded
reciprocal, put right by its remainder, is the float32 division's at every
value next to a border of e4m3 (one of 5 significant bits) for every float32
significand of a scale; the product alone is not."""
import shutil
import subprocess

import pytest

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
static float of(uint32_t u) { float x; memcpy(&x, &u, 4); return x; }
static uint32_t bits(float x) { uint32_t u; memcpy(&u, &x, 4); return u; }
int main(void)
{
    long wrong = 0, product_wrong = 0;
#pragma omp parallel for reduction(+ : wrong, product_wrong)
    for (uint32_t m = 0; m < 1u << 23; ++m) {
        const float scale = of(0x3f800000u | m), inv = 1.0f / scale;
        for (int p = 0; p < 16; ++p) {
            const uint32_t middle = bits((1.0f + p / 16.0f) * scale);
            for (int d = -2; d <= 2; ++d) {
                const float v = of(middle + d), q0 = v * inv;
                const float q = fmaf(fmaf(-q0, scale, v), inv, q0);
                wrong += q != v / scale;
                product_wrong += q0 != v / scale;
            }
        }
    }
    printf("%ld %ld\n", wrong, product_wrong);
    return 0;
}
"""


def test_quotient_of_every_scale(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not installed")
    src, exe = tmp_path / "quotient.c", tmp_path / "quotient"
    src.write_text(SOURCE)
    subprocess.run([gcc, "-std=c99", "-O2", "-ffp-contract=off", "-fopenmp", str(src), "-o", str(exe),
                    "-lm"], check=True)
    wrong, product_wrong = map(int, subprocess.run([str(exe)], check=True, capture_output=True,
                                                   text=True, timeout=300).stdout.split())
    assert wrong == 0 and product_wrong > 0
