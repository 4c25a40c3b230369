/* The kernels that quantize fp32 results divide by the group's scale as
 *   q = x * r,  e = fma(q, s, -x),  y = fma(e, -r, q)
 * with r = 1 / s. This program checks that the code of y is the code of the IEEE quotient x / s for
 * fp32 x and s of any mantissa. A code changes only where the quotient passes a midpoint of two codes
 * (or reaches it: a tie), and every midpoint of e4m3, its subnormals included, is a power of two times
 * an odd number below 32, of int8 an odd half below 127, so an odd number o below 256 times a power of
 * two. In the range where the kernels use this form nothing is subnormal, and a power of two changes no
 * rounding: it is enough to take s in [1, 2) and x around s * o, and to compare on which side of o (or
 * on it) y and the rounded quotient are. Both are within 2 steps of the exact quotient, a step of x
 * moves it by half a step at least, so 5 steps of x on each side of s * o decide.
 *
 * The scale max(amax, eps) / Qmax is formed the same way from the constant r = 1 / Qmax; for it every
 * mantissa of amax is compared with the IEEE quotient.
 *
 * Usage: quotient_codes_fp32 STRIDE OFFSET: the mantissas OFFSET, OFFSET + STRIDE, ... (STRIDE 1: all).
 * Prints the number of mismatches (0 expected).
 * Build: gcc -O2 -fopenmp -ffp-contract=off quotient_codes_fp32.c -lm */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static float from_bits(uint32_t u) {
    float f;
    memcpy(&f, &u, sizeof f);
    return f;
}
static uint32_t bits(float f) {
    uint32_t u;
    memcpy(&u, &f, sizeof u);
    return u;
}
static int side(float v, float o) { return (v > o) - (v < o); }

int main(int argc, char** argv) {
    const long stride = argc > 1 ? atol(argv[1]) : 1, offset = argc > 2 ? atol(argv[2]) : 0;
    long long bad = 0;
#pragma omp parallel for schedule(dynamic, 1024) reduction(+ : bad)
    for (long m = offset; m < (1L << 23); m += stride) {
        const float s = from_bits(0x3F800000u | (uint32_t)m), r = 1.0f / s;
        for (int o = 1; o < 256; o += 2) {
            const uint32_t mid = bits((float)((double)s * o));
            for (int d = -5; d <= 5; ++d) {
                const float x = from_bits(mid + (uint32_t)d);
                const float q = x * r, e = fmaf(q, s, -x), y = fmaf(e, -r, q);
                bad += side(y, (float)o) != side(x / s, (float)o);
            }
        }
        for (int i = 0; i < 2; ++i) {
            const float z = i ? -0.0f : 0.0f, qz = z * r;             /* zeros keep their sign */
            bad += bits(fmaf(fmaf(qz, s, -z), -r, qz)) != bits(z);
            const float qmax = i ? 127.0f : 448.0f, c = 1.0f / qmax, q = s * c;
            bad += fmaf(fmaf(-q, qmax, s), c, q) != s / qmax;
        }
    }
    printf("%lld\n", bad);
    return 0;
}
