/* Host check of the int8 codes' quotient: for a row with amax = max |y| and
 * s = fl32(amax / 127), r = fl32(1 / s), the value fma(fma(-q0, s, y), r, q0)
 * with q0 = fl32(y * r), clamped to +-127, must round to the same whole number
 * (nearest, ties to even) as the correctly rounded quotient fl32(y / s).
 * Checked for every positive normal bf16 amax >= 2^-64 (smaller ones take the
 * division on the device) taken with the given stride, and every bf16 y with
 * 0 <= y <= amax; a negative y mirrors a positive one.
 *   usage: int8_quotient_check [amax stride, default 1 = every amax]
 * Prints the counts; exits 1 on any mismatch. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static float bf16(uint32_t bits)
{
    const uint32_t u = bits << 16;
    float f;
    memcpy(&f, &u, 4);
    return f;
}

int main(int argc, char** argv)
{
    const unsigned stride = argc > 1 ? (unsigned)atoi(argv[1]) : 1u;
    long long pairs = 0, bad = 0;
    for (uint32_t ab = 0x0080; ab < 0x7F80; ab += stride) {
        volatile float amax = bf16(ab);
        if (!(amax >= 0x1p-64f)) continue;
        volatile float s = amax / 127.0f;
        volatile float r = 1.0f / s;
        for (uint32_t yb = 0; yb <= ab; ++yb) {
            volatile float y = bf16(yb);
            volatile float exact = y / s;
            volatile float q0 = y * r;
            volatile float e = fmaf(-q0, s, y);
            volatile float q = fmaf(e, r, q0);
            const float code = rintf(q > 127.0f ? 127.0f : q);
            ++pairs;
            if (code != rintf(exact) || code > 127.0f) {
                if (bad < 5) printf("amax %a y %a: y/s %a, quotient %a\n", (double)amax, (double)y, (double)exact, (double)q);
                ++bad;
            }
        }
    }
    printf("pairs %lld mismatches %lld\n", pairs, bad);
    return bad != 0;
}
