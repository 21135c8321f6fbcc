/* Host check of the routing scores' exponential: its steps, with the constants
 * the kernel uses, against the long double exponential of the C library (64
 * bits of mantissa, off by less than 2^-63).
 * Error bound of the steps, relative to e^x: q(r) 2^-55; r, rounded twice in
 * (-0.35, 0.35), 2 * 2^-55; r q' + 1, in (0.8, 1.2), 2^-53 times |r| < 0.35;
 * the last sum, 2^-53: together below 2^-51.8.
 *   usage: exp_f64_check [count of points, default 20000000]
 * Prints log2 of the largest error; exits 1 where it reaches 2^-51.8. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "exp_coefs.hpp"

static double exp_steps(double x)
{
    const double t = fma(x, moe::kExpLog2E, 0x1.8p+52);
    const double n = t - 0x1.8p+52;
    const double r = fma(-n, moe::kExpLn2Low, fma(-n, moe::kExpLn2, x));
    double p = moe::kExpQ[0];
    for (int i = 1; i < moe::kExpTerms; ++i) p = fma(p, r, moe::kExpQ[i]);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}

int main(int argc, char** argv)
{
    const long count = argc > 1 ? atol(argv[1]) : 20000000;
    double most = 0.0, at = 0.0;
    uint64_t s = 88172645463325252ull;
    for (long i = 0; i < count; ++i) {
        s ^= s << 13, s ^= s >> 7, s ^= s << 17;
        // half of the points over [-200, 200], half next to the ends of the
        // reduced range, where q is worst
        double x = (double)(int64_t)s * (200.0 / 9223372036854775808.0);
        if (i & 1) x = (floor(x) + 0.5) * 0.69314718055994531 * (0.999 + 0.002 * ((double)(s >> 40) * 0x1p-24));
        const double e = (double)fabsl((long double)exp_steps(x) / expl((long double)x) - 1.0L);
        if (!(e <= most)) most = e, at = x;
    }
    printf("points %ld largest error 2^%.2f at %a\n", count, log2(most), at);
    return !(most < exp2(-51.8));
}
