// exp_coefs.hpp -- the constants of the routing scores' fp64 exponential
// (score_kernels.hpp).  Plain C++: a host program checks the steps with them.
#pragma once

namespace moe {

// e^r = 1 + r + r^2 q(r) for |r| <= ln2 / 2: q of degree 9, from the highest
// power down, interpolates (e^r - 1 - r) / r^2 at the 10 Chebyshev nodes of
// that range (worked out to 60 digits), its constant coefficient rounded to
// 1/2.  It is off by less than 2^-55 of e^r; the Taylor sum of as many terms,
// by 2^-46.7.
constexpr int kExpTerms = 10;
constexpr double kExpQ[kExpTerms] = {
    0x1.af38a9b0ec855p-26, 0x1.289185613a3d6p-22, 0x1.71de0dae63bb3p-19, 0x1.a019b90d2ae7ap-16, 0x1.a01a01a7c41d5p-13,
    0x1.6c16c1788bd90p-10, 0x1.11111111109b3p-7,  0x1.5555555553d63p-5,  0x1.5555555555556p-3,  0.5};

constexpr double kExpLog2E = 0x1.71547652b82fep+0;
// ln2 = kExpLn2 + kExpLn2Low, to 2^-110
constexpr double kExpLn2 = 0x1.62e42fefa39efp-1;
constexpr double kExpLn2Low = 0x1.abc9e3b39803fp-56;

}  // namespace moe
