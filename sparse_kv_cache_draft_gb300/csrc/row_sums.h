// What a row's attention comes to, from its maximum and its sum of weights. For the kernels, and for a host compiler.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define OKV_SUMS_FN __host__ __device__ __forceinline__
#else
#define OKV_SUMS_FN inline
#endif

namespace okv {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kMaxFinite = 3.402823466e38f;

struct RowSums {
  float m, l;  // the largest score, in log2 units (-infinity: none), and the sum of 2^(score - m)
};

// A maximum that takes in another one: at most the largest finite number. A score of infinity then has an infinite weight and makes
// the sum infinite, where the difference of two infinities would be no number, as that of a score that is none; against it every finite
// score's weight is zero.
OKV_SUMS_FN float larger_max(float m, float other) { return fminf(fmaxf(m, other), kMaxFinite); }

// Of a block in which a wait ran out: what its rows have so far may be anything, so they count as rows that see nothing.
OKV_SUMS_FN RowSums sums_at_end(bool gave_up, float m, float l) { return gave_up ? RowSums{-INFINITY, 0.f} : RowSums{m, l}; }

// log sum exp(score), -infinity for a row that sees nothing.
OKV_SUMS_FN float lse_of(float m, float l) { return l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2; }

// Whether a row of this log sum draws anything from what it sees: 2^(score - lse log2(e)) has no meaning for one that sees nothing.
OKV_SUMS_FN bool draws(float lse) { return lse != -INFINITY; }

}  // namespace okv
