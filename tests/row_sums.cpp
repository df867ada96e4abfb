// What a row's attention comes to (csrc/row_sums.h) as C functions, for tests/test_row_sums.py.
#include "row_sums.h"

extern "C" {
float lse_at_end(int gave_up, float m, float l) {
  const okv::RowSums s = okv::sums_at_end(gave_up != 0, m, l);
  return okv::lse_of(s.m, s.l);
}
int draws(float lse) { return okv::draws(lse); }
}
