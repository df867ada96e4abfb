// The order of a ring's uses (csrc/ring.h) as C functions, for tests/test_ring_order.py.
#include "ring.h"

using One = okv::RingOrder<1>;
using Two = okv::RingOrder<2>;

extern "C" {
int32_t key(int32_t s, int32_t i) { return s == 1 ? One::key(i) : Two::key(i); }
int32_t value(int32_t s, int32_t i) { return s == 1 ? One::value(i) : Two::value(i); }
int32_t may_be_on_its_way(int32_t s, int32_t use, int32_t ring, int32_t keys, int32_t values) {
  return s == 1 ? One::may_be_on_its_way(use, ring, keys, values) : Two::may_be_on_its_way(use, ring, keys, values);
}
}
