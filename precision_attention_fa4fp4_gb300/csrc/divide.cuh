// divide.cuh -- division by a Divisor on the device.
#pragma once
#include "common.cuh"
#include "rope.h"

namespace fa4 {

FA4_DEV int divide(int n, const Divisor& by) { return (int)((__umulhi((uint32_t)n, by.m) + (uint32_t)n) >> by.s); }
FA4_DEV void divide(int n, const Divisor& by, int& q, int& r) {
  q = divide(n, by);
  r = n - q * by.d;
}

}  // namespace fa4
