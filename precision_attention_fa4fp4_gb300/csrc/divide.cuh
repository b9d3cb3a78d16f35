// divide.cuh -- division by a Divisor on the device, and the order of dependent
// grids.
#pragma once
#include "common.cuh"
#include "rope.h"

namespace fa4 {

// The next grid of the stream may start; what the grids before this one wrote is
// there (of a grid that was launched early).
FA4_DEV void next_may_start() { asm volatile("griddepcontrol.launch_dependents;"); }
FA4_DEV void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

FA4_DEV int divide(int n, const Divisor& by) { return (int)((__umulhi((uint32_t)n, by.m) + (uint32_t)n) >> by.s); }
FA4_DEV void divide(int n, const Divisor& by, int& q, int& r) {
  q = divide(n, by);
  r = n - q * by.d;
}

}  // namespace fa4
