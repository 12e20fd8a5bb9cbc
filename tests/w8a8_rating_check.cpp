// What csrc/w8a8_plan.h rates its plan for M N K at, us (host code).
#include <cstdio>
#include <cstdlib>

#include "w8a8_plan.h"

int main(int, char** argv) {
  const qact::W8Plan p = qact::w8_plan(std::atoll(argv[1]), std::atoll(argv[2]), std::atoll(argv[3]), (size_t)64 << 20);
  std::printf("%.3f\n", p.us);
  return 0;
}
