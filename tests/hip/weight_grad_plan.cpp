// Which way weight_grad.hip does a product (tests only): the library's own rule.
#include "grad_plan.hpp"

// out: way (0 teams, 1 small tiles, 2 large ones), tiles of n and k, tiles done whole, pieces
// of each other one, bytes of the pieces' sums
extern "C" void weight_grad_plan(int32_t type, int64_t m, int64_t n, int64_t ld, int64_t* out) {
    const flashopt::GradPlan p = flashopt::grad_plan(type, m, n, ld, true);
    const int64_t all[] = {p.way, p.tn, p.tk, p.whole, p.splits, (int64_t)(p.part + p.bias)};
    for (int i = 0; i < 6; ++i) out[i] = all[i];
}
