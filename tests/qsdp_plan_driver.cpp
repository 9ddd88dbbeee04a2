// The plan of a tiled product with coded weights, for the tests: host code of the library's header.
#include "qsdp_plan.h"

extern "C" void qsdp_plan(int64_t tokens, int64_t width, int64_t depth, int grad, int64_t *out) {
    const onebit::TilePlan p = onebit::tile_plan(tokens, width, depth, grad != 0);
    const onebit::PlannedShape &s = onebit::kPlannedShapes[p.shape];
    const int64_t all[] = {p.shape, p.tiles_m, p.tiles_n, p.splits, s.tm, s.tn};
    std::copy(all, all + 6, out);
}
