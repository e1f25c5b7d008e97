// Host side of moe_add_norm: how the rows lie, and the kernels of x's type (add_norm.cuh, one file
// for each type).
#include "layer.cuh"

namespace moe {

namespace {

// Of a matrix (size: bytes of an element): may its rows lie on a grid of eight elements whose
// place the first matrix's stride gives?
bool on_grid(const void *p, int64_t stride, int size, int rows, int stride8) {
    return !p || (((uintptr_t)p % (size == 1 ? 8 : 16)) == 0 && (rows == 1 || (stride & 7) == stride8));
}
int size_of(int type) { return type == MOE_T_F32 ? 4 : 2; }

}  // namespace

cudaError_t launch_add_norm(AddNormArgs a, int sms, cudaStream_t s) {
    const int n = a.rows;
    a.stride8 = n == 1 ? 0 : (int)(a.x.stride & 7);
    Grid grid = Grid::kNone;
    if (on_grid(a.x.p, a.x.stride, size_of(a.x.type), n, a.stride8) &&
        on_grid(a.residual.p, a.residual.stride, size_of(a.residual.type), n, a.stride8) &&
        on_grid(a.residual_out.p, a.residual_out.stride, size_of(a.residual.type), n, a.stride8) &&
        on_grid(a.out.p, a.out.stride, size_of(a.out.type), n, a.stride8) &&
        on_grid(a.weight, 0, 2, 1, 0) && on_grid(a.codes, a.codes_stride, 1, n, a.stride8))
        grid = a.hidden % 8 == 0 && a.stride8 == 0 ? Grid::kVectors : Grid::kEnds;
    if (a.x.type == MOE_T_BF16) return add_norm_of<MOE_T_BF16>(a, grid, sms, s);
    if (a.x.type == MOE_T_F16) return add_norm_of<MOE_T_F16>(a, grid, sms, s);
    return add_norm_of<MOE_T_F32>(a, grid, sms, s);
}

}  // namespace moe
