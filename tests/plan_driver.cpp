// plan_driver.cpp -- the products' plans (csrc/matmul_plan.hpp) for tests/test_matmul_plan_host.py.
#include "matmul_plan.hpp"

extern "C" {

// tile, parts of the sum and stages of a part
void plan_tiles(int rows, int cols, int K, int es, int aligned, int* out) {
    const conv2d::Plan p = conv2d::make_plan(rows, cols, K, es, aligned != 0);
    out[0] = p.b;
    out[1] = p.splits;
    out[2] = p.stages;
}

// taken, blocks of 16 rows, of 16 columns, steps of a wave
void plan_few_rows(int rows, int cols, int K, int es, int* out) {
    const conv2d::SkinnyShape k = conv2d::skinny_shape(rows, cols, K, es);
    out[0] = k.fits;
    out[1] = k.two ? 2 : 1;
    out[2] = k.pairs ? 2 : 1;
    out[3] = (int)k.steps;
}

int plan_copies(int M, int K, int N, int es, int forward) {
    return forward ? conv2d::packs_forward(M, K, N, es) : conv2d::packs(M, K, N, es);
}

}
