// Memory and undefined-behaviour check of the host side of the operators (group
// norm, rows in 8 bits, int8 products): workspace sizes, and the argument checks
// with the plans behind them, over a sweep of valid, invalid and extreme sizes.
// Every call of an entry is one that the entry refuses (a workspace of no bytes,
// a missing pointer, a size out of range): nothing touches a GPU.
#include <climits>
#include <cstdio>

#include "conv2d.h"

int main() {
    static char d[64] __attribute__((aligned(64))) = {};
    float* const f = reinterpret_cast<float*>(d);
    long calls = 0, sized = 0, accepted = 0;
    const int dtypes[] = {CONV2D_F32, CONV2D_BF16, 7};
    const int Ns[] = {-1, 0, 1, 2, 513, 70000, 1 << 24, INT_MAX};
    const int Cs[] = {-8, 0, 1, 7, 16, 130, 512, 4095, 4096, 4097, INT_MAX};
    const int Hs[] = {-1, 0, 1, 5, 112, 4100, 1 << 16, INT_MAX / 2, INT_MAX};
    const int Gs[] = {-1, 0, 1, 2, 16, 4096, INT_MAX};
    for (int N : Ns) for (int C : Cs) for (int H : Hs) for (int W : Hs) for (int G : Gs) {
        for (int backward : {0, 1}) sized += conv2d_group_norm_workspace_bytes(N, C, H, W, G, backward) > 0;
        for (int dt : dtypes) for (int ld : {C, INT_MAX}) {
            const int r[] = {
                conv2d_group_norm_nhwc(d, f, f, d, f, f, d, 0, N, C, H, W, G, ld, ld, 1e-5f, dt, CONV2D_ACT_SILU, nullptr),
                conv2d_group_norm_quant_nhwc(d, f, f, d + 16, f, f, f, d, 0, N, C, H, W, G, ld, ld, 1e-5f, dt, CONV2D_ACT_RELU,
                                             nullptr),
                conv2d_group_norm_bwd_nhwc(d, d, f, f, f, f, d, f, f, d, 0, N, C, H, W, G, ld, ld, ld, dt, CONV2D_ACT_NONE,
                                           nullptr)};
            for (int v : r) accepted += v >= 0;
            calls += 3;
        }
    }
    const int Ms[] = {-1, 0, 1, 64, 65, 100, 4100, 1 << 24, (1 << 29) - 1, 1 << 29, (1 << 29) + 1, INT_MAX - 511, INT_MAX};
    const int Ks[] = {-1, 0, 1, 16, 17, 512, 8192, 131071, 131072, INT_MAX};
    const int Os[] = {-1, 0, 1, 16, 65, 1000, 1 << 16, 1 << 27, (1 << 27) + 1, INT_MAX};
    for (int M : Ms) for (int K : Ks) for (int N : Os) {
        const bool need = conv2d_int8_matmul_workspace_bytes(M, K, N) > 0;
        sized += need;
        for (int dt : dtypes) for (int ld : {K, (1 << 22) + 1, INT_MAX}) {
            // refused for the bias, and where a workspace is needed or a stride
            // too long after the plans too
            accepted += conv2d_int8_matmul(d, f, d, f, nullptr, d, d, 0, M, K, N, ld, ld, N, dt, CONV2D_EPI_BIAS, nullptr) >= 0;
            if (need || ld > 1 << 22)
                accepted += conv2d_int8_matmul(d, f, d, f, nullptr, d, d, 0, M, K, N, ld, ld, N, dt, 0, nullptr) >= 0;
            accepted += conv2d_quantize_rows(d, d, f, M, K, ld, ld, dt, nullptr) >= 0;   // over its input
            calls += 3;
        }
    }
    std::printf("operators sanitize ok: %ld calls, %ld sizes\n", calls, sized);
    return accepted == 0 && sized > 0 ? 0 : 1;
}
