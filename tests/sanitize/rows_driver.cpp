// Memory and undefined-behaviour check of the host side of the row operators (RMS
// norm, products with an epilogue and their gradients, dropout): workspace sizes, and
// the argument checks with the plans behind them, over a sweep of valid, invalid and
// extreme sizes.  Every call of an entry is one that the entry refuses: nothing
// touches a GPU.
#include <climits>
#include <cstdio>

#include "conv2d.h"

int main() {
    static char d[256] __attribute__((aligned(64))) = {};
    float* const f = reinterpret_cast<float*>(d);
    const auto* const rng = reinterpret_cast<const unsigned long long*>(d);
    long calls = 0, sized = 0, accepted = 0;
    const int dtypes[] = {CONV2D_F32, CONV2D_BF16, 7};
    const int Ms[] = {-1, 0, 1, 2, 33, 777, 4100, 100352, 1 << 24, (1 << 30) - 1, 1 << 30, INT_MAX};
    const int Cs[] = {-8, 0, 1, 7, 16, 130, 1001, 4096, 16384, 16385, INT_MAX};
    for (int M : Ms) for (int C : Cs) {
        sized += conv2d_rms_norm_bwd_workspace_bytes(M, C) > 0;
        for (int dt : dtypes) for (int ld : {C, INT_MAX}) {
            // outputs over each other or over their input, a missing workspace, p out of range
            const int r[] = {conv2d_rms_norm(d, d + 64, f, d + 128, d + 128, f, M, C, ld, ld, ld, ld, 1e-5f, dt, nullptr),
                             conv2d_rms_norm_quant(d, nullptr, f, nullptr, d, f, f, M, C, ld, ld, ld, ld, 1e-5f, dt, nullptr),
                             conv2d_rms_norm_bwd(d, nullptr, d + 64, f, f, d + 128, f, d, 0, M, C, ld, ld, ld, ld, dt, nullptr),
                             conv2d_dropout(d, nullptr, d + 64, rng, 1.0f, M, C, ld, ld, ld, dt, nullptr)};
            for (int v : r) accepted += v >= 0;
            calls += 4;
        }
    }
    const int Ks[] = {-1, 0, 1, 15, 16, 1001, 8192, 1 << 20, (1 << 20) + 1, INT_MAX};
    const int Ns[] = {-1, 0, 1, 16, 65, 517, 16384, 1 << 20, INT_MAX};
    for (int M : Ms) for (int K : Ks) for (int N : Ns) for (int dt : dtypes) {
        sized += conv2d_matmul_workspace_bytes(M, K, N, dt) > 0;
        sized += conv2d_matmul_bwd_workspace_bytes(M, K, N, dt) > 0;
        for (int act : {-1, (int)CONV2D_ACT_NONE, (int)CONV2D_ACT_GELU, 4}) {
            // refused at the latest for z over y, and for a workspace of no bytes
            accepted += conv2d_matmul(d, d + 64, f, nullptr, d + 128, d + 128, d, 0, M, K, N, K, K, N, N, N, dt, act, nullptr) >= 0;
            if (conv2d_matmul_workspace_bytes(M, K, N, dt))
                accepted += conv2d_matmul(d, d + 64, f, nullptr, nullptr, d + 128, d, 0, M, K, N, K, K, N, N, N, dt, act, nullptr) >= 0;
            accepted += conv2d_matmul_bwd(d, d + 64, d + 128, d + 192, d + 32, d + 96, nullptr, d, 0, M, K, N, N, N, K, K, K, K, dt, act, nullptr) >= 0;
            calls += 3;
        }
    }
    std::printf("rows sanitize ok: %ld calls, %ld sizes\n", calls, sized);
    return accepted == 0 && sized > 0 ? 0 : 1;
}
