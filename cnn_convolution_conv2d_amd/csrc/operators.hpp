// operators.hpp -- what the C entries and the kernels of the operators beside the
// convolutions share (group norm, rows in 8 bits, int8 products).  Apart from
// common.hpp, which every convolution kernel's measured traffic is tied to.
#pragma once

#include "common.hpp"

namespace conv2d {

// One group-norm call on channels-last data, validated on the host.  P pixels
// per image; ld*: elements from one pixel to the next.  y is the output: the
// activations, their 8-bit form (then q_scale holds a scale per pixel) or dx.
struct NormArgs {
    const void* x;
    const void* dy;        // backward only
    const float* gamma;    // null: 1
    const float* beta;     // null: 0
    void* y;
    float* q_scale;
    float* mean;           // [N][G]; forward: written unless null, backward: read
    float* rstd;
    float* dgamma;         // backward only; null: not wanted
    float* dbeta;
    int N, P, C, G;
    long long ldx, ldy, lddy;
    float eps;
    int dtype;             // CONV2D_F32 / CONV2D_BF16
};

// One int8 product, validated on the host: q [M][K], w [N][K], y [M][N], with
// ld*: elements from one row to the next.
struct Int8Args {
    const int8_t* q;
    const int8_t* w;
    const float* q_scale;
    const float* w_scale;
    const float* bias;     // null: none
    void* y;
    int M, K, N;
    long long ldq, ldw, ldy;
    bool relu;
};

// Looks at another workgroup's result before a workgroup computes it itself, set
// by conv2d_set_wait_limit.
int wait_limit();

// Group norm: the bytes of workspace and the three passes (one to four launches
// each; act: CONV2D_ACT_*).
size_t group_norm_workspace(int N, int P, int C, int G, int backward);
hipError_t launch_group_norm(const NormArgs& a, int act, void* ws, hipStream_t st);
hipError_t launch_group_norm_quant(const NormArgs& a, int act, void* ws, hipStream_t st);
hipError_t launch_group_norm_bwd(const NormArgs& a, int act, void* ws, hipStream_t st);

// 8-bit integer products.
size_t int8_matmul_workspace(int M, int K, int N);
bool int8_matmul_supports(int M, int K, int N, long long ldq, long long ldw);
hipError_t launch_int8_matmul(const Int8Args& a, int out_f32, void* ws, hipStream_t st);
hipError_t launch_quantize_rows(const void* x, void* q, float* scale, int M, int K, long long ldx, long long ldq,
                                int dtype, hipStream_t st);

}  // namespace conv2d
