// operators.hpp -- what the C entries and the kernels of the operators beside the
// convolutions share (norms, rows in 8 bits, products, dropout).  Apart from
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

// One RMS-norm call on rows, validated on the host: M rows of C, ld*: elements
// from one row to the next.
struct RmsArgs {
    const void* x;         // backward: dy
    const void* residual;  // null: none; backward: dh
    const float* gamma;    // null: 1
    void* h;               // x + residual, null: not wanted; backward: read
    void* y;               // the norm, its 8-bit form or dx
    float* q_scale;        // with the 8-bit form
    float* rstd;           // [M]; forward: written unless null, backward: read
    float* dgamma;         // backward only; null: not wanted
    int M, C;
    long long ldx, ldr, ldh, ldy;
    float eps;
    int dtype;
};

// One product with its epilogue, validated on the host:
// y [M][N] = act(z) + residual, z = x [M][K] w [N][K]^T + bias.
struct MatmulArgs {
    const void* x;
    const void* w;
    const float* bias;     // null: none
    const void* residual;  // null: none
    void* z;               // null: not wanted
    void* y;
    int M, K, N;
    long long ldx, ldw, ldr, ldz, ldy;
    int dtype, act;
};

// Its gradients: dz = dy act'(z), dx = dz w, dw = dz^T x, dbias = sum_m dz.
struct MatmulBwdArgs {
    const void* dy;
    const void* z;         // null: the activation is none
    const void* x;
    const void* w;
    void* dx;              // each of the three: null: not wanted
    void* dw;
    float* dbias;
    int M, K, N;
    long long lddy, ldz, ldx, ldw, lddx, lddw;
    int dtype, act;
};

// One dropout call, validated on the host.
struct DropoutArgs {
    const void* x;
    const void* residual;             // null: none
    void* y;
    const unsigned long long* rng;    // seed, offset
    uint32_t threshold;               // words below it drop their element
    float scale;
    int M, C;
    long long ldx, ldr, ldy;
    int dtype;
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

// RMS norm; C up to kRmsMostC.
constexpr int kRmsMostC = 16384;
size_t rms_norm_bwd_workspace(int M, int C);
hipError_t launch_rms_norm(const RmsArgs& a, hipStream_t st);
hipError_t launch_rms_norm_quant(const RmsArgs& a, hipStream_t st);
hipError_t launch_rms_norm_bwd(const RmsArgs& a, void* ws, hipStream_t st);

// out[c] = sum of sums[i][c] over i < count, in fp64, in a fixed order; C up to 2^20.
hipError_t launch_join_columns(const float* sums, float* out, int count, int C, hipStream_t st);

// Products with an epilogue and their gradients; strides of what they read up to kMatmulMostLd.
constexpr int kMatmulMostLd = 1 << 20;
bool matmul_supports(int M, int K, int N);
size_t matmul_workspace(int M, int K, int N, int dtype);
size_t matmul_bwd_workspace(int M, int K, int N, int dtype);
hipError_t launch_matmul(const MatmulArgs& a, void* ws, hipStream_t st);
hipError_t launch_matmul_bwd(const MatmulBwdArgs& a, void* ws, hipStream_t st);

// Dropout.
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st);

}  // namespace conv2d
