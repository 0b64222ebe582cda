// group_norm.hip -- group normalisation with an activation on channels-last
// activations: forward, forward quantised to 8 bits for each pixel, backward.
//
//   For image n and group g, over its m = P * C/G values (P = H * W pixels):
//     mean = sum(x) / m,  var = sum((x - mean)^2) / m,  rstd = 1 / sqrt(var + eps)
//     xh = (x - mean) * rstd,  z = xh * gamma[c] + beta[c],  y = act(z)
//   Backward, with dz = dy * act'(z):
//     dbeta[c] = sum dz,  dgamma[c] = sum dz * xh          (over images and pixels)
//     s1 = sum(gamma * dz) / m,  s2 = sum(gamma * dz * xh) / m   (over the group)
//     dx = rstd * (gamma * dz - s1 - xh * s2)
//
// Two launches each.  The first reads the activations once and leaves partial
// statistics per image, chunk of pixels and group in the workspace; the
// second combines an image's partials (a few KB, from L2) in every workgroup,
// then reads the activations again and writes the result.  No atomics: every
// sum has a fixed order.
//
// Every thread keeps V consecutive channels (16 bytes where the channel count
// and the alignment allow) and walks down the pixels of its chunk, R rows of
// threads side by side, so its per-channel constants stay in registers and a
// row of threads reads whole consecutive lines.
//
// Statistics in fp32: a thread sums x - k and (x - k)^2 with k its first
// value of the channel, which bounds the cancellation in M2 = ss - s^2/n by
// the (small) count of its values whatever the mean is; partial means and M2
// are then merged by the exact identity
//   M2 = sum(M2_i) + sum(n_i * (mean_i - mean)^2).
#include "rowvec.hpp"

namespace conv2d {

namespace {

constexpr int kUnroll = 8;      // vector loads in flight per thread
constexpr int kTargetBlocks = 2048;
constexpr int kMaxChunks = 128; // partials that the second launch combines per image

// Values of row r of R in a chunk of np pixels.
__device__ __forceinline__ int row_count(int np, int R, int r) { return np / R + (r < np % R ? 1 : 0); }

// Lanes that work on one group together: a power of two, at most 64, such
// that the block covers all G groups in one go where it can.
__device__ __forceinline__ int lanes_per_group(int G) {
    int L = 64;
    while (L > 1 && (int)blockDim.x / L < G) L >>= 1;
    return L;
}

// Combines an image's chunk partials (mean, M2) into mean and rstd in LDS.
__device__ __forceinline__ void combine_stats(const float2* part, const NormArgs& a, int n, int chunks, int pix,
                                              float2* stat) {
    const int cg = a.C / a.G, L = lanes_per_group(a.G), lane = threadIdx.x % L;
    const float last = (float)(a.P - (chunks - 1) * pix) * cg, full = (float)pix * cg;
    const float total = (float)a.P * cg;
    for (int g = threadIdx.x / L; g < a.G; g += blockDim.x / L) {
        const float2* p = part + (long long)n * chunks * a.G + g;
        float s = 0.0f;
        for (int j = lane; j < chunks; j += L) s += (j == chunks - 1 ? last : full) * p[(long long)j * a.G].x;
        const float mean = lanes_sum(s, L) / total;
        float m2 = 0.0f;
        for (int j = lane; j < chunks; j += L) {
            const float2 e = p[(long long)j * a.G];
            const float d = e.x - mean;
            m2 += e.y + (j == chunks - 1 ? last : full) * d * d;
        }
        m2 = lanes_sum(m2, L);
        if (lane == 0) stat[g] = make_float2(mean, 1.0f / sqrtf(m2 / total + a.eps));
    }
    __syncthreads();
}

// First launch of the forward pass: (mean, M2) of every group of one chunk.
// One workgroup per image and chunk; LDS: R * C pairs.
template <typename T, int V>
__global__ __launch_bounds__(512) void gn_stats_kernel(NormArgs a, int TX, int R, int chunks, int pix, float2* part) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int tx = threadIdx.x % TX, r = threadIdx.x / TX;
    const int p0 = chunk * pix, np = min(pix, a.P - p0);
    const T* x = static_cast<const T*>(a.x) + ((long long)n * a.P + p0) * a.ldx;
    const long long step = (long long)R * a.ldx;
    if (r < R) {
        const int cnt = row_count(np, R, r);
        for (int c = tx * V; c < a.C; c += TX * V) {
            const T* p = x + r * (long long)a.ldx + c;
            float k[V], s[V], ss[V];
#pragma unroll
            for (int j = 0; j < V; ++j) k[j] = s[j] = ss[j] = 0.0f;
            if (cnt > 0) Vec<T, V>::unpack(Vec<T, V>::load(p), k);
            int i = 0;
            for (; i + kUnroll <= cnt; i += kUnroll) {
                typename Vec<T, V>::raw raw[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) raw[u] = Vec<T, V>::load(p + u * step);
                p += kUnroll * step;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float v[V];
                    Vec<T, V>::unpack(raw[u], v);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float d = v[j] - k[j];
                        s[j] += d;
                        ss[j] = fmaf(d, d, ss[j]);
                    }
                }
            }
            for (; i < cnt; ++i, p += step) {
                float v[V];
                Vec<T, V>::unpack(Vec<T, V>::load(p), v);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = v[j] - k[j];
                    s[j] += d;
                    ss[j] = fmaf(d, d, ss[j]);
                }
            }
            const float inv = cnt > 0 ? 1.0f / cnt : 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = s[j] * inv, m2 = ss[j] - s[j] * d;
                lds[r * a.C + c + j] = make_float2(k[j] + d, m2 < 0.0f ? 0.0f : m2);  // a NaN stays
            }
        }
    }
    __syncthreads();
    const int cg = a.C / a.G, L = lanes_per_group(a.G), lane = threadIdx.x % L;
    for (int g = threadIdx.x / L; g < a.G; g += blockDim.x / L) {
        float s = 0.0f;
        for (int e = lane; e < R * cg; e += L) {
            const int er = e / cg;
            s += row_count(np, R, er) * lds[er * a.C + g * cg + e % cg].x;
        }
        const float mean = lanes_sum(s, L) / ((float)np * cg);
        float m2 = 0.0f;
        for (int e = lane; e < R * cg; e += L) {
            const int er = e / cg;
            const float2 v = lds[er * a.C + g * cg + e % cg];
            const float d = v.x - mean;
            m2 += v.y + row_count(np, R, er) * d * d;
        }
        m2 = lanes_sum(m2, L);
        if (lane == 0) part[(long long)blockIdx.x * a.G + g] = make_float2(mean, m2);
    }
}

// A thread's constants for its V channels.
template <int V> struct Affine {
    float mean[V], rg[V], beta[V];   // z = (x - mean) * (rstd * gamma) + beta
    __device__ __forceinline__ void load(const NormArgs& a, const float2* stat, int c) {
        const int cg = a.C / a.G;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 s = stat[(c + j) / cg];
            mean[j] = s.x;
            rg[j] = s.y * (a.gamma ? a.gamma[c + j] : 1.0f);
            beta[j] = a.beta ? a.beta[c + j] : 0.0f;
        }
    }
    __device__ __forceinline__ float z(float x, int j) const { return fmaf(x - mean[j], rg[j], beta[j]); }
};

__device__ __forceinline__ void save_stats(const NormArgs& a, const float2* stat, int n) {
    for (int g = threadIdx.x; g < a.G; g += blockDim.x) {
        if (a.mean) a.mean[(long long)n * a.G + g] = stat[g].x;
        if (a.rstd) a.rstd[(long long)n * a.G + g] = stat[g].y;
    }
}

// Second launch of the forward pass: one workgroup per image and piece of
// opix pixels.  LDS: G pairs.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(512) void gn_apply_kernel(NormArgs a, int TX, int R, int chunks, int pix, int pieces, int opix,
                                const float2* part) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / pieces, piece = blockIdx.x % pieces;
    combine_stats(part, a, n, chunks, pix, lds);
    if (piece == 0) save_stats(a, lds, n);
    const int tx = threadIdx.x % TX, r = threadIdx.x / TX;
    if (r >= R) return;
    const int p0 = piece * opix, np = min(opix, a.P - p0);
    const long long first = (long long)n * a.P + p0 + r;
    const int cnt = row_count(np, R, r);
    const long long xs = (long long)R * a.ldx, ys = (long long)R * a.ldy;
    for (int c = tx * V; c < a.C; c += TX * V) {
        Affine<V> f;
        f.load(a, lds, c);
        const T* p = static_cast<const T*>(a.x) + first * a.ldx + c;
        T* q = static_cast<T*>(a.y) + first * a.ldy + c;
        for (int i = 0; i < cnt; i += 4) {
            typename Vec<T, V>::raw raw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u < cnt) raw[u] = Vec<T, V>::load(p + u * xs);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i + u >= cnt) break;
                float v[V];
                Vec<T, V>::unpack(raw[u], v);
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = activate<ACT>(f.z(v[j], j));
                Vec<T, V>::store(q + u * ys, v);
            }
            p += 4 * xs;
            q += 4 * ys;
        }
    }
}

// Second launch of the quantised forward pass.  LPP lanes (a power of two)
// share a pixel, lane l holds the vectors l, l + LPP, ... of it, J of them at
// most; with J = 0 a pixel's vectors do not fit the registers and are read
// twice.  LDS: G pairs, then mean, rstd * gamma and beta of every channel.
template <typename T, int V, int ACT, int J>
__global__ __launch_bounds__(256) void gn_quant_kernel(NormArgs a, int LPP, int chunks, int pix, int pieces, int opix,
                                                       const float2* part) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / pieces, piece = blockIdx.x % pieces;
    combine_stats(part, a, n, chunks, pix, lds);
    if (piece == 0) save_stats(a, lds, n);
    float* mean = reinterpret_cast<float*>(lds + a.G);
    float* rg = mean + a.C;
    float* beta = rg + a.C;
    const int cg = a.C / a.G;
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        const float2 s = lds[c / cg];
        mean[c] = s.x;
        rg[c] = s.y * (a.gamma ? a.gamma[c] : 1.0f);
        beta[c] = a.beta ? a.beta[c] : 0.0f;
    }
    __syncthreads();
    const int l = threadIdx.x % LPP, sub = threadIdx.x / LPP, subs = blockDim.x / LPP;
    const int p0 = piece * opix, np = min(opix, a.P - p0);
    auto value = [&](float x, int c) { return activate<ACT>(fmaf(x - mean[c], rg[c], beta[c])); };
    for (int i = sub; i < np; i += subs) {
        const long long pixel = (long long)n * a.P + p0 + i;
        const T* p = static_cast<const T*>(a.x) + pixel * a.ldx;
        int8_t* q = static_cast<int8_t*>(a.y) + pixel * a.ldy;
        uint32_t top = 0;
        if constexpr (J > 0) {
            float v[J][V];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (l + j * LPP) * V;
                if (c < a.C) Vec<T, V>::unpack(Vec<T, V>::load(p + c), v[j]);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (l + j * LPP) * V;
                if (c >= a.C) break;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[j][e] = value(v[j][e], c + e);
                    top = max(top, __float_as_uint(v[j][e]) & 0x7fffffffu);
                }
            }
            const RowScale s = row_scale(lanes_max(top, LPP));
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (l + j * LPP) * V;
                if (c < a.C) store_quantised<V>(q + c, v[j], s.inv);
            }
            if (l == 0) a.q_scale[pixel] = s.scale;
        } else {
            for (int c = l * V; c < a.C; c += LPP * V) {
                float v[V];
                Vec<T, V>::unpack(Vec<T, V>::load(p + c), v);
#pragma unroll
                for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(value(v[e], c + e)) & 0x7fffffffu);
            }
            const RowScale s = row_scale(lanes_max(top, LPP));
            for (int c = l * V; c < a.C; c += LPP * V) {
                float v[V];
                Vec<T, V>::unpack(Vec<T, V>::load(p + c), v);
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = value(v[e], c + e);
                store_quantised<V>(q + c, v, s.inv);
            }
            if (l == 0) a.q_scale[pixel] = s.scale;
        }
    }
}

// dz = dy * act'(z).  ReLU's derivative at 0 is 0.
template <int ACT> __device__ __forceinline__ float act_grad(float dy, float z) {
    if (ACT == kActRelu) return z > 0.0f ? dy : z <= 0.0f ? 0.0f : z;  // a NaN stays
    if (ACT == kActSilu) {
        const float e = sigmoid(z);
        return dy * (e * fmaf(z, 1.0f - e, 1.0f));
    }
    return dy;
}

template <int V> struct BwdCoef {
    float mean[V], rstd[V], gamma[V], beta[V];
    __device__ __forceinline__ void load(const NormArgs& a, int n, int c) {
        const int cg = a.C / a.G;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const long long g = (long long)n * a.G + (c + j) / cg;
            mean[j] = a.mean[g];
            rstd[j] = a.rstd[g];
            gamma[j] = a.gamma ? a.gamma[c + j] : 1.0f;
            beta[j] = a.beta ? a.beta[c + j] : 0.0f;
        }
    }
};

// First launch of the backward pass: for every image and chunk the sums of dz
// and dz * xh per channel (pc: [block][2][C]) and, weighted with gamma, per
// group (pg).  LDS: R * C pairs.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(512) void gn_bwd_sums_kernel(NormArgs a, int TX, int R, int chunks, int pix, float* pc, float2* pg) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int tx = threadIdx.x % TX, r = threadIdx.x / TX;
    const int p0 = chunk * pix, np = min(pix, a.P - p0);
    if (r < R) {
        const int cnt = row_count(np, R, r);
        const long long first = (long long)n * a.P + p0 + r;
        const long long xs = (long long)R * a.ldx, ds = (long long)R * a.lddy;
        for (int c = tx * V; c < a.C; c += TX * V) {
            BwdCoef<V> f;
            f.load(a, n, c);
            const T* px = static_cast<const T*>(a.x) + first * a.ldx + c;
            const T* pd = static_cast<const T*>(a.dy) + first * a.lddy + c;
            float A[V], B[V];
#pragma unroll
            for (int j = 0; j < V; ++j) A[j] = B[j] = 0.0f;
            for (int i = 0; i < cnt; i += 4) {
                typename Vec<T, V>::raw rx[4], rd[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i + u < cnt) {
                        rx[u] = Vec<T, V>::load(px + u * xs);
                        rd[u] = Vec<T, V>::load(pd + u * ds);
                    }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i + u >= cnt) break;
                    float x[V], d[V];
                    Vec<T, V>::unpack(rx[u], x);
                    Vec<T, V>::unpack(rd[u], d);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float xh = (x[j] - f.mean[j]) * f.rstd[j];
                        const float dz = act_grad<ACT>(d[j], fmaf(xh, f.gamma[j], f.beta[j]));
                        A[j] += dz;
                        B[j] = fmaf(dz, xh, B[j]);
                    }
                }
                px += 4 * xs;
                pd += 4 * ds;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) lds[r * a.C + c + j] = make_float2(A[j], B[j]);
        }
    }
    __syncthreads();
    // rows into row 0: the sums of the channels
    float* out = pc + (long long)blockIdx.x * 2 * a.C;
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        float2 s = lds[c];
        for (int k = 1; k < R; ++k) {
            s.x += lds[k * a.C + c].x;
            s.y += lds[k * a.C + c].y;
        }
        out[c] = s.x;
        out[a.C + c] = s.y;
        const float g = a.gamma ? a.gamma[c] : 1.0f;
        lds[c] = make_float2(s.x * g, s.y * g);
    }
    __syncthreads();
    const int cg = a.C / a.G, L = lanes_per_group(a.G), lane = threadIdx.x % L;
    for (int g = threadIdx.x / L; g < a.G; g += blockDim.x / L) {
        float s = 0.0f, t = 0.0f;
        for (int e = lane; e < cg; e += L) {
            s += lds[g * cg + e].x;
            t += lds[g * cg + e].y;
        }
        s = lanes_sum(s, L);
        t = lanes_sum(t, L);
        if (lane == 0) pg[(long long)blockIdx.x * a.G + g] = make_float2(s, t);
    }
}

constexpr int kParamChannels = 32;  // channels of one workgroup that sums dgamma and dbeta

// Second launch of the backward pass.  The first `sums` workgroups add the
// channels' partials into dgamma and dbeta, the others write dx, one per
// image and piece of opix pixels.  LDS: max(G, blockDim.x) pairs.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(512) void gn_bwd_apply_kernel(NormArgs a, int TX, int R, int chunks, int pieces, int opix, int sums,
                                    const float* pc, const float2* pg) {
    extern __shared__ float2 lds[];
    if ((int)blockIdx.x < sums) {
        const int c = blockIdx.x * kParamChannels + threadIdx.x % kParamChannels;
        const int row = threadIdx.x / kParamChannels, rows = blockDim.x / kParamChannels;
        const long long count = (long long)a.N * chunks;
        float s = 0.0f, t = 0.0f;
        if (c < a.C) {
            const float* p = pc + c;
#pragma unroll 4
            for (long long i = row; i < count; i += rows) {
                s += p[i * 2 * a.C];
                t += p[i * 2 * a.C + a.C];
            }
        }
        lds[threadIdx.x] = make_float2(s, t);
        __syncthreads();
        if (row == 0 && c < a.C) {
            for (int k = 1; k < rows; ++k) {
                s += lds[k * kParamChannels + threadIdx.x].x;
                t += lds[k * kParamChannels + threadIdx.x].y;
            }
            if (a.dbeta) a.dbeta[c] = s;
            if (a.dgamma) a.dgamma[c] = t;
        }
        return;
    }
    const int b = blockIdx.x - sums;
    const int n = b / pieces, piece = b % pieces;
    const int cg = a.C / a.G;
    {
        const int L = lanes_per_group(a.G), lane = threadIdx.x % L;
        const float inv = 1.0f / ((float)a.P * cg);
        for (int g = threadIdx.x / L; g < a.G; g += blockDim.x / L) {
            const float2* p = pg + (long long)n * chunks * a.G + g;
            float s = 0.0f, t = 0.0f;
            for (int j = lane; j < chunks; j += L) {
                const float2 e = p[(long long)j * a.G];
                s += e.x;
                t += e.y;
            }
            s = lanes_sum(s, L);
            t = lanes_sum(t, L);
            if (lane == 0) lds[g] = make_float2(s * inv, t * inv);
        }
        __syncthreads();
    }
    const int tx = threadIdx.x % TX, r = threadIdx.x / TX;
    if (r >= R) return;
    const int p0 = piece * opix, np = min(opix, a.P - p0);
    const long long first = (long long)n * a.P + p0 + r;
    const int cnt = row_count(np, R, r);
    const long long xs = (long long)R * a.ldx, ds = (long long)R * a.lddy, os = (long long)R * a.ldy;
    for (int c = tx * V; c < a.C; c += TX * V) {
        BwdCoef<V> f;
        f.load(a, n, c);
        float s1[V], s2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 s = lds[(c + j) / cg];
            s1[j] = s.x;
            s2[j] = s.y;
        }
        const T* px = static_cast<const T*>(a.x) + first * a.ldx + c;
        const T* pd = static_cast<const T*>(a.dy) + first * a.lddy + c;
        T* po = static_cast<T*>(a.y) + first * a.ldy + c;
        for (int i = 0; i < cnt; i += 2) {
            typename Vec<T, V>::raw rx[2], rd[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (i + u < cnt) {
                    rx[u] = Vec<T, V>::load(px + u * xs);
                    rd[u] = Vec<T, V>::load(pd + u * ds);
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (i + u >= cnt) break;
                float x[V], d[V];
                Vec<T, V>::unpack(rx[u], x);
                Vec<T, V>::unpack(rd[u], d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (x[j] - f.mean[j]) * f.rstd[j];
                    const float dz = act_grad<ACT>(d[j], fmaf(xh, f.gamma[j], f.beta[j]));
                    d[j] = f.rstd[j] * (fmaf(f.gamma[j], dz, -s1[j]) - xh * s2[j]);
                }
                Vec<T, V>::store(po + u * os, d);
            }
            px += 2 * xs;
            pd += 2 * ds;
            po += 2 * os;
        }
    }
}

// ------------------------------------------------------------------ host

// Elements of one vector access: the most that divides the channel count and
// every row stride, up to 16 bytes, with every pointer aligned to it.
int vector_width(const NormArgs& a, int elem, int out_elem) {
    int v = 16 / elem;
    auto ok = [&](const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; };
    while (v > 1 && !(a.C % v == 0 && a.ldx % v == 0 && a.ldy % v == 0 && (!a.dy || a.lddy % v == 0) &&
                      ok(a.x, v * elem) && ok(a.y, v * out_elem) && ok(a.dy, v * elem)))
        v >>= 1;
    return v;
}

struct Plan {
    int TX, R, block, chunks, pix, pieces, opix;
};

// Threads: TX across the channel vectors, R rows of them, the block size of
// 256 to 512 that leaves the fewest idle.  Chunks: about kTargetBlocks
// workgroups in all, at most kMaxChunks per image, at least 4 pixels a thread.
Plan make_plan(int N, int P, int C, int V) {
    Plan p;
    const int cv = C / V;
    p.TX = cv < 256 ? cv : 256;
    int best = 0;
    p.block = 256;
    for (int b = 256; b <= 512; b += 64) {
        const int used = b / p.TX * p.TX * 4096 / b;
        if (used > best) best = used, p.block = b;
    }
    p.R = p.block / p.TX;
    auto split = [&](int target, int most, int least, int* count, int* size) {
        long long k = (target + (long long)N - 1) / N;
        const long long cap = (P + (long long)p.R * least - 1) / ((long long)p.R * least);
        k = k < cap ? k : cap;
        k = k < most ? k : most;
        k = k < 1 ? 1 : k;
        const long long each = (P + k - 1) / k;
        *size = (int)((each + p.R - 1) / p.R * p.R);
        *count = (int)((P + (long long)*size - 1) / *size);
    };
    split(kTargetBlocks, kMaxChunks, 4, &p.chunks, &p.pix);
    split(kTargetBlocks, 1 << 20, 4, &p.pieces, &p.opix);
    return p;
}

template <typename T, int V> hipError_t forward(const NormArgs& a, int act, void* ws, hipStream_t st) {
    const Plan p = make_plan(a.N, a.P, a.C, V);
    float2* part = static_cast<float2*>(ws);
    gn_stats_kernel<T, V><<<a.N * p.chunks, p.block, (size_t)p.R * a.C * 8, st>>>(a, p.TX, p.R, p.chunks, p.pix, part);
    auto k = act == kActSilu ? gn_apply_kernel<T, V, kActSilu>
             : act == kActRelu ? gn_apply_kernel<T, V, kActRelu> : gn_apply_kernel<T, V, kActNone>;
    k<<<a.N * p.pieces, p.block, (size_t)a.G * 8, st>>>(a, p.TX, p.R, p.chunks, p.pix, p.pieces, p.opix, part);
    return hipGetLastError();
}

template <typename T, int V, int ACT> hipError_t quantised_apply(const NormArgs& a, const Plan& p, const float2* part,
                                                                 hipStream_t st) {
    const int cv = a.C / V;
    int lpp = 1;
    while (lpp < cv && lpp < 64) lpp <<= 1;
    const int j = (cv + lpp - 1) / lpp;
    auto k = j == 1 ? gn_quant_kernel<T, V, ACT, 1> : j == 2 ? gn_quant_kernel<T, V, ACT, 2>
             : j <= 4 ? gn_quant_kernel<T, V, ACT, 4> : gn_quant_kernel<T, V, ACT, 0>;
    const size_t lds = (size_t)a.G * 8 + (size_t)a.C * 12;
    k<<<a.N * p.pieces, 256, lds, st>>>(a, lpp, p.chunks, p.pix, p.pieces, p.opix, part);
    return hipGetLastError();
}

template <typename T, int V> hipError_t quantised(const NormArgs& a, int act, void* ws, hipStream_t st) {
    const Plan p = make_plan(a.N, a.P, a.C, V);
    float2* part = static_cast<float2*>(ws);
    gn_stats_kernel<T, V><<<a.N * p.chunks, p.block, (size_t)p.R * a.C * 8, st>>>(a, p.TX, p.R, p.chunks, p.pix, part);
    return act == kActSilu ? quantised_apply<T, V, kActSilu>(a, p, part, st)
           : act == kActRelu ? quantised_apply<T, V, kActRelu>(a, p, part, st)
                             : quantised_apply<T, V, kActNone>(a, p, part, st);
}

template <typename T, int V, int ACT> hipError_t backward_act(const NormArgs& a, void* ws, hipStream_t st) {
    const Plan p = make_plan(a.N, a.P, a.C, V);
    const long long blocks = (long long)a.N * p.chunks;
    float2* pg = static_cast<float2*>(ws);
    float* pc = reinterpret_cast<float*>(pg + blocks * a.G);
    gn_bwd_sums_kernel<T, V, ACT><<<(int)blocks, p.block, (size_t)p.R * a.C * 8, st>>>(a, p.TX, p.R, p.chunks, p.pix,
                                                                                      pc, pg);
    const int sums = a.dgamma || a.dbeta ? (a.C + kParamChannels - 1) / kParamChannels : 0;
    const size_t lds = (size_t)(a.G > p.block ? a.G : p.block) * 8;
    gn_bwd_apply_kernel<T, V, ACT><<<sums + a.N * p.pieces, p.block, lds, st>>>(a, p.TX, p.R, p.chunks, p.pieces,
                                                                               p.opix, sums, pc, pg);
    return hipGetLastError();
}

template <typename T, int V> hipError_t backward(const NormArgs& a, int act, void* ws, hipStream_t st) {
    return act == kActSilu ? backward_act<T, V, kActSilu>(a, ws, st)
           : act == kActRelu ? backward_act<T, V, kActRelu>(a, ws, st) : backward_act<T, V, kActNone>(a, ws, st);
}

}  // namespace

// The most partials that any vector width plans, so that one figure holds for
// every alignment.
size_t group_norm_workspace(int N, int P, int C, int G, int backward) {
    size_t most = 0;
    for (int v = 1; v <= 8; v <<= 1) {
        if (C % v) break;
        const Plan p = make_plan(N, P, C, v);
        const size_t bytes = (size_t)N * p.chunks * (G + (backward ? (size_t)C : 0)) * 8;
        most = bytes > most ? bytes : most;
    }
    return most;
}

// Grids are one-dimensional: the largest must fit 2^31 - 1 workgroups.
bool group_norm_supports(int N, int P, int C) {
    for (int v = 1; v <= 8; v <<= 1) {
        if (C % v) break;
        const Plan p = make_plan(N, P, C, v);
        if ((long long)N * p.chunks + C >= 0x7fffffffLL || (long long)N * p.pieces + C >= 0x7fffffffLL) return false;
    }
    return true;
}

#define CONV2D_NORM_DISPATCH(FN, OUT_ELEM)                                            \
    if (a.dtype == 0 /* CONV2D_F32 */) {                                              \
        const int v = vector_width(a, 4, OUT_ELEM ? OUT_ELEM : 4);                    \
        return v == 4 ? FN<float, 4>(a, act, ws, st)                                  \
               : v == 2 ? FN<float, 2>(a, act, ws, st) : FN<float, 1>(a, act, ws, st); \
    }                                                                                 \
    const int v = vector_width(a, 2, OUT_ELEM ? OUT_ELEM : 2);                        \
    return v == 8 ? FN<bf16_t, 8>(a, act, ws, st) : v == 4 ? FN<bf16_t, 4>(a, act, ws, st) \
           : v == 2 ? FN<bf16_t, 2>(a, act, ws, st) : FN<bf16_t, 1>(a, act, ws, st)

hipError_t launch_group_norm(const NormArgs& a, int act, void* ws, hipStream_t st) {
    CONV2D_NORM_DISPATCH(forward, 0);
}

hipError_t launch_group_norm_quant(const NormArgs& a, int act, void* ws, hipStream_t st) {
    CONV2D_NORM_DISPATCH(quantised, 1);
}

hipError_t launch_group_norm_bwd(const NormArgs& a, int act, void* ws, hipStream_t st) {
    CONV2D_NORM_DISPATCH(backward, 0);
}

}  // namespace conv2d
