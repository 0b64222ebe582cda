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
// Three forms.
//
// Streaming, two launches.  The first reads the activations once and leaves
// partial statistics per image, chunk of pixels and group in the workspace;
// the second combines an image's partials (a few KB, from L2) in every
// workgroup, then reads the activations again and writes the result.  (The
// quantised pass of small images: one launch, in which every workgroup takes
// its image's statistics itself.)
//
// Resident, one launch: a workgroup loads one (image, group) whole into
// registers, takes its statistics there and writes the result, so memory is
// read once.  Forward and backward take it where a group fits and is either
// small (latency counts) or has whole 64-byte pieces of every pixel.
//
// Joined, for large tensors of which no workgroup can hold a group: a workgroup
// keeps a chunk of an image in registers and takes the statistics of the
// image's other chunks from the workspace, so memory is read once here too.
// 112x112x128 over 32 images with SiLU 59 us, where streaming takes 71 and the
// bytes alone 42; backward of 56x56x256 over 64 images 103 us for 116 (bytes: 63).
//
// Every sum has a fixed order: equal calls give equal bits.
//
// Every thread keeps V consecutive channels (16 bytes where the channel count
// and the alignment allow) and walks down the pixels of its chunk, R rows of
// threads side by side, so its per-channel constants stay in registers and a
// row of threads reads whole consecutive lines.
//
// Statistics.  Streaming and joined: a thread sums d = x - k and d^2, k its
// first value of the channel, and M2 = sum(d^2) - sum(d)^2 / n; partial means and
// M2 are merged the same way, with d = mean_i - mean_0 weighted by the counts,
// and the M2_i added.  Where what lies first (a channel, a pixel, a chunk) is far
// from the rest, sum(d^2) exceeds M2 by up to the count, and fp32 sums would lose
// as much (196 pixels of 4096 channels, the first one at 300: rstd off by 3e-5):
// the sums are fp64, and each partial result is rounded to fp32 once.  That costs
// 1 to 3% of a large tensor's time (112x112x128 over 32 images 56.7 us for 55.2)
// and up to 1.2 us of a small one's.
// Resident: the mean from an fp64 sum, then the deviations from it in a second
// pass over the registers.
#include "mfma.hpp"
#include "operators.hpp"
#include "rowvec.hpp"

namespace conv2d {

namespace {

constexpr int kBatch = 4;       // vector loads in flight per thread (forward)
constexpr int kBatchBwd = 4;    // of x and of dy each (backward)
constexpr int kTargetBlocks = 512;
constexpr int kMaxChunks = 128; // partials that the second launch combines per image

// x / d for 0 <= x < 2^20, d > 0: (x + 1/2) / d is at least 1 / 2d away from the
// next integer, more than the reciprocal's error can move it.  (The kernels are
// a few KB of code that is fetched anew at every launch, so short code counts
// for small tensors; an integer division is some 25 instructions.)
__device__ __forceinline__ int small_div(int x, int d) {
    return (int)(((float)x + 0.5f) * __builtin_amdgcn_rcpf((float)d));
}

// A thread's part of np pixels that R rows of threads share, thread row r:
// the pixels r, r + R, ...
struct Part {
    int first, cnt;   // first: a pixel inside even if cnt is 0
    __device__ __forceinline__ Part(int np, int R, int r) {
        const int every = np / R;
        cnt = r < R ? every + (r < np - every * R) : 0;
        first = min(r, np - 1);
    }
};

// 1 / n to 2^-45 of itself: the hardware's reciprocal and one Newton step (the
// division is three times the code).
__device__ __forceinline__ double inverse(double n) {
    const double r = __builtin_amdgcn_rcp(n);
    return fma(fma(-n, r, 1.0), r, r);
}

// Threads that work on one of `count` things together: 2^lanes_per of them,
// at most 64, such that the block covers all of them in one go where it can.
__device__ __forceinline__ int lanes_per(int count) {
    int lg = 6;
    while (lg > 0 && (int)(blockDim.x >> lg) < count) --lg;
    return lg;
}

// B vectors of a thread, `step` elements apart, from value i of cnt on.  Loads
// past the end repeat the last value (or the first, where there is none), so
// that all B are issued together.
template <typename T, int V, int B> struct Batch {
    typename Vec<T, V>::raw raw[B];
    __device__ __forceinline__ void load(const T* p, long long step, int i, int cnt) {
#pragma unroll
        for (int u = 0; u < B; ++u) raw[u] = Vec<T, V>::load(p + max(min(i + u, cnt - 1), 0) * step);
    }
};

// Combines an image's chunk partials (mean, M2) into mean and rstd in LDS, in
// one pass: with d = mean_i - mean_0, M2 = sum(M2_i) + sum(n d^2) - sum(n d)^2 / N.
__device__ __forceinline__ void combine_stats(const float2* part, const NormArgs& a, int n, int chunks, int pix,
                                              float2* stat) {
    const int cg = a.C / a.G, lg = lanes_per(a.G), L = 1 << lg, lane = threadIdx.x & (L - 1);
    const double last = (double)(a.P - (chunks - 1) * pix) * cg, full = (double)pix * cg;
    const double inv = inverse((double)a.P * cg);
    for (int g = threadIdx.x >> lg; g < a.G; g += blockDim.x >> lg) {
        const float2* p = part + (long long)n * chunks * a.G + g;
        const float base = p[0].x;
        double s = 0.0, ss = 0.0;
        for (int j0 = lane; j0 < chunks; j0 += 4 * L) {
            float2 e[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) e[u] = p[(long long)min(j0 + u * L, chunks - 1) * a.G];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + u * L;
                const double w = j >= chunks ? 0.0 : j == chunks - 1 ? last : full, d = (double)e[u].x - base;
                s = fma(w, d, s);
                ss += fma(w * d, d, (double)(j >= chunks ? 0.0f : e[u].y));
            }
        }
        s = lanes_sum(s, L);
        ss = lanes_sum(ss, L);
        const double shift = s * inv;
        const float var = (float)((ss - s * shift) * inv);
        if (lane == 0)
            stat[g] = make_float2((float)(base + shift), 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps));  // a NaN stays
    }
    __syncthreads();
}

// A thread's running sums of x - k and (x - k)^2 for its V channels, k the first
// value of each; finish: (mean, M2) of `cnt` values to LDS, (0, 0) of none.
template <typename T, int V> struct Moments {
    typename Vec<T, V>::raw first;
    float k[V];
    double s[V], ss[V];
    __device__ __forceinline__ void start(const typename Vec<T, V>::raw& f) {
        first = f;
        Vec<T, V>::unpack(f, k);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = ss[j] = 0.0;
    }
    __device__ __forceinline__ void add(const typename Vec<T, V>::raw& r, bool inside) {
        float v[V];
        Vec<T, V>::unpack(inside ? r : first, v);   // past the end: adds nothing
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double d = (double)v[j] - k[j];
            s[j] += d;
            ss[j] = fma(d, d, ss[j]);
        }
    }
    __device__ __forceinline__ void finish(int cnt, float2* out) const {
        const double inv = cnt > 0 ? inverse(cnt) : 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double d = s[j] * inv;
            const float m2 = (float)(ss[j] - s[j] * d);
            out[j] = cnt > 0 ? make_float2((float)(k[j] + d), m2 < 0.0f ? 0.0f : m2) : make_float2(0.0f, 0.0f);  // a NaN stays
        }
    }
};

// The same for `cnt` vectors that stream past.
template <typename T, int V, int B = kBatch>
__device__ __forceinline__ void stream_moments(const T* p, long long step, int cnt, float2* out) {
    Batch<T, V, B> b;
    b.load(p, step, 0, cnt);
    Moments<T, V> m;
    m.start(b.raw[0]);
#pragma clang loop unroll(disable)
    for (int i = 0; i < cnt; i += B) {
#pragma unroll
        for (int u = 0; u < B; ++u) m.add(b.raw[u], i + u < cnt);
        b.load(p, step, i + B, cnt);
    }
    m.finish(cnt, out);
}

// A chunk's (mean, M2) of every group from its R x C entries in LDS, merged in
// one pass as in combine_stats: row `row` of the threads has one value more
// below `more`.  put(g, mean, M2) on one lane of every group.
template <typename PUT>
__device__ __forceinline__ void merge_rows(const float2* lds, const NormArgs& a, int np, int R, PUT put) {
    const int cg = a.C / a.G, lg = lanes_per(a.G), L = 1 << lg, lane = threadIdx.x & (L - 1);
    const int few = np / R, more = np - few * R, count = R * cg;
    const double inv = inverse((double)np * cg);
    for (int g = threadIdx.x >> lg; g < a.G; g += blockDim.x >> lg) {
        const float2* e = lds + g * cg;
        const float base = e[0].x;
        double s = 0.0, ss = 0.0;
        for (int k0 = lane; k0 < count; k0 += 4 * L) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = min(k0 + u * L, count - 1), row = small_div(k, cg);
                const float2 v = e[row * a.C + k - row * cg];
                const bool in = k0 + u * L < count;   // rows without values hold (0, 0)
                const double w = in ? few + (row < more) : 0, d = (double)v.x - base;
                s = fma(w, d, s);
                ss += fma(w * d, d, (double)(in ? v.y : 0.0f));
            }
        }
        s = lanes_sum(s, L);
        ss = lanes_sum(ss, L);
        const double shift = s * inv;
        const float mean = (float)(base + shift), m2 = (float)(ss - s * shift);
        if (lane == 0) put(g, mean, m2 < 0.0f ? 0.0f : m2);   // a NaN stays
    }
}

// First launch of the streaming forward pass: (mean, M2) of every group of
// one chunk.  One workgroup per image and chunk; LDS: R * C pairs.
template <typename T, int V>
__global__ __launch_bounds__(512) void gn_stats_kernel(NormArgs a, int TX, int R, int chunks, int pix, float2* part) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x - n * chunks;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX;
    const int p0 = chunk * pix, np = min(pix, a.P - p0);
    const Part part_of(np, R, r);
    if (r < R)
        for (int at = tx * V; at < a.C; at += TX * V) {
            const int c = vector_start<V>(at, a.C);
            stream_moments<T, V>(static_cast<const T*>(a.x) + ((long long)n * a.P + p0 + part_of.first) * a.ldx + c,
                                 (long long)R * a.ldx, part_of.cnt, lds + r * a.C + c);
        }
    __syncthreads();
    merge_rows(lds, a, np, R, [&](int g, float mean, float m2) {
        part[(long long)blockIdx.x * a.G + g] = make_float2(mean, m2);
    });
}

// A thread's constants for its V channels.  The mean is subtracted first: x *
// (rstd gamma) + (beta - mean rstd gamma) takes one instruction less, but is off
// by 2^-24 of |mean| rstd gamma, 0.02 in a group that is constant at 1000.
template <int V> struct Affine {
    float mean[V], rg[V], beta[V];
    __device__ __forceinline__ void prepare(const NormArgs& a, int c) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            rg[j] = a.gamma ? a.gamma[c + j] : 1.0f;
            beta[j] = a.beta ? a.beta[c + j] : 0.0f;
        }
    }
    __device__ __forceinline__ void finish(float m, float r, int j) {
        mean[j] = m;
        rg[j] *= r;
    }
    __device__ __forceinline__ float z(float x, int j) const { return fmaf(x - mean[j], rg[j], beta[j]); }
};
// the same from the groups' (mean, rstd)
template <int V> __device__ __forceinline__ void finish_affine(Affine<V>& f, const float2* stat, int c, int cg) {
    int g = small_div(c, cg), left = (g + 1) * cg - c;   // channels of group g from c on
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (left == 0) ++g, left = cg;
        --left;
        const float2 s = stat[g];
        f.finish(s.x, s.y, j);
    }
}

__device__ __forceinline__ void save_stats(const NormArgs& a, const float2* stat, int n) {
    for (int g = threadIdx.x; g < a.G; g += blockDim.x) {
        if (a.mean) a.mean[(long long)n * a.G + g] = stat[g].x;
        if (a.rstd) a.rstd[(long long)n * a.G + g] = stat[g].y;
    }
}

// Second launch of the streaming forward pass: one workgroup per image and
// chunk.  The first loads are under way while the partials are combined.
// LDS: G pairs.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(512) void gn_apply_kernel(NormArgs a, int TX, int R, int chunks, int pix,
                                                       const float2* part) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, piece = blockIdx.x - n * chunks;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX;
    const int p0 = piece * pix, np = min(pix, a.P - p0);
    const Part part_of(np, R, r);
    const long long first = (long long)n * a.P + p0 + part_of.first;
    const int cnt = part_of.cnt, c0 = vector_start<V>(tx * V, a.C);
    const long long xs = (long long)R * a.ldx, ys = (long long)R * a.ldy;
    Batch<T, V, kBatch> b;
    b.load(static_cast<const T*>(a.x) + first * a.ldx + c0, xs, 0, cnt);
    Affine<V> f;
    f.prepare(a, c0);
    combine_stats(part, a, n, chunks, pix, lds);
    if (piece == 0) save_stats(a, lds, n);
    const T* p = static_cast<const T*>(a.x) + first * a.ldx + c0;
    T* q = static_cast<T*>(a.y) + first * a.ldy + c0;
    finish_affine<V>(f, lds, c0, a.C / a.G);
#pragma clang loop unroll(disable)
    for (int at = tx * V, i = 0; cnt > 0;) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            float v[V];
            Vec<T, V>::unpack(b.raw[u], v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = activate<ACT>(f.z(v[j], j));
            if (i + u < cnt) Vec<T, V>::store(q + (i + u) * ys, v);
        }
        i += kBatch;
        if (i >= cnt) {   // more than blockDim.x vectors across: the next channels
            at += TX * V;
            if (at >= a.C) break;
            const int c = vector_start<V>(at, a.C);
            i = 0;
            p = static_cast<const T*>(a.x) + first * a.ldx + c;
            q = static_cast<T*>(a.y) + first * a.ldy + c;
            f.prepare(a, c);
            finish_affine<V>(f, lds, c, a.C / a.G);
        }
        b.load(p, xs, i, cnt);
    }
}

// Quantises a thread's `cnt` pixels, `subs` apart from pixel `first` on, B of
// them at a time (the first B in b).  LPP lanes (a power of two) share a pixel;
// a lane outside the row has nothing of it.
template <typename T, int V, int ACT, int B, typename F>
__device__ __forceinline__ void quantise_pixels(const NormArgs& a, const F& f, Batch<T, V, B>& b, long long first, int cnt,
                                                int subs, int c, int l, bool in, int LPP) {
    const T* p = static_cast<const T*>(a.x) + first * a.ldx + c;
    int8_t* q = static_cast<int8_t*>(a.y) + first * a.ldy + c;
    const long long xs = (long long)subs * a.ldx, qs = (long long)subs * a.ldy;
#pragma clang loop unroll(disable)
    for (int i = 0; i < cnt; i += B) {
        float v[B][V];
        uint32_t top[B];
#pragma unroll
        for (int u = 0; u < B; ++u) {   // past the last pixel: not used
            top[u] = 0;
            Vec<T, V>::unpack(b.raw[u], v[u]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[u][j] = activate<ACT>(f.z(v[u][j], j));
                top[u] = max(top[u], __float_as_uint(v[u][j]) & 0x7fffffffu);
            }
        }
        b.load(p, xs, i + B, cnt);
#pragma unroll
        for (int u = 0; u < B; ++u) top[u] = lanes_max(in ? top[u] : 0, LPP);
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const RowScale s = row_scale(top[u]);
            if (i + u < cnt) {
                if (in) store_quantised<V>(q + (i + u) * qs, v[u], s.inv);
                if (l == 0) a.q_scale[first + (long long)(i + u) * subs] = s.scale;
            }
        }
    }
}

// Second launch of the quantised forward pass.  LPP lanes (a power of two)
// share a pixel, lane l holds the vectors l, l + LPP, ... of it.  LDS: G pairs.
// One vector a lane: two pixels at a time, constants in registers.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(256) void gn_quant_kernel(NormArgs a, int LPP, int chunks, int pix, const float2* part) {
    extern __shared__ float2 lds[];
    constexpr int B = 2;
    const int n = blockIdx.x / chunks, piece = blockIdx.x - n * chunks;
    const int sub = small_div(threadIdx.x, LPP), l = threadIdx.x - sub * LPP, subs = small_div(blockDim.x, LPP);
    const bool in = l * V < a.C;
    const int p0 = piece * pix, np = min(pix, a.P - p0), c = in ? vector_start<V>(l * V, a.C) : 0;
    const Part part_of(np, subs, sub);
    const long long first = (long long)n * a.P + p0 + part_of.first;
    const int cnt = part_of.cnt;
    Batch<T, V, B> b;
    b.load(static_cast<const T*>(a.x) + first * a.ldx + c, (long long)subs * a.ldx, 0, cnt);
    Affine<V> f;
    f.prepare(a, c);
    combine_stats(part, a, n, chunks, pix, lds);
    if (piece == 0) save_stats(a, lds, n);
    finish_affine<V>(f, lds, c, a.C / a.G);
    quantise_pixels<T, V, ACT, B>(a, f, b, first, cnt, subs, c, l, in, LPP);
}

// The whole quantised pass in one launch, for small images: every workgroup
// takes the statistics of its image itself, from the cache, rather than wait
// for a launch that takes them.  LDS: R * C pairs, then G.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(512) void gn_quant_whole_kernel(NormArgs a, int LPP, int chunks, int pix) {
    extern __shared__ float2 lds[];
    constexpr int B = 2, BS = 8;
    const int n = blockIdx.x / chunks, piece = blockIdx.x - n * chunks;
    const int sub = small_div(threadIdx.x, LPP), l = threadIdx.x - sub * LPP, subs = small_div(blockDim.x, LPP);
    const bool in = l * V < a.C;
    const int c = in ? vector_start<V>(l * V, a.C) : 0;
    const long long image = (long long)n * a.P, step = (long long)subs * a.ldx;
    Affine<V> f;
    f.prepare(a, c);
    {
        const Part of(a.P, subs, sub);
        const T* p = static_cast<const T*>(a.x) + (image + of.first) * a.ldx + c;
        Moments<T, V> m;
#pragma clang loop unroll(disable)
        for (int i = 0; i == 0 || i < of.cnt; i += BS) {
            Batch<T, V, BS> b;
            b.load(p, step, i, of.cnt);
            if (i == 0) m.start(b.raw[0]);
#pragma unroll
            for (int u = 0; u < BS; ++u) m.add(b.raw[u], i + u < of.cnt);
        }
        if (in) m.finish(of.cnt, lds + sub * a.C + c);
    }
    const int p0 = piece * pix, np = min(pix, a.P - p0);
    const Part part_of(np, subs, sub);
    const long long first = image + p0 + part_of.first;
    Batch<T, V, B> b;
    b.load(static_cast<const T*>(a.x) + first * a.ldx + c, step, 0, part_of.cnt);
    __syncthreads();
    float2* stat = lds + subs * a.C;
    const float total = (float)a.P * (a.C / a.G);
    merge_rows(lds, a, a.P, subs, [&](int g, float mean, float m2) {
        stat[g] = make_float2(mean, 1.0f / sqrtf(m2 / total + a.eps));
    });
    __syncthreads();
    if (piece == 0) save_stats(a, stat, n);
    finish_affine<V>(f, stat, c, a.C / a.G);
    quantise_pixels<T, V, ACT, B>(a, f, b, first, part_of.cnt, subs, c, l, in, LPP);
}

// The same for pixels of more than 64 vectors: a wave per pixel, constants
// from LDS (after the G pairs: mean, rstd gamma and beta of every channel),
// the pixel read a second time (from the cache) when it is stored.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(256) void gn_quant_wide_kernel(NormArgs a, int chunks, int pix, const float2* part) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, piece = blockIdx.x - n * chunks;
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
    const int l = threadIdx.x & 63;
    const int p0 = piece * pix, np = min(pix, a.P - p0);
    auto values = [&](const T* p, int c, float (&v)[V]) {
        Vec<T, V>::unpack(Vec<T, V>::load(p + c), v);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = activate<ACT>(fmaf(v[e] - mean[c + e], rg[c + e], beta[c + e]));
    };
    for (int i = threadIdx.x >> 6; i < np; i += 4) {
        const long long pixel = (long long)n * a.P + p0 + i;
        const T* p = static_cast<const T*>(a.x) + pixel * a.ldx;
        uint32_t top = 0;
#pragma unroll 4
        for (int at = l * V; at < a.C; at += 64 * V) {
            float v[V];
            values(p, vector_start<V>(at, a.C), v);
#pragma unroll
            for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
        }
        const RowScale s = row_scale(lanes_max(top, 64));
#pragma unroll 4
        for (int at = l * V; at < a.C; at += 64 * V) {
            float v[V];
            const int c = vector_start<V>(at, a.C);
            values(p, c, v);
            store_quantised<V>(static_cast<int8_t*>(a.y) + pixel * a.ldy + c, v, s.inv);
        }
        if (l == 0) a.q_scale[pixel] = s.scale;
    }
}

// A thread's constants of the backward pass, and an element's dz from
// xc = x - mean.  scale = gamma * rstd; sums of dz * xc are multiplied with rstd
// at their end.  ONE: its channels are of one group.  ReLU's derivative at 0 is
// 0; a NaN stays.
template <int V, bool ONE = false> struct Slope {
    float mean[ONE ? 1 : V], rstd[ONE ? 1 : V], scale[V], beta[V];
    static constexpr __device__ __forceinline__ int at(int j) { return ONE ? 0 : j; }
    __device__ __forceinline__ void load(const NormArgs& a, int n, int c) {
        const int cg = a.C / a.G;
        int g = small_div(c, cg), left = (g + 1) * cg - c;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (left == 0) ++g, left = cg;
            --left;
            if (!ONE || j == 0) {
                mean[at(j)] = a.mean[(long long)n * a.G + g];
                rstd[at(j)] = a.rstd[(long long)n * a.G + g];
            }
            scale[j] = rstd[at(j)] * (a.gamma ? a.gamma[c + j] : 1.0f);
            beta[j] = a.beta ? a.beta[c + j] : 0.0f;
        }
    }
    __device__ __forceinline__ float xc(float x, int j) const { return x - mean[at(j)]; }
    template <int ACT> __device__ __forceinline__ float dz(float dy, float xc, int j) const {
        if (ACT == kActNone) return dy;
        const float z = fmaf(xc, scale[j], beta[j]);
        if (ACT == kActRelu) return z > 0.0f ? dy : z <= 0.0f ? 0.0f : z;
        const float e = sigmoid(z);
        return dy * fmaf(z * e, 1.0f - e, e);
    }
};

// Sums of a workgroup's channels over its R rows of threads (pairs in LDS:
// R * cols) into row 0, L lanes to a channel.
__device__ __forceinline__ void sum_rows(float2* lds, int R, int cols) {
    const int lg = lanes_per(cols), L = 1 << lg, lane = threadIdx.x & (L - 1);
    for (int c = threadIdx.x >> lg; c < cols; c += blockDim.x >> lg) {
        float s = 0.0f, t = 0.0f;
        for (int k = lane; k < R; k += L) {
            s += lds[k * cols + c].x;
            t += lds[k * cols + c].y;
        }
        s = lanes_sum(s, L);
        t = lanes_sum(t, L);
        if (lane == 0) lds[c] = make_float2(s, t);
    }
    __syncthreads();
}

// A chunk's two sums of every group, weighted with gamma, from those of its
// channels in LDS.  put(g, sum, sum) on one lane of every group.
template <typename PUT> __device__ __forceinline__ void weigh_groups(const float2* lds, const NormArgs& a, PUT put) {
    const int cg = a.C / a.G, lg = lanes_per(a.G), L = 1 << lg, lane = threadIdx.x & (L - 1);
    for (int g = threadIdx.x >> lg; g < a.G; g += blockDim.x >> lg) {
        float s = 0.0f, t = 0.0f;
        for (int c = g * cg + lane; c < (g + 1) * cg; c += L) {
            const float w = a.gamma ? a.gamma[c] : 1.0f;
            s = fmaf(w, lds[c].x, s);
            t = fmaf(w, lds[c].y, t);
        }
        s = lanes_sum(s, L);
        t = lanes_sum(t, L);
        if (lane == 0) put(g, s, t);
    }
}

// Adds an image's chunks: out[g] = the group's two sums over m.
__device__ __forceinline__ void add_chunks(const float2* part, const NormArgs& a, int chunks, float2* out) {
    const int lg = lanes_per(a.G), L = 1 << lg, lane = threadIdx.x & (L - 1);
    const float inv = 1.0f / ((float)a.P * (a.C / a.G));
    for (int g = threadIdx.x >> lg; g < a.G; g += blockDim.x >> lg) {
        const float2* p = part + g;
        float s = 0.0f, t = 0.0f;
        for (int j0 = lane; j0 < chunks; j0 += 4 * L) {
            float2 e[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) e[u] = p[(long long)min(j0 + u * L, chunks - 1) * a.G];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s += j0 + u * L < chunks ? e[u].x : 0.0f;
                t += j0 + u * L < chunks ? e[u].y : 0.0f;
            }
        }
        s = lanes_sum(s, L);
        t = lanes_sum(t, L);
        if (lane == 0) out[g] = make_float2(s * inv, t * inv);
    }
    __syncthreads();
}

// A thread's sums of dz and dz * xc for its V channels; finish: those of dz and
// dz * xh to LDS.
template <typename T, int V, int ACT, typename F> struct SlopeSums {
    float A[V], B[V];
    __device__ __forceinline__ SlopeSums() {
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = B[j] = 0.0f;
    }
    __device__ __forceinline__ void add(const F& f, const typename Vec<T, V>::raw& rx, const typename Vec<T, V>::raw& rd,
                                        bool inside) {
        float x[V], d[V];
        Vec<T, V>::unpack(rx, x);
        Vec<T, V>::unpack(rd, d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xc = f.xc(x[j], j), dz = f.template dz<ACT>(d[j], xc, j);
            A[j] += inside ? dz : 0.0f;
            B[j] = inside ? fmaf(dz, xc, B[j]) : B[j];
        }
    }
    __device__ __forceinline__ void finish(const F& f, float2* out) const {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = make_float2(A[j], B[j] * f.rstd[F::at(j)]);
    }
};

// The same for `cnt` pixels from `first` on, R apart, that stream past.
template <typename T, int V, int ACT, typename F, int NB = kBatchBwd>
__device__ __forceinline__ void stream_slopes(const NormArgs& a, int n, int c, long long first, int cnt, int R,
                                              float2* out) {
    const T* px = static_cast<const T*>(a.x) + first * a.ldx + c;
    const T* pd = static_cast<const T*>(a.dy) + first * a.lddy + c;
    const long long xs = (long long)R * a.ldx, ds = (long long)R * a.lddy;
    Batch<T, V, NB> bx, bd;
    bx.load(px, xs, 0, cnt);
    bd.load(pd, ds, 0, cnt);
    F f;
    f.load(a, n, c);
    SlopeSums<T, V, ACT, F> sums;
#pragma clang loop unroll(disable)
    for (int i = 0; i < cnt; i += NB) {
#pragma unroll
        for (int u = 0; u < NB; ++u) sums.add(f, bx.raw[u], bd.raw[u], i + u < cnt);
        bx.load(px, xs, i + NB, cnt);
        bd.load(pd, ds, i + NB, cnt);
    }
    sums.finish(f, out);
}

// First launch of the streaming backward pass: for every image and chunk the
// sums of dz and dz * xh per channel (pc: [block][2][C]) and, weighted with
// gamma, per group (pg).  LDS: R * C pairs.
template <typename T, int V, int ACT, int NB>
__global__ __launch_bounds__(512) void gn_bwd_sums_kernel(NormArgs a, int TX, int R, int chunks, int pix, float* pc,
                                                          float2* pg) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x - n * chunks;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX;
    const int p0 = chunk * pix, np = min(pix, a.P - p0);
    if (r < R) {
        const Part part_of(np, R, r);
        const long long first = (long long)n * a.P + p0 + part_of.first;
        for (int at = tx * V; at < a.C; at += TX * V) {
            const int c = vector_start<V>(at, a.C);
            stream_slopes<T, V, ACT, Slope<V>, NB>(a, n, c, first, part_of.cnt, R, lds + r * a.C + c);
        }
    }
    __syncthreads();
    sum_rows(lds, R, a.C);
    float* out = pc + (long long)blockIdx.x * 2 * a.C;
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        out[c] = lds[c].x;
        out[a.C + c] = lds[c].y;
    }
    weigh_groups(lds, a, [&](int g, float s, float t) { pg[(long long)blockIdx.x * a.G + g] = make_float2(s, t); });
}

constexpr int kParamChannels = 32;  // channels of one workgroup that sums dgamma and dbeta

// Adds `count` partials of kParamChannels channels into dgamma and dbeta, in
// fp64: they may be many and of one sign.  LDS: blockDim.x pairs.
__device__ __forceinline__ void sum_params(const NormArgs& a, const float* pc, long long count, int block, double2* lds) {
    const int c = block * kParamChannels + threadIdx.x % kParamChannels;
    const int row = threadIdx.x / kParamChannels, rows = blockDim.x / kParamChannels;
    double s = 0.0, t = 0.0;
    if (c < a.C) {
        const float* p = pc + c;
#pragma unroll 8
        for (long long i = row; i < count; i += rows) {
            s += p[i * 2 * a.C];
            t += p[i * 2 * a.C + a.C];
        }
    }
    lds[threadIdx.x] = make_double2(s, t);
    __syncthreads();
    if (row == 0 && c < a.C) {
        for (int k = 1; k < rows; ++k) {
            s += lds[k * kParamChannels + threadIdx.x].x;
            t += lds[k * kParamChannels + threadIdx.x].y;
        }
        if (a.dbeta) a.dbeta[c] = (float)s;
        if (a.dgamma) a.dgamma[c] = (float)t;
    }
}

// Second launch of the streaming backward pass.  The first `sums` workgroups
// add the channels' partials into dgamma and dbeta, the others write dx, one
// per image and chunk.  LDS: G pairs, or blockDim.x fp64 ones.
template <typename T, int V, int ACT, int NB>
__global__ __launch_bounds__(512) void gn_bwd_apply_kernel(NormArgs a, int TX, int R, int chunks, int pix, int sums,
                                                           const float* pc, const float2* pg) {
    extern __shared__ double2 lds_pairs[];
    if ((int)blockIdx.x < sums) {
        sum_params(a, pc, (long long)a.N * chunks, blockIdx.x, lds_pairs);
        return;
    }
    float2* const lds = reinterpret_cast<float2*>(lds_pairs);
    const int b = blockIdx.x - sums;
    const int n = b / chunks, piece = b - n * chunks;
    const int cg = a.C / a.G;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX;
    const int p0 = piece * pix, np = min(pix, a.P - p0);
    const Part part_of(np, R, r);
    const long long first = (long long)n * a.P + p0 + part_of.first;
    const int cnt = part_of.cnt, c0 = vector_start<V>(tx * V, a.C);
    const long long xs = (long long)R * a.ldx, ds = (long long)R * a.lddy, os = (long long)R * a.ldy;
    Batch<T, V, NB> bx, bd;
    bx.load(static_cast<const T*>(a.x) + first * a.ldx + c0, xs, 0, cnt);
    bd.load(static_cast<const T*>(a.dy) + first * a.lddy + c0, ds, 0, cnt);
    Slope<V> f;
    f.load(a, n, c0);
    add_chunks(pg + (long long)n * chunks * a.G, a, chunks, lds);
    const T* px = static_cast<const T*>(a.x) + first * a.ldx + c0;
    const T* pd = static_cast<const T*>(a.dy) + first * a.lddy + c0;
    T* po = static_cast<T*>(a.y) + first * a.ldy + c0;
    float s1[V], s2[V];   // rstd * s1, rstd^2 * s2
    auto group_sums = [&](int c) {
        int g = small_div(c, cg), left = (g + 1) * cg - c;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (left == 0) ++g, left = cg;
            --left;
            const float2 s = lds[g];
            s1[j] = s.x * f.rstd[j];
            s2[j] = s.y * f.rstd[j] * f.rstd[j];
        }
    };
    group_sums(c0);
#pragma clang loop unroll(disable)
    for (int at = tx * V, i = 0; cnt > 0;) {
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            float x[V], d[V];
            Vec<T, V>::unpack(bx.raw[u], x);
            Vec<T, V>::unpack(bd.raw[u], d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xc = f.xc(x[j], j), dz = f.template dz<ACT>(d[j], xc, j);
                d[j] = fmaf(dz, f.scale[j], -fmaf(xc, s2[j], s1[j]));
            }
            if (i + u < cnt) Vec<T, V>::store(po + (i + u) * os, d);
        }
        i += NB;
        if (i >= cnt) {
            at += TX * V;
            if (at >= a.C) break;
            const int c = vector_start<V>(at, a.C);
            i = 0;
            px = static_cast<const T*>(a.x) + first * a.ldx + c;
            pd = static_cast<const T*>(a.dy) + first * a.lddy + c;
            po = static_cast<T*>(a.y) + first * a.ldy + c;
            f.load(a, n, c);
            group_sums(c);
        }
        bx.load(px, xs, i, cnt);
        bd.load(pd, ds, i, cnt);
    }
}

// ------------------------------------------------------------------ resident

// What the compiler knows of a vector ends here: it would keep the values that
// it unpacked before, twice the registers, rather than unpack them again.
__device__ __forceinline__ void forget(uint4& v) { asm("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }
__device__ __forceinline__ void forget(uint2& v) { asm("" : "+v"(v.x), "+v"(v.y)); }
__device__ __forceinline__ void forget(uint32_t& v) { asm("" : "+v"(v)); }
__device__ __forceinline__ void forget(uint16_t&) {}

// Sums over the workgroup; every thread gets them.  LDS: 2 * 16 floats, not
// in use by an earlier call.
__device__ __forceinline__ float2 block_sum(float s, float t, float* lds) {
    s = lanes_sum(s, 64);
    t = lanes_sum(t, 64);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        lds[threadIdx.x >> 6] = s;
        lds[16 + (threadIdx.x >> 6)] = t;
    }
    __syncthreads();
    s = t = 0.0f;
    for (int w = 0; w < waves; ++w) {
        s += lds[w];
        t += lds[16 + w];
    }
    return make_float2(s, t);
}

// One fp64 sum.  LDS: 16 doubles, not in use by an earlier call.
__device__ __forceinline__ double block_sum(double s, double* lds) {
    s = lanes_sum(s, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += lds[w];
    return s;
}

// Forward: one workgroup per (image, group), NV vectors of it in each thread.
// The mean from an fp64 sum, so that a constant group's is its value: the
// deviations are multiplied with rstd, up to 1 / sqrt(eps).
template <typename T, int V, int ACT, int NV>
__global__ __launch_bounds__(1024) void gn_resident_kernel(NormArgs a, int TX, int R) {
    __shared__ double lds64[16];
    __shared__ float lds[32];
    const int b = xcd_tile_index(), n = b / a.G, g = b - n * a.G, cg = a.C / a.G;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX, c = g * cg + tx * V;
    const Part part_of(a.P, R, r);
    const long long first = (long long)n * a.P + part_of.first;
    const int cnt = part_of.cnt;
    Batch<T, V, NV> x;
    x.load(static_cast<const T*>(a.x) + first * a.ldx + c, (long long)R * a.ldx, 0, cnt);
    Affine<V> f;
    f.prepare(a, c);
    double total = 0.0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float v[V];
        Vec<T, V>::unpack(x.raw[u], v);
        double t = v[0];
#pragma unroll
        for (int j = 1; j < V; ++j) t += v[j];
        total += u < cnt ? t : 0.0;
    }
    const double inv = inverse((double)a.P * cg);
    const float mean = (float)(block_sum(total, lds64) * inv);
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float v[V], t = 0.0f;
        Vec<T, V>::unpack(x.raw[u], v);
#pragma unroll
        for (int j = 0; j < V; ++j) t = fmaf(v[j] - mean, v[j] - mean, t);
        s += u < cnt ? t : 0.0f;
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, 0.0f, lds).x / ((float)a.P * cg) + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[b] = mean;
        if (a.rstd) a.rstd[b] = rstd;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) f.finish(mean, rstd, j);
    T* q = static_cast<T*>(a.y) + first * a.ldy + c;
    const long long ys = (long long)R * a.ldy;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float v[V];
        Vec<T, V>::unpack(x.raw[u], v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = activate<ACT>(f.z(v[j], j));
        if (u < cnt) Vec<T, V>::store(q + u * ys, v);
    }
}

// Backward: the same, with the channels' sums of this image to pc
// ([image][2][C]), or, for a single image (pc null), to dgamma and dbeta themselves.
// LDS: R * C/G pairs.
template <typename T, int V, int ACT, int NV>
__global__ __launch_bounds__(1024) void gn_bwd_resident_kernel(NormArgs a, int TX, int R, float* pc) {
    extern __shared__ float2 rows[];
    __shared__ float lds[32];
    const int b = xcd_tile_index(), n = b / a.G, g = b - n * a.G, cg = a.C / a.G;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX, c = g * cg + tx * V;
    const Part part_of(a.P, R, r);
    const long long first = (long long)n * a.P + part_of.first;
    const int cnt = part_of.cnt;
    Batch<T, V, NV> bx, bd;
    bx.load(static_cast<const T*>(a.x) + first * a.ldx + c, (long long)R * a.ldx, 0, cnt);
    bd.load(static_cast<const T*>(a.dy) + first * a.lddy + c, (long long)R * a.lddy, 0, cnt);
    Slope<V, true> f;
    f.load(a, n, c);
    SlopeSums<T, V, ACT, Slope<V, true>> sums;
#pragma unroll
    for (int u = 0; u < NV; ++u) sums.add(f, bx.raw[u], bd.raw[u], u < cnt);
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s = fmaf(f.scale[j], sums.A[j], s);
        t = fmaf(f.scale[j], sums.B[j], t);
    }
    if (r < R) sums.finish(f, rows + r * cg + tx * V);
    const float2 sum = block_sum(s, t, lds);   // and the rows are in LDS
    const float m = (float)a.P * cg, s1 = sum.x / m, s2 = sum.y / m * f.rstd[0] * f.rstd[0];
    T* po = static_cast<T*>(a.y) + first * a.ldy + c;
    const long long os = (long long)R * a.ldy;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float x[V], d[V];
        if constexpr (sizeof(T) == 2) {
            forget(bx.raw[u]);
            forget(bd.raw[u]);
        }
        Vec<T, V>::unpack(bx.raw[u], x);
        Vec<T, V>::unpack(bd.raw[u], d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xc = f.xc(x[j], j), dz = f.template dz<ACT>(d[j], xc, j);
            d[j] = fmaf(dz, f.scale[j], -fmaf(xc, s2, s1));
        }
        if (u < cnt) Vec<T, V>::store(po + u * os, d);
    }
    if (!a.dgamma && !a.dbeta) return;
    sum_rows(rows, R, cg);
    for (int k = threadIdx.x; k < cg; k += blockDim.x) {
        if (!pc) {
            if (a.dbeta) a.dbeta[g * cg + k] = rows[k].x;
            if (a.dgamma) a.dgamma[g * cg + k] = rows[k].y;
        } else {
            pc[(long long)n * 2 * a.C + g * cg + k] = rows[k].x;
            pc[(long long)n * 2 * a.C + a.C + g * cg + k] = rows[k].y;
        }
    }
}

// ------------------------------------------------------------------ joined

// Tensors that no workgroup can hold a group of, read from memory once all the
// same: every workgroup keeps a chunk of an image in registers, puts the chunk's
// partial statistics of every group into the workspace, takes those of its
// image's other chunks from there and finishes its own.
//
// A pair of partials is one 64-bit word, so that it is its own flag: a launch
// before fills the words with kMissing, which no pair is (its NaNs are made
// one pattern), and whoever has a pair puts it in the place of kMissing, once.
//
// No workgroup depends on another being resident: after `polls` looks at words
// that stay missing it computes the chunk's partials itself, by the same
// arithmetic, and puts them there.  The input may be the output too: a
// workgroup writes only after it has seen all words of its own chunk, so one
// that reads that chunk in its place and then still finds a word missing has
// read what was there before, and the word it offers otherwise is dropped.
typedef unsigned long long word_t;
constexpr word_t kMissing = ~0ull;

__device__ __forceinline__ word_t pair_word(float x, float y) {
    const uint32_t nan = 0x7fc00000u, lo = x == x ? __float_as_uint(x) : nan, hi = y == y ? __float_as_uint(y) : nan;
    return (word_t)hi << 32 | lo;
}

__device__ __forceinline__ void put_word(word_t* at, word_t w) {
    word_t expected = kMissing;
    __hip_atomic_compare_exchange_strong(at, &expected, w, __ATOMIC_RELAXED, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ word_t look(const word_t* at) {
    return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(256) void gn_clear_kernel(word_t* words, long long count) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) words[i] = kMissing;
}

// An image's `count` words, [chunk][G], into LDS; help(chunk) for a chunk of
// which words stay missing (the whole workgroup, with a barrier at its end).
// Ends with a barrier.
template <typename HELP>
__device__ __forceinline__ void gather(const word_t* words, int count, int G, int polls, word_t* lds, HELP help) {
    __shared__ int missing;
    constexpr int B = 4;
    for (;;) {
        int miss = 0x7fffffff, left = polls;
        if (threadIdx.x == 0) missing = miss;
        for (int e0 = threadIdx.x; e0 < count; e0 += B * blockDim.x) {
            word_t w[B];
#pragma unroll
            for (int u = 0; u < B; ++u) w[u] = look(words + min(e0 + u * (int)blockDim.x, count - 1));
#pragma unroll
            for (int u = 0; u < B; ++u) {
                const int e = min(e0 + u * (int)blockDim.x, count - 1);
                for (; w[u] == kMissing && left > 0; --left) {
                    __builtin_amdgcn_s_sleep(2);
                    w[u] = look(words + e);
                }
                if (w[u] == kMissing) miss = min(miss, e / G);
                lds[e] = w[u];
            }
        }
        __syncthreads();
        if (miss != 0x7fffffff) atomicMin(&missing, miss);
        __syncthreads();
        const int m = missing;
        __syncthreads();
        if (m == 0x7fffffff) return;
        help(m);
    }
}

// Vectors are worked on one after the other: all at once, as the compiler would
// order them, unpacked values push the resident ones out to memory.
__device__ __forceinline__ void one_by_one() { __builtin_amdgcn_sched_barrier(0); }

// A chunk's rows behind a buffer descriptor: 32-bit offsets, loads past the
// chunk's last pixel give zeros and stores there are dropped.
template <int NV> struct Chunk {
    __amdgpu_buffer_rsrc_t rows;
    uint32_t at, step;
    // elem bytes an element, pixels `ld` apart; the thread starts at pixel r,
    // channel c, or outside
    __device__ __forceinline__ Chunk(const void* p, long long pixel, long long ld, int elem, int np, int C, int R, int r,
                                     int c, bool in)
        : rows(make_rsrc(static_cast<const char*>(p) + pixel * ld * elem, (uint32_t)(((np - 1) * ld + C) * elem))),
          at(in ? (uint32_t)((r * ld + c) * elem) : (uint32_t)kOOB),
          step((uint32_t)(R * ld * elem)) {}
    __device__ __forceinline__ void load(uint4 (&v)[NV]) const {
#pragma unroll
        for (int u = 0; u < NV; ++u) v[u] = load16(rows, (int)(at + u * step));
    }
};

// Channels h .. h + 3 of a 16-byte vector.
template <typename T> __device__ __forceinline__ typename Vec<T, 4>::raw four_of(const uint4& v, int h) {
    if constexpr (sizeof(T) == 4) return v;
    else return h ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y);
}

// Forward (QUANT: with the quantisation of every pixel, whose vectors are then
// TX lanes, a power of two, of one wave).  LDS: R * C pairs, or the image's
// words and G pairs if those are more.
template <typename T, int V, int ACT, int NV, bool QUANT>
__global__ __launch_bounds__(256, 4) void gn_joined_kernel(NormArgs a, int TX, int R, int chunks, int pix, int polls,
                                                           word_t* words) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x - n * chunks;
    const int r = small_div(threadIdx.x, TX), tx = threadIdx.x - r * TX;
    const bool in = r < R && tx * V < a.C;
    const int c = in ? tx * V : 0;
    const long long image = (long long)n * a.P;
    const int p0 = chunk * pix, np = min(pix, a.P - p0);
    const int cnt = in ? Part(np, R, r).cnt : 0;
    words += (long long)n * chunks * a.G;
    uint4 raw[NV];
    Chunk<NV>(a.x, image + p0, a.ldx, sizeof(T), np, a.C, R, r, c, in).load(raw);
    constexpr int H = 4;   // channels at a time: all of bf16's, in fp64, would push out 61 registers
#pragma unroll
    for (int h = 0; h < V; h += H) {
        Moments<T, H> m;
        m.start(four_of<T>(raw[0], h));
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            m.add(four_of<T>(raw[u], h), u < cnt);
            one_by_one();
        }
        if (in) m.finish(cnt, lds + r * a.C + c + h);
    }
    __syncthreads();
    merge_rows(lds, a, np, R, [&](int g, float mean, float m2) { put_word(words + chunk * a.G + g, pair_word(mean, m2)); });
    __syncthreads();
    gather(words, chunks * a.G, a.G, polls, reinterpret_cast<word_t*>(lds), [&](int other) {
        const int q0 = other * pix, nq = min(pix, a.P - q0);
        const Part of(nq, R, r);
#pragma clang loop unroll(disable)
        for (int k = in ? c : a.C; k < min(c + V, a.C); ++k)   // channel by channel: few registers
            stream_moments<T, 1, 1>(static_cast<const T*>(a.x) + (image + q0 + of.first) * a.ldx + k,
                                    (long long)R * a.ldx, of.cnt, lds + r * a.C + k);
        __syncthreads();
        merge_rows(lds, a, nq, R, [&](int g, float mean, float m2) { put_word(words + other * a.G + g, pair_word(mean, m2)); });
        __syncthreads();
    });
    Affine<V> f;
    f.prepare(a, c);
    float2* stat = lds + chunks * a.G;
    combine_stats(lds, a, 0, chunks, pix, stat);
    if (chunk == 0) save_stats(a, stat, n);
    finish_affine<V>(f, stat, c, a.C / a.G);
    const Chunk<NV> out(a.y, image + p0, a.ldy, QUANT ? 1 : sizeof(T), np, a.C, R, r, c, in);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float v[V];
        forget(raw[u]);
        Vec<T, V>::unpack(raw[u], v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = activate<ACT>(f.z(v[j], j));
        if constexpr (!QUANT) {
            store16(out.rows, (int)(out.at + u * out.step), Vec<T, V>::pack(v));
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
            const RowScale s = row_scale(lanes_max(in ? top : 0, TX));
            if (u < cnt) {
                store_quantised<V>(static_cast<int8_t*>(a.y) + (image + p0 + r + u * R) * a.ldy + c, v, s.inv);
                if (tx == 0) a.q_scale[image + p0 + r + u * R] = s.scale;
            }
        }
        one_by_one();
    }
}

// Backward, for vectors that lie in one group; the channels' sums of every
// chunk go to pc ([block][2][C]).  LDS as in the forward pass.
template <typename T, int V, int ACT, int NV>
__global__ __launch_bounds__(256, 3) void gn_bwd_joined_kernel(NormArgs a, int TX, int R, int chunks, int pix, int polls,
                                                               word_t* words, float* pc) {
    extern __shared__ float2 lds[];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x - n * chunks;
    const int r = small_div(threadIdx.x, TX), c = (threadIdx.x - r * TX) * V;
    const int p0 = chunk * pix, np = min(pix, a.P - p0);
    const int cnt = Part(np, R, r).cnt;
    const bool in = r < R;
    const long long image = (long long)n * a.P;
    words += (long long)n * chunks * a.G;
    typedef Slope<V, true> F;
    uint4 rx[NV];
    float dz[NV][V];   // kept: the sigmoid and its slope are most of the pass's arithmetic
    float scale[V], mean, rstd;
    {
        uint4 rd[NV];
        Chunk<NV>(a.x, image + p0, a.ldx, sizeof(T), np, a.C, R, r, c, in).load(rx);
        Chunk<NV>(a.dy, image + p0, a.lddy, sizeof(T), np, a.C, R, r, c, in).load(rd);
        F f;
        f.load(a, n, c);
        SlopeSums<T, V, ACT, F> sums;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float x[V], d[V];
            Vec<T, V>::unpack(u < cnt ? rx[u] : rx[0], x);
            Vec<T, V>::unpack(rd[u], d);   // outside: 0, and so is dz
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xc = f.xc(x[j], j);
                dz[u][j] = f.template dz<ACT>(d[j], xc, j);
                sums.A[j] += dz[u][j];
                sums.B[j] = fmaf(dz[u][j], xc, sums.B[j]);
            }
            one_by_one();
        }
        if (in) sums.finish(f, lds + r * a.C + c);
#pragma unroll
        for (int j = 0; j < V; ++j) scale[j] = f.scale[j];
        mean = f.mean[0];
        rstd = f.rstd[0];
    }
    __syncthreads();
    sum_rows(lds, R, a.C);
    if (a.dgamma || a.dbeta) {
        float* out = pc + (long long)blockIdx.x * 2 * a.C;
        for (int k = threadIdx.x; k < a.C; k += blockDim.x) {
            out[k] = lds[k].x;
            out[a.C + k] = lds[k].y;
        }
    }
    weigh_groups(lds, a, [&](int g, float s, float t) { put_word(words + chunk * a.G + g, pair_word(s, t)); });
    __syncthreads();
    gather(words, chunks * a.G, a.G, polls, reinterpret_cast<word_t*>(lds), [&](int other) {
        const int q0 = other * pix;
        const Part of(min(pix, a.P - q0), R, r);
#pragma clang loop unroll(disable)
        for (int k = in ? c : a.C; k < min(c + V, a.C); ++k)
            stream_slopes<T, 1, ACT, Slope<1, true>, 1>(a, n, k, image + q0 + of.first, of.cnt, R, lds + r * a.C + k);
        __syncthreads();
        sum_rows(lds, R, a.C);
        weigh_groups(lds, a, [&](int g, float s, float t) { put_word(words + other * a.G + g, pair_word(s, t)); });
        __syncthreads();
    });
    float2* sums = lds + chunks * a.G;
    add_chunks(lds, a, chunks, sums);
    const float2 sum = sums[small_div(c, a.C / a.G)];
    const float s1 = sum.x * rstd, s2 = sum.y * rstd * rstd;
    const Chunk<NV> out(a.y, image + p0, a.ldy, sizeof(T), np, a.C, R, r, c, in);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float x[V], d[V];
        forget(rx[u]);
        Vec<T, V>::unpack(rx[u], x);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = fmaf(dz[u][j], scale[j], -fmaf(x[j] - mean, s2, s1));
        store16(out.rows, (int)(out.at + u * out.step), Vec<T, V>::pack(d));
        one_by_one();
    }
}

__global__ __launch_bounds__(256) void gn_params_kernel(NormArgs a, const float* pc, long long count) {
    __shared__ double2 lds[256];
    sum_params(a, pc, count, blockIdx.x, lds);
}

// An image's `count` partials of kParamChannels channels into one: out [N][2][C].
// `sums` workgroups an image.
__global__ __launch_bounds__(256) void gn_image_params_kernel(NormArgs a, const float* pc, int count, int sums, float* out) {
    __shared__ double2 lds[256];
    const int image = blockIdx.x / sums;
    out += (long long)image * 2 * a.C;
    a.dbeta = out;
    a.dgamma = out + a.C;
    sum_params(a, pc + (long long)image * count * 2 * a.C, count, blockIdx.x - image * sums, lds);
}

// ------------------------------------------------------------------ host

// Elements of one vector access: the most that divides `unit` (the channel
// count, or a group's) and every row stride, up to 16 bytes, with every
// pointer aligned to it.
int vector_width(const NormArgs& a, int unit, int elem, int out_elem) {
    int v = 16 / elem;
    auto ok = [&](const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; };
    while (v > 1 && !(unit % v == 0 && a.ldx % v == 0 && a.ldy % v == 0 && (!a.dy || a.lddy % v == 0) &&
                      ok(a.x, v * elem) && ok(a.y, v * out_elem) && ok(a.dy, v * elem)))
        v >>= 1;
    return v;
}

// The streaming form's, of large tensors: 16 bytes whatever the alignment, the
// last vector of a row over part of the one before, unless the output is an
// input too (a thread would read what another has written) or the row is
// shorter.  bf16, 531 channels (one element an access otherwise): 98 MB 73 us
// against 213, backward 117 against 283; 20 MB 27 against 41, 40 against 51; 11
// MB 22 against 23, 32 against 30; 4 MB 14.5 against 16.6, 17.8 against 19.9.
// 252 channels (four elements): 100 MB 71 against 84, 10 MB 17.5 against 14.4.
constexpr long long kRaggedBytes = 8 << 20;

int row_width(const NormArgs& a, int elem, int out_elem) {
    const int most = 16 / elem;
    if (a.C < most || a.y == a.x || a.y == a.dy || (long long)a.N * a.P * a.C * elem < kRaggedBytes)
        return vector_width(a, a.C, elem, out_elem);
    return most;
}

// The quantised pass in one launch: images of at most kWholeVectors vectors, no
// more workgroups than compute units.  Through norm and product, against two
// launches: 200 images of 8x8x64 (512 vectors) 12.7 us for 15.2, 32 of 14x14x256
// (6272) 16.1 for 17.6; 3 of 16x7x512 (7168) 16.2 for 15.2, one of 28x28x128
// (12544) 17.5 for 14.3.
constexpr int kWholeThreads = 512, kWholeBlocks = 256;
constexpr long long kWholeVectors = 6400;

struct Plan {
    int TX, R, block, chunks, pix;
};

// run(images, first) for all images, `per` workgroups of `threads` each: a launch
// counts its threads in 32 bits, so that very many images (of one pixel, say)
// take several.
template <typename F> hipError_t in_launches(const NormArgs& a, long long per, int threads, F run) {
    const long long most = 0xff000000LL / (per * threads);   // 2^24 left for workgroups beside them
    const int elem = a.dtype == 0 /* CONV2D_F32 */ ? 4 : 2;
    for (long long n = 0; n < a.N; n += most) {
        NormArgs s = a;
        auto pixels = [&](const void* p, long long ld, int bytes) { return p ? static_cast<const char*>(p) + n * a.P * ld * bytes : nullptr; };
        s.N = (int)(a.N - n < most ? a.N - n : most);
        s.x = pixels(a.x, a.ldx, elem);
        s.dy = pixels(a.dy, a.lddy, elem);
        s.y = const_cast<char*>(pixels(a.y, a.ldy, a.q_scale ? 1 : elem));
        if (a.q_scale) s.q_scale += n * a.P;
        if (a.mean) s.mean += n * a.G;
        if (a.rstd) s.rstd += n * a.G;
        run(s, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int param_blocks(const NormArgs& a) { return a.dgamma || a.dbeta ? (a.C + kParamChannels - 1) / kParamChannels : 0; }

// Threads: TX across the channel vectors, R rows of them, the block size of
// 256 to 512 that leaves the fewest idle.  Chunks: kTargetBlocks workgroups
// in all or a few less (two for each compute unit, of equal size: they run at
// once), at most kMaxChunks per image, of a whole number of pixels a thread,
// two at least where there are more than 64: the second launch waits for all of
// an image's partials (4 images of 28x28x256, quantised and multiplied: 98
// chunks 19.9 us, 49 16.3).
Plan make_plan(int N, int P, int C, int V) {
    Plan p;
    const int cv = (C + V - 1) / V;
    p.TX = cv < 256 ? cv : 256;
    int best = 0;
    p.block = 256;
    for (int b = 256; b <= 512; b += 64) {
        const int used = b / p.TX * p.TX * 4096 / b;
        if (used > best) best = used, p.block = b;
    }
    p.R = p.block / p.TX;
    long long k = kTargetBlocks / N;
    k = k < 1 ? 1 : k < kMaxChunks ? k : kMaxChunks;
    long long each = (P + k - 1) / k;
    if (k > 64 && each < 2 * p.R) each = 2 * p.R;
    each = (each + p.R - 1) / p.R * p.R;
    p.pix = (int)(each < 0x7fffffff ? each : 0x7fffffff);
    p.chunks = (int)((P + (long long)p.pix - 1) / p.pix);
    return p;
}

// The resident form: threads and the vectors of each, or nv = 0 where the
// group does not fit (most: the largest nv that leaves 1024 threads their
// registers) or is not worth it.  Each
// workgroup reads C/G channels of every pixel: below 64 bytes that splits the
// memory's lines over several workgroups, which costs more than the second
// read once the tensor is large.
struct Resident {
    int TX, R, block, nv;
};

constexpr long long kResidentBytes = 8 << 20;
constexpr long long kResidentUnitBytes = 48 << 10;

Resident make_resident(const NormArgs& a, int V, int elem, int most) {
    Resident p = {0, 0, 0, 0};
    const int cg = a.C / a.G;
    p.TX = cg / V;
    const long long bytes = (long long)a.N * a.P * a.C * elem;
    if ((long long)a.N * a.G < 256 && (long long)a.P * cg * elem > kResidentUnitBytes) return p;
    if (p.TX > 256 || (bytes > kResidentBytes && cg * elem < 64)) return p;
    for (p.block = 256; p.block <= 1024; p.block *= 2) {
        p.R = p.block / p.TX;
        const long long nv = (a.P + (long long)p.R - 1) / p.R;
        if (nv <= (p.block == 1024 ? most : 4)) {
            p.nv = nv <= 2 ? 2 : nv <= 4 ? 4 : 8;
            return p;
        }
    }
    return p;
}

template <typename T, int V, int ACT> hipError_t forward_resident(const NormArgs& a, const Resident& p, hipStream_t st) {
    auto k = p.nv == 2 ? gn_resident_kernel<T, V, ACT, 2> : p.nv == 4 ? gn_resident_kernel<T, V, ACT, 4>
                         : gn_resident_kernel<T, V, ACT, 8>;
    return in_launches(a, a.G, p.block, [&](const NormArgs& s, long long) { k<<<s.N * s.G, p.block, 0, st>>>(s, p.TX, p.R); });
}

template <typename T, int V> hipError_t forward(const NormArgs& a, int act, void* ws, hipStream_t st) {
    const Plan p = make_plan(a.N, a.P, a.C, V);
    float2* part = static_cast<float2*>(ws);
    auto k = act == kActSilu ? gn_apply_kernel<T, V, kActSilu>
             : act == kActRelu ? gn_apply_kernel<T, V, kActRelu> : gn_apply_kernel<T, V, kActNone>;
    return in_launches(a, p.chunks, p.block, [&](const NormArgs& s, long long n) {
        float2* at = part + n * p.chunks * a.G;
        gn_stats_kernel<T, V><<<s.N * p.chunks, p.block, (size_t)p.R * a.C * 8, st>>>(s, p.TX, p.R, p.chunks, p.pix, at);
        k<<<s.N * p.chunks, p.block, (size_t)a.G * 8, st>>>(s, p.TX, p.R, p.chunks, p.pix, at);
    });
}

template <typename T, int V, int ACT> hipError_t quantised_act(const NormArgs& a, void* ws, hipStream_t st) {
    const Plan p = make_plan(a.N, a.P, a.C, V);
    const int cv = (a.C + V - 1) / V;
    const bool wide = cv > 64;
    const size_t lds = (size_t)a.G * 8 + (wide ? (size_t)a.C * 12 : 0);
    if (lds > 65536) {
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e == hipSuccess) e = ensure_dynamic_lds<gn_quant_wide_kernel<T, V, ACT>>((int)lds, dev);
        if (e != hipSuccess) return e;
    }
    int lpp = 1;
    while (lpp < cv) lpp <<= 1;
    return in_launches(a, p.chunks, p.block, [&](const NormArgs& s, long long n) {
        float2* part = static_cast<float2*>(ws) + n * p.chunks * a.G;
        gn_stats_kernel<T, V><<<s.N * p.chunks, p.block, (size_t)p.R * a.C * 8, st>>>(s, p.TX, p.R, p.chunks, p.pix, part);
        if (wide) gn_quant_wide_kernel<T, V, ACT><<<s.N * p.chunks, 256, lds, st>>>(s, p.chunks, p.pix, part);
        else gn_quant_kernel<T, V, ACT><<<s.N * p.chunks, 256, lds, st>>>(s, lpp, p.chunks, p.pix, part);
    });
}

template <typename T, int V, int ACT> hipError_t quantised_whole(const NormArgs& a, hipStream_t st) {
    int lpp = 1;
    while (lpp * V < a.C) lpp <<= 1;
    const int subs = kWholeThreads / lpp;
    int chunks = kWholeBlocks / a.N;
    int pix = (a.P + chunks - 1) / chunks;
    pix = (pix + subs - 1) / subs * subs;
    chunks = (a.P + pix - 1) / pix;
    gn_quant_whole_kernel<T, V, ACT><<<a.N * chunks, kWholeThreads, ((size_t)subs * a.C + a.G) * 8, st>>>(a, lpp, chunks, pix);
    return hipGetLastError();
}

template <typename T, int V> hipError_t quantised(const NormArgs& a, int act, void* ws, hipStream_t st) {
    if (a.N <= kWholeBlocks && (a.C + V - 1) / V <= 64 && (long long)a.P * ((a.C + V - 1) / V) <= kWholeVectors)
        return act == kActSilu ? quantised_whole<T, V, kActSilu>(a, st)
               : act == kActRelu ? quantised_whole<T, V, kActRelu>(a, st) : quantised_whole<T, V, kActNone>(a, st);
    return act == kActSilu ? quantised_act<T, V, kActSilu>(a, ws, st)
           : act == kActRelu ? quantised_act<T, V, kActRelu>(a, ws, st) : quantised_act<T, V, kActNone>(a, ws, st);
}

template <typename T, int V, int ACT> hipError_t backward_resident(const NormArgs& a, const Resident& p, float* pc,
                                                                   hipStream_t st) {
    const size_t lds = (size_t)p.R * (a.C / a.G) * 8;
    auto run = [&](auto kernel_of) {
        constexpr auto kernel = kernel_of();
        hipError_t e = hipSuccess;
        if (lds > 60000) {   // 64 KB with the kernel's own few bytes
            int dev = 0;
            e = hipGetDevice(&dev);
            if (e == hipSuccess) e = ensure_dynamic_lds<kernel>((int)lds, dev);
        }
        if (e != hipSuccess) return e;
        return in_launches(a, a.G, p.block, [&](const NormArgs& s, long long n) {
            kernel<<<s.N * s.G, p.block, lds, st>>>(s, p.TX, p.R, a.N > 1 ? pc + n * 2 * a.C : nullptr);
        });
    };
    const hipError_t e = p.nv == 2 ? run([] { return gn_bwd_resident_kernel<T, V, ACT, 2>; })
                                    : run([] { return gn_bwd_resident_kernel<T, V, ACT, 4>; });
    if (e != hipSuccess) return e;
    if (a.N > 1 && param_blocks(a)) gn_params_kernel<<<param_blocks(a), 256, 0, st>>>(a, pc, a.N);
    return hipGetLastError();
}

template <typename T, int V, int ACT> hipError_t backward_act(const NormArgs& a, void* ws, hipStream_t st) {
    const Plan p = make_plan(a.N, a.P, a.C, V);
    const long long blocks = (long long)a.N * p.chunks;
    float2* pg = static_cast<float2*>(ws);
    float* pc = reinterpret_cast<float*>(pg + blocks * a.G);
    // threads of one or two pixels take them one by one: a batch of four would do
    // the arithmetic of four, with four times the code to fetch (15 images of
    // 18x46x108 in fp32: 13.4 us for 14.6; forward, with little of either, even)
    const bool few = p.pix <= 2 * p.R;
    auto first = few ? gn_bwd_sums_kernel<T, V, ACT, 1> : gn_bwd_sums_kernel<T, V, ACT, kBatchBwd>;
    auto second = few ? gn_bwd_apply_kernel<T, V, ACT, 1> : gn_bwd_apply_kernel<T, V, ACT, kBatchBwd>;
    const size_t lds = (size_t)(a.G > 2 * p.block ? a.G : 2 * p.block) * 8;
    // dgamma and dbeta along with dx, unless there are several launches of that
    int sums = param_blocks(a), launches = 0;
    const hipError_t e = in_launches(a, p.chunks, p.block, [&](const NormArgs& s, long long n) {
        ++launches;
        first<<<s.N * p.chunks, p.block, (size_t)p.R * a.C * 8, st>>>(s, p.TX, p.R, p.chunks, p.pix,
                                                                      pc + n * p.chunks * 2 * a.C, pg + n * p.chunks * a.G);
    });
    if (e != hipSuccess) return e;
    if (launches > 1 && sums) {
        gn_params_kernel<<<sums, 256, 0, st>>>(a, pc, blocks);
        sums = 0;
    }
    return in_launches(a, p.chunks, p.block, [&](const NormArgs& s, long long n) {
        second<<<sums + s.N * p.chunks, p.block, lds, st>>>(s, p.TX, p.R, p.chunks, p.pix, sums, pc, pg + n * p.chunks * a.G);
    });
}

template <typename T, int V> hipError_t backward(const NormArgs& a, int act, void* ws, hipStream_t st) {
    return act == kActSilu ? backward_act<T, V, kActSilu>(a, ws, st)
           : act == kActRelu ? backward_act<T, V, kActRelu>(a, ws, st) : backward_act<T, V, kActNone>(a, ws, st);
}

// The joined form: 256 threads, of which TX are the vectors of a pixel, R rows
// of them, nv vectors a thread; nv = 0 where it is not taken.
struct Joined {
    int TX, R, chunks, pix, nv;
    size_t lds;
};

// Vectors of a thread: with 16 four workgroups fit a compute unit's registers,
// with 7 of x and 7 of dz (as fp32) three.  Shorter chunks, of which more fit,
// wait more often (56x56x256 over 64 images backward: 7 vectors 103 us, 4
// vectors at four workgroups 127; forward 112x112x128 over 32, with fp32 sums:
// 55.7, at 8 vectors and six workgroups 64).
constexpr int kJoinedMost = 16, kJoinedMostBwd = 7;

// Bytes of x from which one read saves more than the clearing launch and the
// exchange cost (bf16, 256 channels of 56x56).  Forward: 3 MB 13.0 us against
// 12.5 streaming, 8 MB 13.3 against 17.0 (112x112x64 12.7 against 15.1), 16 MB 15.9
// against 19.4.  Quantised: 16 MB 19.6 against 21.0, 24 MB 25.1 against 25.4, 32
// MB 26.0 against 29.0.  Backward: 32 MB 44.5 against 38.2, 48 MB 57.9 against
// 56.7, 64 MB 70 against 75, 128 MB 123 against 146.
constexpr long long kJoinedBytes = 12 << 20, kJoinedBytesQuant = 24 << 20, kJoinedBytesBwd = 48 << 20;

// Every workgroup reads its image's words: at most a quarter of what it reads of x.
constexpr int kJoinedWords = 2048;

// Wider pixels leave a chunk few of them, and a chunk keeps 8 bytes a channel
// for dgamma and dbeta.
constexpr int kJoinedAcross = 64;

// The plan for 16-byte vectors of V elements, whatever the tensor's size.
// most: vectors of a thread (of x and of dy, where both are kept).
Joined plan_joined(int P, int C, int G, int V, bool quant, int most) {
    Joined p = {0, 0, 0, 0, 0, 0};
    const int cv = C / V;
    p.TX = cv;
    if (quant)
        for (p.TX = 1; p.TX < cv;) p.TX <<= 1;
    if (p.TX > kJoinedAcross) return p;
    p.R = 256 / p.TX;
    const long long per = (long long)p.R * most, chunks = (P + per - 1) / per;
    if (chunks * G > kJoinedWords) return p;
    long long each = (P + chunks - 1) / chunks;
    each = (each + p.R - 1) / p.R * p.R;
    p.pix = (int)each;
    p.chunks = (int)((P + each - 1) / each);
    p.nv = each / p.R > most / 2 ? most : most / 2;
    const int rows = p.R * C, words = (p.chunks + 1) * G;
    p.lds = (size_t)(rows > words ? rows : words) * 8;
    return p;
}

Joined make_joined(const NormArgs& a, int V, int elem, bool quant, int most) {
    Joined p = {0, 0, 0, 0, 0, 0};
    if (V * elem != 16) return p;
    if ((long long)a.N * a.P * a.C * elem < (a.dy ? kJoinedBytesBwd : quant ? kJoinedBytesQuant : kJoinedBytes)) return p;
    p = plan_joined(a.P, a.C, a.G, V, quant, most);
    // 32-bit offsets in a chunk, one step past its end included
    const long long ld = a.ldx > a.ldy ? (a.ldx > a.lddy ? a.ldx : a.lddy) : (a.ldy > a.lddy ? a.ldy : a.lddy);
    if ((long long)p.R * (p.nv + 1) * ld * elem > 0x7fffff00LL) p.nv = 0;
    return p;
}

hipError_t clear_words(void* ws, long long count, hipStream_t st) {
    const long long blocks = (count + 1023) / 1024;
    gn_clear_kernel<<<(int)(blocks < 1024 ? blocks : 1024), 256, 0, st>>>(static_cast<word_t*>(ws), count);
    return hipGetLastError();
}

template <typename T, int V, int ACT, bool QUANT>
hipError_t joined_act(const NormArgs& a, const Joined& p, void* ws, hipStream_t st) {
    const hipError_t e = clear_words(ws, (long long)a.N * p.chunks * a.G, st);
    if (e != hipSuccess) return e;
    auto k = p.nv == kJoinedMost ? gn_joined_kernel<T, V, ACT, kJoinedMost, QUANT>
                                 : gn_joined_kernel<T, V, ACT, kJoinedMost / 2, QUANT>;
    return in_launches(a, p.chunks, 256, [&](const NormArgs& s, long long n) {
        k<<<s.N * p.chunks, 256, p.lds, st>>>(s, p.TX, p.R, p.chunks, p.pix, wait_limit(),
                                              static_cast<word_t*>(ws) + n * p.chunks * a.G);
    });
}

template <typename T, int V, bool QUANT>
hipError_t joined(const NormArgs& a, int act, const Joined& p, void* ws, hipStream_t st) {
    return act == kActSilu ? joined_act<T, V, kActSilu, QUANT>(a, p, ws, st)
           : act == kActRelu ? joined_act<T, V, kActRelu, QUANT>(a, p, ws, st)
                             : joined_act<T, V, kActNone, QUANT>(a, p, ws, st);
}

template <typename T, int V, int ACT> hipError_t joined_bwd_act(const NormArgs& a, const Joined& p, void* ws, hipStream_t st) {
    const long long blocks = (long long)a.N * p.chunks;
    hipError_t e = clear_words(ws, blocks * a.G, st);
    if (e != hipSuccess) return e;
    word_t* words = static_cast<word_t*>(ws);
    float* pc = reinterpret_cast<float*>(words + blocks * a.G);
    auto k = p.nv == kJoinedMostBwd ? gn_bwd_joined_kernel<T, V, ACT, kJoinedMostBwd>
                                    : gn_bwd_joined_kernel<T, V, ACT, kJoinedMostBwd / 2>;
    e = in_launches(a, p.chunks, 256, [&](const NormArgs& s, long long n) {
        k<<<s.N * p.chunks, 256, p.lds, st>>>(s, p.TX, p.R, p.chunks, p.pix, wait_limit(), words + n * p.chunks * a.G,
                                              pc + n * p.chunks * 2 * a.C);
    });
    const int sums = param_blocks(a);
    if (e == hipSuccess && sums) {
        float* images = pc + blocks * 2 * a.C;
        e = in_launches(a, sums, 256, [&](const NormArgs& s, long long n) {
            gn_image_params_kernel<<<s.N * sums, 256, 0, st>>>(s, pc + n * p.chunks * 2 * a.C, p.chunks, sums, images + n * 2 * a.C);
        });
        if (e != hipSuccess) return e;
        gn_params_kernel<<<sums, 256, 0, st>>>(a, images, a.N);
        e = hipGetLastError();
    }
    return e;
}

template <typename T, int V> hipError_t joined_bwd(const NormArgs& a, int act, const Joined& p, void* ws, hipStream_t st) {
    return act == kActSilu ? joined_bwd_act<T, V, kActSilu>(a, p, ws, st)
           : act == kActRelu ? joined_bwd_act<T, V, kActRelu>(a, p, ws, st)
                             : joined_bwd_act<T, V, kActNone>(a, p, ws, st);
}

}  // namespace

// The most partials that any vector width plans, so that one figure holds for
// every alignment (the resident backward pass keeps at most a pair per image
// and channel, which is less).
size_t group_norm_workspace(int N, int P, int C, int G, int backward) {
    size_t most = 0;
    for (int v = 1; v <= 8 && v <= C; v <<= 1) {
        const Plan p = make_plan(N, P, C, v);
        const size_t bytes = (size_t)N * p.chunks * (G + (backward ? (size_t)C : 0)) * 8;
        most = bytes > most ? bytes : most;
    }
    for (int v = 4; v <= 8; v <<= 1)
        for (int quant = 0; quant < (backward ? 1 : 2); ++quant) {
            if (C % v) break;
            const Joined p = plan_joined(P, C, G, v, quant, backward ? kJoinedMostBwd : kJoinedMost);
            const size_t bytes = p.nv ? (size_t)N * (p.chunks * (G + (backward ? (size_t)C : 0)) + (backward ? C : 0)) * 8 : 0;
            most = bytes > most ? bytes : most;
        }
    return most;
}

#define CONV2D_NORM_WIDTH(FN, WIDTH, ...)                                                           \
    const int v = WIDTH;                                                                            \
    if (a.dtype == 0 /* CONV2D_F32 */) {                                                            \
        return v == 4 ? FN<float, 4>(__VA_ARGS__) : v == 2 ? FN<float, 2>(__VA_ARGS__) : FN<float, 1>(__VA_ARGS__); \
    }                                                                                               \
    return v == 8 ? FN<bf16_t, 8>(__VA_ARGS__) : v == 4 ? FN<bf16_t, 4>(__VA_ARGS__)                \
           : v == 2 ? FN<bf16_t, 2>(__VA_ARGS__) : FN<bf16_t, 1>(__VA_ARGS__)

template <typename T, int V>
static hipError_t forward_group(const NormArgs& a, int act, const Resident& p, hipStream_t st) {
    return act == kActSilu ? forward_resident<T, V, kActSilu>(a, p, st)
           : act == kActRelu ? forward_resident<T, V, kActRelu>(a, p, st) : forward_resident<T, V, kActNone>(a, p, st);
}
template <typename T, int V>
static hipError_t backward_group(const NormArgs& a, int act, const Resident& p, float* pc,
                                                              hipStream_t st) {
    return act == kActSilu ? backward_resident<T, V, kActSilu>(a, p, pc, st)
           : act == kActRelu ? backward_resident<T, V, kActRelu>(a, p, pc, st)
                             : backward_resident<T, V, kActNone>(a, p, pc, st);
}

hipError_t launch_group_norm(const NormArgs& a, int act, void* ws, hipStream_t st) {
    const int elem = a.dtype == 0 ? 4 : 2, cg = a.C / a.G;
    const Resident p = make_resident(a, vector_width(a, cg, elem, elem), elem, 8);
    if (p.nv) {
        CONV2D_NORM_WIDTH(forward_group, vector_width(a, cg, elem, elem), a, act, p, st);
    }
    const Joined j = make_joined(a, vector_width(a, a.C, elem, elem), elem, false, kJoinedMost);
    if (j.nv) return elem == 4 ? joined<float, 4, false>(a, act, j, ws, st) : joined<bf16_t, 8, false>(a, act, j, ws, st);
    CONV2D_NORM_WIDTH(forward, row_width(a, elem, elem), a, act, ws, st);
}

hipError_t launch_group_norm_quant(const NormArgs& a, int act, void* ws, hipStream_t st) {
    const int elem = a.dtype == 0 ? 4 : 2;
    const Joined j = make_joined(a, vector_width(a, a.C, elem, 1), elem, true, kJoinedMost);
    if (j.nv) return elem == 4 ? joined<float, 4, true>(a, act, j, ws, st) : joined<bf16_t, 8, true>(a, act, j, ws, st);
    CONV2D_NORM_WIDTH(quantised, row_width(a, elem, 1), a, act, ws, st);
}

hipError_t launch_group_norm_bwd(const NormArgs& a, int act, void* ws, hipStream_t st) {
    const int elem = a.dtype == 0 ? 4 : 2, cg = a.C / a.G;
    const Resident p = make_resident(a, vector_width(a, cg, elem, elem), elem, 4);
    if (p.nv) {
        CONV2D_NORM_WIDTH(backward_group, vector_width(a, cg, elem, elem), a, act, p, static_cast<float*>(ws), st);
    }
    const Joined j = make_joined(a, vector_width(a, cg, elem, elem), elem, false, kJoinedMostBwd);
    if (j.nv) return elem == 4 ? joined_bwd<float, 4>(a, act, j, ws, st) : joined_bwd<bf16_t, 8>(a, act, j, ws, st);
    CONV2D_NORM_WIDTH(backward, row_width(a, elem, elem), a, act, ws, st);
}

}  // namespace conv2d
