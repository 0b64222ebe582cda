// rms_norm.hip -- root-mean-square norm of rows, with the addition of a
// residual before it, the norm in 8 bits for each row, and its gradients.
//
//   h = x + residual,  rstd = 1 / sqrt(sum_c h^2 / C + eps),  y = h rstd gamma
//   backward, with xh = h rstd and t = gamma dy:
//     dx = rstd (t - xh sum_c(t xh) / C) + dh,   dgamma[c] = sum_m dy xh
//
// Bound by memory.  A row lives in the registers of its lanes (a part of a
// wave, a wave, or a workgroup of up to 1024 threads), so each tensor passes
// once, a row is read whole before it is written (the outputs may lie over the
// inputs), and one reduction over the lanes joins a row's sum.  Workgroups walk
// rows, with gamma (and dgamma's sums) in registers.  16384 x 4096 bf16 with the
// residual: 100 us forward and 99 backward, 5.4 TB/s of what has to move.
#include "operators.hpp"
#include "rowvec.hpp"

namespace conv2d {

namespace {

constexpr int kThreads = 256;   // of a workgroup, more where a row has more lanes

// Lanes, and 16-byte vectors of a lane, that hold a row.
struct RowShape {
    int vec, lanes, per;
};

// The first elements of the row's last vector that belong to the one before it
// too (vector_start): they count once in the row's sums.
template <int V> __device__ __forceinline__ int shared_elements(int c, int C) { return c - vector_start<V>(c, C); }

template <int V> __device__ __forceinline__ void load_floats(const float* p, float (&v)[V]) {
    if constexpr (V > 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            float u[4];
            Vec<float, 4>::unpack(Vec<float, 4>::load(p + k), u);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k + e] = u[e];
        }
    } else {
        Vec<float, V>::unpack(Vec<float, V>::load(p), v);
    }
}
template <int V> __device__ __forceinline__ void store_floats(float* p, const float (&v)[V]) {
    if constexpr (V > 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4) Vec<float, 4>::store(p + k, {v[k], v[k + 1], v[k + 2], v[k + 3]});
    } else {
        Vec<float, V>::store(p, v);
    }
}

// Sum over a row's lanes; `red`: 16 values for the waves of a row of more than
// one (then the row has the workgroup alone).
template <typename S> __device__ __forceinline__ S row_sum(S v, int lanes, S* red) {
    v = lanes_sum(v, lanes < 64 ? lanes : 64);
    if (lanes <= 64) return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < lanes >> 6; ++w) v += red[w];
    return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, int lanes, uint32_t* red) {
    v = lanes_max(v, lanes < 64 ? lanes : 64);
    if (lanes <= 64) return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < lanes >> 6; ++w) v = max(v, red[w]);
    return v;
}

// 1 / rms from the row's values.  fp32 squares, unless their sum leaves the
// range where they are exact to their last bits (values above 2^60 or a row
// below 2^-40): then once more in fp64, where none overflows or vanishes.
template <int V, int J>
__device__ __forceinline__ float row_rstd(const float (&h)[J][V], int l, int lanes, int C, float eps, double* red) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * lanes) * V;
        if (c >= C) break;
        const int skip = shared_elements<V>(c, C);
#pragma unroll
        for (int e = 0; e < V; ++e) s += e >= skip ? h[j][e] * h[j][e] : 0.0f;
    }
    s = row_sum(s, lanes, reinterpret_cast<float*>(red));
    if (s >= 0x1p-80f && s <= 0x1p120f) return 1.0f / sqrtf(s / (float)C + eps);
    double d = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * lanes) * V;
        if (c >= C) break;
        const int skip = shared_elements<V>(c, C);
#pragma unroll
        for (int e = 0; e < V; ++e) d += e >= skip ? (double)h[j][e] * h[j][e] : 0.0;
    }
    return (float)(1.0 / sqrt(row_sum(d, lanes, red) / C + (double)eps));
}

// Whether the next row's loads are in flight while one is normalised: rows of one
// vector a lane have few otherwise (100352 x 256 bf16: 47.8 us without, 43.3 with;
// gradients 46.0 and 44.4; but 16384 x 4096, two vectors a lane, 104 and 107).
template <int J> constexpr bool kAhead = J == 1;

// `lanes` threads a row, J vectors of V elements a thread.
template <typename T, int V, int J, int NT, bool QUANT>
__global__ __launch_bounds__(NT) void rms_norm_kernel(RmsArgs a, int lanes) {
    __shared__ double red[16];
    const int l = threadIdx.x % lanes, rows = blockDim.x / lanes;
    float gamma[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * lanes) * V;
        if (c >= a.C) break;
        if (a.gamma) load_floats<V>(a.gamma + vector_start<V>(c, a.C), gamma[j]);
        else
#pragma unroll
            for (int e = 0; e < V; ++e) gamma[j][e] = 1.0f;
    }
    // a row of several waves has the workgroup alone, so that barriers are met by all
    const long long step = (long long)gridDim.x * rows;
    typename Vec<T, V>::raw x[J], r[J];
    auto fetch = [&](long long row) __attribute__((always_inline)) {
        const T* const px = static_cast<const T*>(a.x) + row * a.ldx;
        const T* const pr = static_cast<const T*>(a.residual) + (a.residual ? row * a.ldr : 0);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + j * lanes) * V;
            if (c >= a.C) break;
            x[j] = Vec<T, V>::load(px + vector_start<V>(c, a.C));
            if (a.residual) r[j] = Vec<T, V>::load(pr + vector_start<V>(c, a.C));
        }
    };
    long long row = (long long)blockIdx.x * rows + threadIdx.x / lanes;
    if (kAhead<J> && row < a.M) fetch(row);
    for (; row < a.M; row += step) {
        if (!kAhead<J>) fetch(row);
        float h[J][V];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if ((l + j * lanes) * V >= a.C) break;
            Vec<T, V>::unpack(x[j], h[j]);
            if (a.residual) {
                float v[V];
                Vec<T, V>::unpack(r[j], v);
#pragma unroll
                for (int e = 0; e < V; ++e) h[j][e] += v[e];
            }
        }
        if (kAhead<J> && row + step < a.M) fetch(row + step);
        const float rstd = row_rstd<V, J>(h, l, lanes, a.C, a.eps, red);
        if (a.rstd && l == 0) a.rstd[row] = rstd;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + j * lanes) * V;
            if (c >= a.C) break;
            if (a.h) Vec<T, V>::store(static_cast<T*>(a.h) + row * a.ldh + vector_start<V>(c, a.C), h[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[j][e] = h[j][e] * rstd * gamma[j][e];
                top = max(top, __float_as_uint(h[j][e]) & 0x7fffffffu);
            }
            if constexpr (!QUANT) Vec<T, V>::store(static_cast<T*>(a.y) + row * a.ldy + vector_start<V>(c, a.C), h[j]);
        }
        if constexpr (QUANT) {
            const RowScale s = row_scale(row_max(top, lanes, reinterpret_cast<uint32_t*>(red)));
            if (l == 0) a.q_scale[row] = s.scale;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (l + j * lanes) * V;
                if (c >= a.C) break;
                store_quantised<V>(static_cast<int8_t*>(a.y) + row * a.ldy + vector_start<V>(c, a.C), h[j], s.inv);
            }
        }
    }
}

// Partial sums of dgamma: [workgroup][C], a lane's over its rows in fp32, a workgroup's
// over its lanes in fp64, rounded once.
template <typename T, int V, int J, int NT>
__global__ __launch_bounds__(NT) void rms_norm_bwd_kernel(RmsArgs a, int lanes, float* sums) {
    __shared__ float red[16];
    extern __shared__ float joined[];   // [rows of a workgroup][C]
    const int l = threadIdx.x % lanes, group = threadIdx.x / lanes, rows = blockDim.x / lanes;
    float gamma[J][V], dgamma[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * lanes) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            dgamma[j][e] = 0.0f;
            gamma[j][e] = 1.0f;
        }
        if (c < a.C && a.gamma) load_floats<V>(a.gamma + vector_start<V>(c, a.C), gamma[j]);
    }
    const long long step = (long long)gridDim.x * rows;
    typename Vec<T, V>::raw x[J], d[J], r[J], dh[J];
    float next_rstd;
    auto fetch = [&](long long row) __attribute__((always_inline)) {
        const T* const ph = static_cast<const T*>(a.h) + row * a.ldh;
        const T* const pd = static_cast<const T*>(a.x) + row * a.ldx;
        const T* const pr = static_cast<const T*>(a.residual) + (a.residual ? row * a.ldr : 0);
        next_rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + j * lanes) * V;
            if (c >= a.C) break;
            x[j] = Vec<T, V>::load(ph + vector_start<V>(c, a.C));
            d[j] = Vec<T, V>::load(pd + vector_start<V>(c, a.C));
            if (a.residual) r[j] = Vec<T, V>::load(pr + vector_start<V>(c, a.C));
        }
    };
    long long row = (long long)blockIdx.x * rows + group;
    if (kAhead<J> && row < a.M) fetch(row);
    for (; row < a.M; row += step) {
        if (!kAhead<J>) fetch(row);
        const float rstd = next_rstd;
        float xh[J][V], t[J][V], s = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + j * lanes) * V;
            if (c >= a.C) break;
            const int skip = shared_elements<V>(c, a.C);
            Vec<T, V>::unpack(x[j], xh[j]);
            Vec<T, V>::unpack(d[j], t[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                xh[j][e] *= rstd;
                dgamma[j][e] = fmaf(t[j][e], xh[j][e], dgamma[j][e]);
                t[j][e] *= gamma[j][e];
                s += e >= skip ? t[j][e] * xh[j][e] : 0.0f;
            }
            dh[j] = r[j];
        }
        if (kAhead<J> && row + step < a.M) fetch(row + step);
        const float mean = row_sum(s, lanes, red) / (float)a.C;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + j * lanes) * V;
            if (c >= a.C) break;
            float v[V] = {};
            if (a.residual) Vec<T, V>::unpack(dh[j], v);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = fmaf(rstd, t[j][e] - xh[j][e] * mean, v[e]);
            Vec<T, V>::store(static_cast<T*>(a.y) + row * a.ldy + vector_start<V>(c, a.C), v);
        }
    }
    if (!sums) return;
    sums += (long long)blockIdx.x * a.C;
    if (rows == 1) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + j * lanes) * V;
            if (c < a.C) store_floats<V>(sums + vector_start<V>(c, a.C), dgamma[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * lanes) * V;
        if (c < a.C) store_floats<V>(joined + group * a.C + vector_start<V>(c, a.C), dgamma[j]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        double s = 0.0;
        for (int g = 0; g < rows; ++g) s += joined[g * a.C + c];
        sums[c] = (float)s;
    }
}

// The workgroups' sums of each column, added: COLS columns a workgroup, 1024 / COLS
// threads a column.  32 columns are whole lines, 16 leave more threads to a column (777
// sums of 1001 columns: 4.2 us, with 16 threads a column 6.5).
template <int COLS>
__global__ __launch_bounds__(1024) void join_columns_kernel(const float* sums, float* out, int count, int C) {
    constexpr int GROUPS = 1024 / COLS;
    __shared__ double part[COLS][GROUPS + 1];
    const int first = blockIdx.x * COLS, column = threadIdx.x % COLS, c = first + column, k = threadIdx.x / COLS;
    double s = 0.0;
    if (c < C) {
#pragma unroll 8
        for (int i = k; i < count; i += GROUPS) s += sums[(long long)i * C + c];
    }
    part[column][k] = s;
    __syncthreads();
    const int row = threadIdx.x / GROUPS, lane = threadIdx.x % GROUPS;   // GROUPS lanes add a column
    const double t = lanes_sum(part[row][lane], GROUPS);
    if (lane == 0 && first + row < C) out[first + row] = (float)t;
}

// ------------------------------------------------------------------ host

// Elements of a vector: 16 bytes whatever the alignment, the last vector of a
// row over part of the one before, unless the row is shorter.
int vector_elements(int C, int es) {
    int v = 16 / es;
    while (v > C) v >>= 1;
    return v;
}

// 16 elements a lane at most: with 32 the gradients' sums leave the registers (with 1024
// threads a row and fp32 they do already: 4096 x 16384 300 us, 3.5 TB/s).
constexpr int kMostElements = 16;

RowShape row_shape(int M, int C, int es) {
    RowShape s;
    s.vec = vector_elements(C, es);
    const int vecs = (C + s.vec - 1) / s.vec;
    // few rows: a vector a lane; many: as many as give a row to one wave.  Lanes are a power
    // of two, so a row just longer than one has half of its lanes nearly empty (3699 x 8256
    // bf16 65 us, 8192 columns 47.6)
    s.lanes = 1;
    const int per = M >= 1024 ? kMostElements / s.vec : 1;
    while (s.lanes < 1024 && s.lanes * (s.lanes < 64 ? 1 : per) < vecs) s.lanes <<= 1;
    s.per = (vecs + s.lanes - 1) / s.lanes;
    return s;
}

int block_of(const RowShape& s) { return s.lanes > 64 ? s.lanes : kThreads; }

template <typename T, int V, int J, int NT, bool QUANT> hipError_t forward(const RmsArgs& a, const RowShape& s, hipStream_t st) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const int threads = block_of(s), rows = threads / s.lanes;
    const long long all = ((long long)a.M + rows - 1) / rows;
    // four waves for every vector unit (16384 x 4096 bf16 99.8 us, with eight 106.9)
    const long long most = (long long)cu_count(dev) * (1024 / threads);
    rms_norm_kernel<T, V, J, NT, QUANT><<<(unsigned)(all < most ? all : most), threads, 0, st>>>(a, s.lanes);
    return hipGetLastError();
}

// Rows that a lane sums in fp32 before fp64 takes over.
constexpr int kMostRows = 512;

// Workgroups of the gradients, each with sums of its own to join: two waves for every
// vector unit, or one workgroup for every compute unit, of at least two rows (16384 x
// 4096 bf16: 98.8 us with 512 workgroups, 104 with 768, 107 with 1024).
long long bwd_blocks(int M, const RowShape& s) {
    const int threads = block_of(s), rows = threads / s.lanes;
    const long long all = ((long long)M + rows - 1) / rows, least = (all + kMostRows - 1) / kMostRows;
    long long blocks = 2 * 4 * 64 * 256 / threads;
    if (blocks > (all + 1) / 2) blocks = (all + 1) / 2;
    if (blocks < 256) blocks = 256;
    if (blocks > all) blocks = all;
    return blocks > least ? blocks : least;
}

template <typename T, int V, int J, int NT> hipError_t backward(const RmsArgs& a, const RowShape& s, float* sums, hipStream_t st) {
    const int threads = block_of(s), rows = threads / s.lanes;
    const long long blocks = bwd_blocks(a.M, s);
    rms_norm_bwd_kernel<T, V, J, NT><<<(unsigned)blocks, threads, a.dgamma && rows > 1 ? rows * a.C * 4 : 0, st>>>(
        a, s.lanes, a.dgamma ? sums : nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dgamma) return e;
    return launch_join_columns(sums, a.dgamma, (int)blocks, a.C, st);
}

enum Pass { kForward, kQuant, kBackward };

template <Pass P, typename T, int V, int J, int NT = kThreads> hipError_t run(const RmsArgs& a, const RowShape& s, float* sums, hipStream_t st) {
    if constexpr (P == kBackward) return backward<T, V, J, NT>(a, s, sums, st);
    else return forward<T, V, J, NT, P == kQuant>(a, s, st);
}

template <Pass P, typename T, int V, int NT> hipError_t by_count(const RmsArgs& a, const RowShape& s, float* sums, hipStream_t st) {
    if (s.per == 1) return run<P, T, V, 1, NT>(a, s, sums, st);
    if constexpr (V == 4)
        if (s.per > 2) return run<P, T, V, 4, NT>(a, s, sums, st);
    return run<P, T, V, 2, NT>(a, s, sums, st);
}

template <Pass P, typename T, int V> hipError_t by_lanes(const RmsArgs& a, const RowShape& s, float* sums, hipStream_t st) {
    return s.lanes <= kThreads ? by_count<P, T, V, kThreads>(a, s, sums, st)
           : s.lanes <= 512 ? by_count<P, T, V, 512>(a, s, sums, st) : by_count<P, T, V, 1024>(a, s, sums, st);
}

template <Pass P> hipError_t launch(const RmsArgs& a, float* sums, hipStream_t st) {
    const bool f32 = a.dtype == 0 /* CONV2D_F32 */;
    const RowShape s = row_shape(a.M, a.C, f32 ? 4 : 2);
    if (f32)
        return s.vec == 4 ? by_lanes<P, float, 4>(a, s, sums, st)
               : s.vec == 2 ? run<P, float, 2, 1>(a, s, sums, st) : run<P, float, 1, 1>(a, s, sums, st);
    return s.vec == 8 ? by_lanes<P, bf16_t, 8>(a, s, sums, st)
           : s.vec == 4 ? run<P, bf16_t, 4, 1>(a, s, sums, st)
           : s.vec == 2 ? run<P, bf16_t, 2, 1>(a, s, sums, st) : run<P, bf16_t, 1, 1>(a, s, sums, st);
}

}  // namespace

hipError_t launch_join_columns(const float* sums, float* out, int count, int C, hipStream_t st) {
    if (C >= 2048) join_columns_kernel<32><<<(C + 31) / 32, 1024, 0, st>>>(sums, out, count, C);
    else join_columns_kernel<16><<<(C + 15) / 16, 1024, 0, st>>>(sums, out, count, C);
    return hipGetLastError();
}

// One figure for either type.
size_t rms_norm_bwd_workspace(int M, int C) {
    const long long u = bwd_blocks(M, row_shape(M, C, 2)), v = bwd_blocks(M, row_shape(M, C, 4));
    return (size_t)(u > v ? u : v) * C * 4;
}

hipError_t launch_rms_norm(const RmsArgs& a, hipStream_t st) { return launch<kForward>(a, nullptr, st); }
hipError_t launch_rms_norm_quant(const RmsArgs& a, hipStream_t st) { return launch<kQuant>(a, nullptr, st); }
hipError_t launch_rms_norm_bwd(const RmsArgs& a, void* ws, hipStream_t st) {
    return launch<kBackward>(a, static_cast<float*>(ws), st);
}

}  // namespace conv2d
