// dropout.hip -- dropout of rows, with an optional residual:
//
//   y[m][c] = residual[m][c] + (word(m, c) >= p 2^32 ? x[m][c] / (1 - p) : 0)
//
// word(m, c) is one 32-bit word of a counter-based generator, so the mask is
// computed where it is needed and never stored, and the gradient is the same
// call on dy.  The generator is Philox4x32 with 10 rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): a
// counter of four words, (c / 4, m, offset), goes through rounds of two
// 32x32 -> 64-bit products and exclusive ors under the key, the seed, and word
// c % 4 of the result is the element's.
//
// Bound by memory, behind which the words' arithmetic (20 products of a quarter of the
// rate for 4 elements) hides: 16384 x 4096 bf16 with a residual 78 us, 5.1 TB/s, and 54
// without one, where it hides just so.
#include "operators.hpp"
#include "rowvec.hpp"

namespace conv2d {

namespace {

__device__ __forceinline__ void words4(uint32_t col4, uint32_t row, uint64_t seed, uint64_t offset, uint32_t (&w)[4]) {
    uint32_t c0 = col4, c1 = row, c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

// V elements at columns c .. c + V - 1 (c a multiple of V, V of 4).
template <typename T, int V>
__device__ __forceinline__ void drop(float (&v)[V], const float (&r)[V], int c, int row, uint64_t seed, uint64_t offset,
                                     uint32_t threshold, float scale) {
#pragma unroll
    for (int g = 0; g < V / 4; ++g) {
        uint32_t w[4];
        words4((uint32_t)(c / 4 + g), (uint32_t)row, seed, offset, w);
#pragma unroll
        // selected, not multiplied by 0: a NaN or infinity that is dropped is gone
        for (int e = 0; e < 4; ++e) v[4 * g + e] = r[4 * g + e] + (w[e] >= threshold ? v[4 * g + e] * scale : 0.0f);
    }
}

// Threads walk the rows' vectors in order, `gridDim.x * 256` vectors (step_rows
// rows and step_vecs vectors) at a time.
template <typename T, int V, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, int vecs, long long step_rows, int step_vecs) {
    const uint64_t seed = a.rng[0], offset = a.rng[1];
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    long long row = i / vecs;
    int vec = (int)(i - row * vecs);
    while (row < a.M) {
        const int c = vec * V;
        const T* x = static_cast<const T*>(a.x) + row * a.ldx + c;
        const T* r = static_cast<const T*>(a.residual) + (RES ? row * a.ldr + c : 0);
        T* y = static_cast<T*>(a.y) + row * a.ldy + c;
        float v[V], rv[V] = {};
        if (c <= a.C - V) {   // (c + V may pass 2^31)
            Vec<T, V>::unpack(Vec<T, V>::load(x), v);
            if constexpr (RES) Vec<T, V>::unpack(Vec<T, V>::load(r), rv);
            drop<T, V>(v, rv, c, (int)row, seed, offset, a.threshold, a.scale);
            Vec<T, V>::store(y, v);
        } else {
            // a row's end: shifted into place where that saves loads (65536 x 1004 bf16: 100
            // us, element by element 110; 65536 x 1001 fp32: 176 and 158)
            if constexpr (V > 4) {
                typedef typename Vec<T, V>::raw raw;
                Vec<T, V>::unpack(__builtin_bit_cast(raw, load_piece<T>(x, a.C - c, a.C)), v);
                if constexpr (RES) Vec<T, V>::unpack(__builtin_bit_cast(raw, load_piece<T>(r, a.C - c, a.C)), rv);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[e] = c + e < a.C ? load_f32<T>(x, e) : 0.0f;
                    if constexpr (RES) rv[e] = c + e < a.C ? load_f32<T>(r, e) : 0.0f;
                }
            }
            drop<T, V>(v, rv, c, (int)row, seed, offset, a.threshold, a.scale);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c + e < a.C) store_f32<T>(y, e, v[e]);
        }
        row += step_rows;
        vec += step_vecs;
        if (vec >= vecs) {
            vec -= vecs;
            ++row;
        }
    }
}

template <typename T, bool RES> hipError_t dropout(const DropoutArgs& a, hipStream_t st) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    constexpr int V = 16 / (int)sizeof(T);
    constexpr auto kernel = dropout_kernel<T, V, RES>;
    const int vecs = a.C / V + (a.C % V != 0);
    const long long all = ((long long)a.M * vecs + 255) / 256;
    const long long most = (long long)cu_count(dev) * blocks_per_cu<kernel>(256, dev);
    const long long blocks = all < most ? all : most;
    kernel<<<(unsigned)blocks, 256, 0, st>>>(a, vecs, blocks * 256 / vecs, (int)(blocks * 256 % vecs));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st) {
    if (a.dtype == 0 /* CONV2D_F32 */) return a.residual ? dropout<float, true>(a, st) : dropout<float, false>(a, st);
    return a.residual ? dropout<bf16_t, true>(a, st) : dropout<bf16_t, false>(a, st);
}

}  // namespace conv2d
