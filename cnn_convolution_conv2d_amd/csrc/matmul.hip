// matmul.hip -- products of fp32 or bf16 rows with bias, activation and residual
// in the epilogue, and their gradients.
//
//   forward    z = x w^T + bias,  y = act(z) + residual      sums over k
//   backward   dz = dy act'(z),   dx = dz w                  sums over n
//                                 dw = dz^T x,  dbias = sum dz   sums over m
//
// All three are one product, C[r][c] = sum_s B(r, s) A(c, s), whose operands lie
// in memory with the summed index s either contiguous (rows of s) or strided (a
// row for every s): forward A = w and B = x contiguous; dx A = w strided; dw A = x
// and B = dz both strided.  An operand comes into LDS as it lies in memory, and is
// turned on the way to the registers.
//
// A workgroup has a tile of C and walks s in stages of 128 bytes.  The matrix unit
// takes 16 bytes of s of a lane: 8 bf16 in one 16x16x32 product, 4 fp32 in
// four 16x16x4 (which see s in another order, the same for both operands).  Tiles
// of few results and a long s are split along s; the pieces' fp32 sums go to the
// workspace and a second launch adds them, in order, and finishes.
//
//   tile    aligned operands: stages copied from memory into two LDS buffers without
//           passing through registers, tiles of 256, 128 or 64.  8192^3 bf16 with bias, SiLU
//           and residual: 806 us, 1364 TFLOP/s (770 without the epilogue; the matrix units
//           are busy for 71% of the cycles, at the 1.7 GHz that the socket's power leaves);
//           dx and dw of 8192 x 4096 -> 4096: 194 and 190 us, 1430 TFLOP/s.  fp32, 4096^3:
//           938 us, 147 TFLOP/s; dx 920, dw 954, whose 256 registers leave 7 in scratch.  No
//           bank conflicts, in transposing reads neither.
//   staged  operands of any alignment, through registers.  Where K is no whole number of
//           16-byte pieces, large products copy x and w to whole pieces first and take the
//           tiles.  A whole K with other strides or addresses is not copied: 4096^3 bf16 with
//           rows 4097 apart 217 us, 4096 apart 114.
//   skinny  up to 32 rows of the forward product: the weights stream through registers.
//           One row of 4096, 16384 columns: 134 MB in 26.7 us, 5.0 TB/s.
#include <type_traits>

#include "matmul_plan.hpp"
#include "operators.hpp"
#include "tiles.hpp"

namespace conv2d {

namespace {

enum { kGelu = 3 };   // CONV2D_ACT_GELU; the others as in rowvec.hpp

// 1 - Phi(x), Phi the standard normal's distribution function, for x >= 0:
// exp(-x^2 / 2) times a polynomial in 1 / (1 + 0.3 x), fitted by least squares of the
// relative error, weighted towards its maximum, up to x = 15 (6e-8).  In fp32 the
// exponential's argument is off by up to 3 u of itself (u = 2^-24), 1.5 x^2 u of the
// value, beside some 7 u of the other steps: 7 u up to x = 1, 10 u up to 3, 23 u up to
// 5, 125 u up to 13.  So GELU keeps most of its digits on the negative side, where
// 1 + erf has none left, and as many as z's own rounding (x^2 u there) leaves it.
__device__ __forceinline__ float normal_above(float x) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, x, 1.0f));
    float q = 3.842540085315704e-2f;
    q = fmaf(q, t, -1.6939479112625122e-1f);
    q = fmaf(q, t, 2.2913166880607605e-1f);
    q = fmaf(q, t, -7.704469561576843e-2f);
    q = fmaf(q, t, 1.429063081741333e-1f);
    q = fmaf(q, t, 9.452608972787857e-2f);
    q = fmaf(q, t, 1.2196046113967896e-1f);
    q = fmaf(q, t, 1.1948209255933762e-1f);
    q = fmaf(q, t, 7.495440513594076e-6f);
    return q * __builtin_amdgcn_exp2f(x * x * -0.72134752044448170f);   // log2(e) / 2
}

__device__ __forceinline__ float normal_below(float z) {
    const float above = normal_above(fabsf(z));
    return z > 0.0f ? 1.0f - above : above;
}

// V values; one choice for all of them.
template <int V> __device__ __forceinline__ void activate(float (&v)[V], int act) {
    if (act == kActRelu) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = v[e] < 0.0f ? 0.0f : v[e];
    } else if (act == kActSilu) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= sigmoid(v[e]);
    } else if (act == kGelu) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= normal_below(v[e]);
    }
}

__device__ __forceinline__ float activation_slope(float z, int act) {
    if (act == kActRelu) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;   // of a NaN: NaN
    if (act == kActSilu) {
        const float e = sigmoid(z);
        return e * (1.0f + z * (1.0f - e));
    }
    // Phi(z) + z phi(z)
    return normal_below(z) + z * 0.398942280401432678f * __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
}

// One product C[r][c], r < rows, c < cols, sums over s < K.
struct Product {
    const void* a;          // columns' operand: [cols][K], or [K][cols] strided
    const void* b;          // rows' operand: [rows][K], or [K][rows] strided
    long long lda, ldb;
    int rows, cols, K;
    const float* bias;      // the epilogue: null where there is none
    const void* residual;
    void* z;
    void* y;
    long long ldr, ldz, ldy;
    int act;
};

// ------------------------------------------------------------------ fragments

// A lane's 16 bytes of s of one row of a 16x16 block.
template <typename T> struct Frag;
template <> struct Frag<bf16_t> {
    bf16x8 v;
};
template <> struct Frag<float> {
    f32x4 v;
};

__device__ __forceinline__ void multiply(f32x4& acc, const Frag<bf16_t>& a, const Frag<bf16_t>& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void multiply(f32x4& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], acc, 0, 0, 0);
}

// Neighbours share an operand, the turns of the order included.
template <typename T, int TI, int TJ>
__device__ __forceinline__ void products(f32x4 (&acc)[TI][TJ], const Frag<T> (&a)[TI], const Frag<T> (&b)[TJ]) {
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int n = 0; n < TI; ++n) {
            const int i = j & 1 ? TI - 1 - n : n;
            multiply(acc[i][j], a[i], b[j]);
        }
}

// ---- a stage of an operand in LDS: 128 bytes of s of B indexes.
//
// Contiguous: a row of 128 bytes for every index, its 16-byte pieces permuted
// (slot_of).  Strided: a row of B elements for every s, in blocks of 16 indexes;
// the blocks of a row are permuted by a few bits of s, so that the rows that are
// read together (bf16: 8 of them half a wave, 32 bytes of each; fp32: 4 of a
// wave, 64 bytes of each) lie in different banks.
template <typename T, int B> __device__ __forceinline__ int block_swizzle(int s) {
    if constexpr (sizeof(T) == 4) return (s >> 2) & 3;
    else if constexpr (B >= 128) return (s & 3) | ((s >> 1) & 4);   // rows 0-3 and 8-11, or 4-7 and 12-15
    else return ((s >> 1) & 1) | ((s >> 2) & 2);                    // two rows to a line of the banks
}

// Byte of element c (a multiple of 16 bytes) of row s of a strided stage.
template <typename T, int B> __device__ __forceinline__ int strided_byte(int s, int c) {
    constexpr int ES = (int)sizeof(T);
    return s * B * ES + ((c >> 4) ^ block_swizzle<T, B>(s)) * 16 * ES + (c & 15) * ES;
}

// A lane's fragment of block `block` of 16 indexes, step `step` (0 or 1) of 64 bytes
// of s, of the operand `base` bytes into a stage.  The whole offset is one sum: the
// compiler follows a short chain of additions from a buffer to an access, and takes a
// read at the end of a longer one to need every copy in flight.
template <typename T, int B, bool STRIDED>
__device__ __forceinline__ Frag<T> fragment(const char* stage, int base, int block, int step) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    Frag<T> f;
    if constexpr (!STRIDED) {
        f.v = *reinterpret_cast<const decltype(f.v)*>(stage + (base + block * 16 * kStageK + slot_of(i, 4 * step + g) * 16));
    } else if constexpr (sizeof(T) == 4) {
        const int at = base + 4 * g * B * 4 + (block ^ block_swizzle<T, B>(4 * g)) * 64 + i * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.v[j] = *reinterpret_cast<const float*>(stage + (at + (16 * step + j) * B * 4));
    } else {
        // the transposing read: 16 lanes name the 8-byte parts of 4 rows of 16
        // elements, and each gets one column
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
        const int s = 8 * g + (i >> 2), at = base + s * B * 2 + (block ^ block_swizzle<T, B>(s)) * 32 + (i & 3) * 8;
        s16x4 h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(stage + (at + (32 * step + 4 * j) * B * 2)));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return f;
}

// ------------------------------------------------------------------ epilogue

// V consecutive results.  Those of 16 bytes pass the caches by, which the next
// workgroups need for operands.
template <typename T, int V> __device__ __forceinline__ void store_whole(T* p, const float (&v)[V]) {
    if constexpr (sizeof(T) * V == 16)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, Vec<T, V>::pack(v)), reinterpret_cast<u32x4_unaligned*>(p));
    else Vec<T, V>::store(p, v);
}
// `left` of them, at most V.
template <typename T, int V> __device__ __forceinline__ void store_values(T* p, int left, const float (&v)[V]) {
    if (left >= V) {
        store_whole<T, V>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < left) store_f32<T>(p, e, v[e]);
    }
}

// The biases of columns c ..: 0 where there is none.
template <int V> __device__ __forceinline__ void load_bias(const Product& p, int c, float (&v)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = p.bias && c + e < p.cols ? p.bias[c + e] : 0.0f;
}

// V consecutive results of row r from column c on: from the sums (biases added) to z and y.
template <typename T, int V>
__device__ __forceinline__ void finish(const Product& p, long long r, int c, float (&v)[V]) {
    const int left = p.cols - c;
    if (p.z) store_values<T, V>(static_cast<T*>(p.z) + r * p.ldz + c, left, v);
    activate<V>(v, p.act);
    if (p.residual) {
        const T* const at = static_cast<const T*>(p.residual) + r * p.ldr + c;
        if (left >= V) {
            float u[V];
            Vec<T, V>::unpack(Vec<T, V>::load(at), u);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += u[e];
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < left) v[e] += load_f32<T>(at, e);
        }
    }
    store_values<T, V>(static_cast<T*>(p.y) + r * p.ldy + c, left, v);
}

// A wave's results, TI*16 columns x TJ*16 rows from (m0, n0): block by block of
// 16 rows through the wave's own two pieces of LDS (16 x TI*16 fp32 each, the next
// block is written before one is read), so that whole rows leave, 16 bytes of the
// output type a lane.  In the 16x16 result lane l holds, in register r, column
// 4 (l >> 4) + r of row l & 15.  kSums: the sums themselves, of a part of s, to `sums`;
// kPlain: no bias, activation, residual and z (the gradients).
//
// A wave whose results all exist, all but those at the matrix's edges, needs no
// conditions, and issues the residual's loads together, ahead of the first block (as
// many as 48 registers hold).
enum Output { kEpilogue, kPlain, kSums };

template <typename T, int TI, int TJ, Output MODE>
__device__ __forceinline__ void write_results(const Product& p, f32x4 (&acc)[TI][TJ], char* lds, int m0, int n0, float* sums) {
    using OUT = std::conditional_t<MODE == kSums, float, T>;
    constexpr int V = kPiece<OUT>, PIECES = TI * 16 / V, ROW = TI * 64, MASK = (TI * 4 < 16 ? TI * 4 : 16) - 1;
    constexpr int ITS = 16 * PIECES / 64, STEP = 64 / PIECES;   // rows between a lane's in a block
    static_assert(64 % PIECES == 0, "a lane's columns stay");
    const int lane = threadIdx.x & 63, r0 = lane / PIECES, q0 = lane % PIECES * (V / 4);
    const int c = n0 + lane % PIECES * V;
    float bias[V] = {};
    if constexpr (MODE == kEpilogue) load_bias<V>(p, c, bias);
    auto put = [&](int j) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
            *reinterpret_cast<f32x4*>(lds + ((j & 1) * 16 + (lane & 15)) * ROW + ((i * 4 + (lane >> 4)) ^ (lane & 15 & MASK)) * 16) = acc[i][j];
    };
    auto get = [&](int j, int it, float (&v)[V]) __attribute__((always_inline)) {
        const int r = r0 + it * STEP;
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const f32x4 u = *reinterpret_cast<const f32x4*>(lds + ((j & 1) * 16 + r) * ROW + ((q0 + h) ^ (r & MASK)) * 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * h + k] = MODE == kEpilogue ? u[k] + bias[4 * h + k] : u[k];
        }
    };
    if (m0 + TJ * 16 <= p.rows && n0 + TI * 16 <= p.cols) {
        const long long row = m0 + r0;
        OUT* const y = MODE == kSums ? reinterpret_cast<OUT*>(sums) + row * p.cols + c : static_cast<OUT*>(p.y) + row * p.ldy + c;
        const long long ldy = MODE == kSums ? p.cols : p.ldy;
        constexpr int AHEAD = TJ * ITS <= 12 ? TJ : 12 / ITS;
        typename Vec<T, V>::raw residual[AHEAD][ITS] = {};
        const T* const pr = static_cast<const T*>(p.residual) + (p.residual ? row * p.ldr + c : 0);
        auto fetch = [&](int j) __attribute__((always_inline)) {
            if (MODE != kEpilogue || !p.residual) return;
#pragma unroll
            for (int it = 0; it < ITS; ++it) residual[j % AHEAD][it] = Vec<T, V>::load(pr + (j * 16 + it * STEP) * p.ldr);
        };
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) fetch(j);
        put(0);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            if (j + 1 < TJ) put(j + 1);
            wave_lds_fence();
            float v[ITS][V];
#pragma unroll
            for (int it = 0; it < ITS; ++it) get(j, it, v[it]);
            if constexpr (MODE == kEpilogue) {
                if (p.z) {
#pragma unroll
                    for (int it = 0; it < ITS; ++it)
                        store_whole<T, V>(static_cast<T*>(p.z) + (row + j * 16 + it * STEP) * p.ldz + c, v[it]);
                }
                activate<ITS * V>(reinterpret_cast<float(&)[ITS * V]>(v), p.act);
            }
#pragma unroll
            for (int it = 0; it < ITS; ++it) {
                if constexpr (MODE == kEpilogue) {
                    float u[V];
                    Vec<T, V>::unpack(residual[j % AHEAD][it], u);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[it][e] += u[e];
                }
                store_whole<OUT, V>(y + (j * 16 + it * STEP) * ldy, v[it]);
            }
            if (j + AHEAD < TJ) fetch(j + AHEAD);
            wave_lds_fence();
        }
        return;
    }
    put(0);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        if (j + 1 < TJ) put(j + 1);
        wave_lds_fence();
#pragma unroll 1
        for (int it = 0; it < ITS; ++it) {
            const int m = m0 + j * 16 + r0 + it * STEP;
            float v[V];
            get(j, it, v);
            if (m >= p.rows || c >= p.cols) continue;
            if constexpr (MODE == kSums) store_values<float, V>(sums + (long long)m * p.cols + c, p.cols - c, v);
            else if constexpr (MODE == kPlain) store_values<T, V>(static_cast<T*>(p.y) + m * p.ldy + c, p.cols - c, v);
            else finish<T, V>(p, m, c, v);
        }
        wave_lds_fence();
    }
}

// ------------------------------------------------------------------ operands of any alignment

// A thread's pieces of an operand's stage: in registers, then in LDS.
template <typename T, int B, int NT, bool STRIDED> struct Staged {
    static constexpr int N = B * 8 / NT, E = kPiece<T>, S = kStageK / (int)sizeof(T);
    static_assert(N * NT == B * 8, "pieces split evenly");
    uint4 v[N];
    // indexes i0 .. of `count`, s from s0 to `send`, rows of `row` elements.  A stage whose pieces are all whole
    // is read without conditions, contiguous rows past the last being the last again
    // (their results are not written).
    __device__ __forceinline__ void load(const T* p, long long ld, int i0, int count, int s0, int send, int row) {
        const bool whole = s0 + S <= send && (!STRIDED || i0 + B <= count);
        if (whole) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int e = n * NT + threadIdx.x;
                const int i = STRIDED ? i0 + e % (B / E) * E : min(i0 + e / 8, count - 1), s = s0 + (STRIDED ? e / (B / E) : e % 8 * E);
                v[n] = load_bytes<16>(p + (STRIDED ? s * ld + i : i * ld + s));
            }
            return;
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int e = n * NT + threadIdx.x;
            const int i = i0 + (STRIDED ? e % (B / E) * E : e / 8), s = s0 + (STRIDED ? e / (B / E) : e % 8 * E);
            const bool in = i < count && s < send;
            v[n] = in ? load_piece<T>(p + (STRIDED ? s * ld + i : i * ld + s), STRIDED ? count - i : send - s, row) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void store(char* stage) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int e = n * NT + threadIdx.x;
            const int at = STRIDED ? strided_byte<T, B>(e / (B / E), e % (B / E) * E) : slot_of(e / 8, e % 8) * 16;
            *reinterpret_cast<uint4*>(stage + at) = v[n];
        }
    }
};

// Operands of any alignment pass through registers: the loads of a stage are in
// flight during the products of the one before.
template <typename T, int BM, int BN, int WM, int WN, bool TA, bool TB, Output MODE>
__global__ __launch_bounds__(WM * WN * 64) void matmul_staged_kernel(Product p, int tm, int tn, int stages, float* sums) {
    constexpr int NT = WM * WN * 64, TI = BN / WN / 16, TJ = BM / WM / 16, S = kStageK / (int)sizeof(T);
    constexpr int STAGE = (BM + BN) * kStageK, OUTB = WM * WN * 32 * TI * 64;
    __shared__ uint4 lds[(STAGE > OUTB ? STAGE : OUTB) / 16];
    char* const sa = reinterpret_cast<char*>(lds);
    const int wave = threadIdx.x >> 6, wm = wave / WN, wn = wave % WN;
    const TileAt t = tile_at(tm, tn, BM, BN);
    const int s0 = t.split * stages * S, send = min(p.K, s0 + stages * S);
    f32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Staged<T, BN, NT, TA> a;
    Staged<T, BM, NT, TB> b;
    auto load = [&](int s) __attribute__((always_inline)) {
        a.load(static_cast<const T*>(p.a), p.lda, t.n0, p.cols, s, send, TA ? p.cols : p.K);
        b.load(static_cast<const T*>(p.b), p.ldb, t.m0, p.rows, s, send, TB ? p.rows : p.K);
    };
    load(s0);
    for (int s = s0; s < send; s += S) {
        __syncthreads();
        a.store(sa);
        b.store(sa + BN * kStageK);
        __syncthreads();
        if (s + S < send) load(s + S);
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            Frag<T> fa[TI], fb[TJ];
#pragma unroll
            for (int i = 0; i < TI; ++i) fa[i] = fragment<T, BN, TA>(sa, 0, wn * TI + i, step);
#pragma unroll
            for (int j = 0; j < TJ; ++j) fb[j] = fragment<T, BM, TB>(sa, BN * kStageK, wm * TJ + j, step);
            products<T, TI, TJ>(acc, fa, fb);
        }
    }
    __syncthreads();
    write_results<T, TI, TJ, MODE>(p, acc, sa + wave * (32 * TI * 64), t.m0 + wm * TJ * 16, t.n0 + wn * TI * 16,
                                   sums + (long long)t.split * p.rows * p.cols);
}

// ------------------------------------------------------------------ aligned operands

// A wave's copies of an operand's stage into LDS, 1 KB each, straight from
// memory: a lane's slot in LDS is fixed (16 bytes times its number), so it fetches
// what belongs there.
template <typename T, int B, int NW, bool STRIDED> struct Copies {
    static constexpr int N = B / 8 / NW, ES = (int)sizeof(T), S = kStageK / ES;
    static_assert(N * NW * 8 == B, "copies split evenly");
    const char* base;
    long long step;          // bytes of a stage
    int off[N];              // of this lane's pieces, within the stage
    uint32_t row, tail;      // strided: bytes of a row, and of the tile's part of one
    __amdgpu_buffer_rsrc_t r;
    int piece;               // contiguous: this lane's first s
    // indexes i0 .. of `count`, from s0 on
    __device__ __forceinline__ void init(const void* p, long long ld, int i0, int count, int K, int s0, int wave, int lane) {
        const int n = min(count - i0, B);
        if constexpr (STRIDED) {
            base = static_cast<const char*>(p) + ((long long)s0 * ld + i0) * ES;
            step = (long long)S * ld * ES;
            row = (uint32_t)(ld * ES);
            tail = ((uint32_t)n * ES + 15) & ~15u;   // whole pieces: an aligned one that holds an element is read whole
#pragma unroll
            for (int c = 0; c < N; ++c) {
                const int at = (c * NW + wave) * 1024 + lane * 16, s = at / (B * ES), in = at % (B * ES);
                const int block = (in / (16 * ES)) ^ block_swizzle<T, B>(s);
                off[c] = s * (int)row + block * (16 * ES) + in % (16 * ES);
            }
        } else {
            // row (c * NW + wave) * 8 + lane / 8: its bits 1 to 3 are those of wave * 8 + lane / 8 for even NW
            static_assert(NW % 2 == 0, "a wave's copies share their rows' bit 3");
            const int lr = lane >> 3;
            piece = ((lane & 7) ^ (((wave * 8 + lr) >> 1) & 7)) * (16 / ES) + s0;
            r = make_rsrc(static_cast<const char*>(p) + (long long)i0 * ld * ES,
                          (uint32_t)((long long)(n - 1) * ld * ES + ((long long)K * ES + 15 & ~15LL)));
#pragma unroll
            for (int c = 0; c < N; ++c) off[c] = (int)(((c * NW + wave) * 8 + lr) * ld + piece) * ES;
        }
    }
    // stage `n` from the first, of s below send; past it zeros are written
    __device__ __forceinline__ void copy(char* stage, int n, int s0, int send, int wave) const {
        if constexpr (STRIDED) {
            // bytes of the rows that are left, with no branch between the products
            const int left = min(send - s0 - n * S, S);
            const auto rs = make_rsrc(base + n * step, ((uint32_t)(left - 1) * row + tail) & (uint32_t)~((left - 1) >> 31));
#pragma unroll
            for (int c = 0; c < N; ++c) copy_kb(rs, stage + (c * NW + wave) * 1024, off[c]);
        } else {
            const bool in = piece + n * S < send;
#pragma unroll
            for (int c = 0; c < N; ++c) copy_kb(r, stage + (c * NW + wave) * 1024, in ? off[c] + n * kStageK : kOOB);
        }
    }
};

// Stage n + 2 is copied into the buffer that stage n has just been read from, a
// whole stage ahead of its use; the reads of a step are issued one step before its
// products, across the stages' border too, so there is one barrier per stage.
template <typename T, int BM, int BN, int WM, int WN, bool TA, bool TB, Output MODE>
__global__ __launch_bounds__(WM * WN * 64) void matmul_tile_kernel(Product p, int tm, int tn, int stages, float* sums) {
    constexpr int NW = WM * WN, TI = BN / WN / 16, TJ = BM / WM / 16, S = kStageK / (int)sizeof(T);
    constexpr int STAGE = (BM + BN) * kStageK;
    static_assert(NW * 32 * TI * 64 <= STAGE, "results fit a stage");
    __shared__ uint4 lds0[STAGE / 16], lds1[STAGE / 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const TileAt t = tile_at(tm, tn, BM, BN);
    const int s0 = t.split * stages * S, send = min(p.K, s0 + stages * S), count = (send - s0 + S - 1) / S;
    Copies<T, BN, NW, TA> ca;
    Copies<T, BM, NW, TB> cb;
    ca.init(p.a, p.lda, t.n0, p.cols, p.K, s0, wave, lane);
    cb.init(p.b, p.ldb, t.m0, p.rows, p.K, s0, wave, lane);
    f32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Frag<T> fa[2][TI], fb[2][TJ];
    // every buffer a restrict argument of one function: the compiler then does not
    // make the reads of one wait for the copies into the other
    auto loop = [&](char* __restrict__ b0, char* __restrict__ b1) __attribute__((always_inline)) {
        auto copy = [&](char* stage, int n) __attribute__((always_inline)) {
            ca.copy(stage, n, s0, send, wave);
            cb.copy(stage + BN * kStageK, n, s0, send, wave);
        };
        auto read = [&](const char* stage, int step, int set) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < TI; ++i) fa[set][i] = fragment<T, BN, TA>(stage, 0, wn * TI + i, step);
#pragma unroll
            for (int j = 0; j < TJ; ++j) fb[set][j] = fragment<T, BM, TB>(stage, BN * kStageK, wm * TJ + j, step);
        };
        // the products of a set, with the reads (and copies) issued before them in the
        // source spread between them: the compiler would otherwise sink the reads below
        // the products to save registers, and the next step would wait for them
        constexpr int READS = (TA ? (sizeof(T) == 4 ? 4 : 2) : 1) * TI + (TB ? (sizeof(T) == 4 ? 4 : 2) : 1) * TJ;
        constexpr int MATH = TI * TJ * (sizeof(T) == 4 ? 4 : 1), PER = MATH / READS > 0 ? MATH / READS : 1;
        auto multiply_set = [&](int set, bool copies) __attribute__((always_inline)) {
            products<T, TI, TJ>(acc, fa[set], fb[set]);
#pragma unroll
            for (int i = 0; i < READS; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (copies) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // From the second step of stage n, whose operands have been read, to the second
        // step of the next.  At the barrier this wave's reads of `cur` are complete and its
        // copies of the next stage have landed.  (The loop turns here, where no copy is in
        // flight: after the turn the compiler cannot tell the buffers of copies and
        // transposing reads apart.)
        auto stage = [&](char* cur, char* next, int n) __attribute__((always_inline)) {
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            read(next, 0, 0);
            copy(cur, n + 2);
            multiply_set(1, true);
            read(next, 1, 1);
            multiply_set(0, false);
        };
        ca.copy(b0, 0, s0, send, wave);
        ca.copy(b1, 1, s0, send, wave);
        cb.copy(b0 + BN * kStageK, 0, s0, send, wave);
        cb.copy(b1 + BN * kStageK, 1, s0, send, wave);
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        read(b0, 0, 0);
        read(b0, 1, 1);
        multiply_set(0, false);
        for (int n = 0; n + 1 < count; n += 2) {
            stage(b0, b1, n);
            if (n + 2 < count) stage(b1, b0, n + 1);
        }
        multiply_set(1, false);
    };
    loop(reinterpret_cast<char*>(lds0), reinterpret_cast<char*>(lds1));
    __builtin_amdgcn_s_waitcnt(0x0070);   // no copy is in flight when the buffers take the results
    __syncthreads();
    write_results<T, TI, TJ, MODE>(p, acc, reinterpret_cast<char*>(lds0) + wave * (32 * TI * 64), t.m0 + wm * TJ * 16,
                                   t.n0 + wn * TI * 16, sums + (long long)t.split * p.rows * p.cols);
}

// Adds the parts of a product that was split along s and finishes.  `groups` (a power
// of two up to 32) threads share a piece of 16 bytes of results, each adds every
// groups-th part, and the first adds theirs: a fixed order, and enough loads in
// flight where the results are few.
template <typename T>
__global__ __launch_bounds__(256) void matmul_join_kernel(Product p, const float* sums, int splits, int groups) {
    constexpr int V = kPiece<T>;
    __shared__ float part[256][V + 1];
    const int per = 256 / groups, group = threadIdx.x / per;
    const int pieces = (p.cols + V - 1) / V;
    const long long i = (long long)blockIdx.x * per + threadIdx.x % per, total = (long long)p.rows * p.cols;
    const long long r = i / pieces;
    const int c = (int)(i - r * pieces) * V;
    const bool in = r < p.rows;
    float v[V] = {};
    if (in) {
        const float* at = sums + group * total + r * p.cols + c;
        const long long step = groups * total;
        if (c + V <= p.cols) {
#pragma unroll 4
            for (int k = group; k < splits; k += groups, at += step) {
#pragma unroll
                for (int h = 0; h < V; h += 4) {
                    float u[4];
                    Vec<float, 4>::unpack(Vec<float, 4>::load(at + h), u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[h + e] += u[e];
                }
            }
        } else {
            for (int k = group; k < splits; k += groups, at += step)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (c + e < p.cols) v[e] += at[e];
        }
    }
    if (groups > 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) part[threadIdx.x][e] = v[e];
        __syncthreads();
        if (group) return;
        for (int g = 1; g < groups; ++g)
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += part[g * per + threadIdx.x][e];
    }
    if (!in) return;
    float bias[V];
    load_bias<V>(p, c, bias);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += bias[e];
    finish<T, V>(p, r, c, v);
}

// ------------------------------------------------------------------ few rows

// Up to 32 rows of the forward product, which reading the weights bounds: they stream
// from memory straight into the matrix unit's registers.  One workgroup: NG * 16
// columns, MT * 16 rows, all of s; its waves split s, 128 bytes of a row at a time (so
// that a step reads whole lines), and join in LDS.  Columns are the rows of the 16x16
// result, so a lane ends with 4 consecutive ones of one row.  The loads of U steps
// stand before their products.
template <typename T, int MT, int NG, int U, bool ALIGNED>
__global__ __launch_bounds__(1024) void matmul_skinny_kernel(Product p) {
    extern __shared__ f32x4 joined[];   // [wave][NG][MT][64]
    constexpr int ES = (int)sizeof(T), E = kPiece<T>, S = kStageK / ES;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * (NG * 16), row = lane & 15, c = lane >> 4;
    const T* const pa = static_cast<const T*>(p.a) + (long long)n0 * p.lda;
    const T* const pb = static_cast<const T*>(p.b);
    const auto ra = make_rsrc(pa, (uint32_t)(((min(p.cols - n0, NG * 16) - 1) * p.lda + p.K) * ES));
    const auto rb = make_rsrc(pb, (uint32_t)(((p.rows - 1) * p.ldb + p.K) * ES));
    f32x4 acc[NG][MT];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[g][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // 16 bytes of row r of an operand, 0 past its last row and past K.  Unaligned ones
    // that all end inside their rows (`whole`, the wave's) are plain loads, the rows past
    // the last its own again (their results are not written).
    auto fetch = [&](const T* base, __amdgpu_buffer_rsrc_t rs, long long ld, int r, int left, int s, bool whole) __attribute__((always_inline)) {
        Frag<T> f;
        if constexpr (ALIGNED) f.v = __builtin_bit_cast(decltype(f.v), load16(rs, r < left && s < p.K ? (int)(r * ld + s) * ES : kOOB));
        else if (whole) f.v = __builtin_bit_cast(decltype(f.v), load_bytes<16>(base + min(r, left - 1) * ld + s));
        else f.v = __builtin_bit_cast(decltype(f.v), r < left && s < p.K ? load_piece<T>(base + r * ld + s, p.K - s, p.K) : make_uint4(0, 0, 0, 0));
        return f;
    };
    const int stride = waves * S;
    for (int s0 = wave * S; s0 < p.K; s0 += stride * U) {
        Frag<T> a[U][2][NG], b[U][2][MT];
        auto fetch_all = [&](bool whole) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int s = s0 + u * stride + h * (S / 2) + c * E;
#pragma unroll
                    for (int g = 0; g < NG; ++g) a[u][h][g] = fetch(pa, ra, p.lda, g * 16 + row, p.cols - n0, s, whole);
#pragma unroll
                    for (int t = 0; t < MT; ++t) b[u][h][t] = fetch(pb, rb, p.ldb, t * 16 + row, p.rows, s, whole);
                }
        };
        if (!ALIGNED && s0 + (U - 1) * stride + S <= p.K) fetch_all(true);
        else fetch_all(false);
        __builtin_amdgcn_sched_barrier(0);   // or the compiler sinks loads below products, to save registers
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int t = 0; t < MT; ++t) multiply(acc[g][t], a[u][h][g], b[u][h][t]);
    }
    constexpr int COUNT = NG * MT * 64;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t) joined[wave * COUNT + (g * MT + t) * 64 + lane] = acc[g][t];
    __syncthreads();
    for (int e = threadIdx.x; e < COUNT; e += blockDim.x) {
        f32x4 sum = joined[e];
        for (int k = 1; k < waves; ++k) sum += joined[k * COUNT + e];
        const int tile = e >> 6, m = tile % MT * 16 + (e & 15), n = n0 + tile / MT * 16 + ((e & 63) >> 4) * 4;
        if (m >= p.rows || n >= p.cols) continue;
        float v[4], bias[4];
        load_bias<4>(p, n, bias);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = sum[k] + bias[k];
        finish<T, 4>(p, m, n, v);
    }
}

// ------------------------------------------------------------------ whole pieces

// Copies of two matrices [rows][K] whose rows are whole 16-byte pieces, zeros past K.
template <typename T> struct Packed {
    const T* from;
    T* to;
    long long ld, rows;
};

template <typename T>
__global__ __launch_bounds__(256) void matmul_pack_kernel(Packed<T> a, Packed<T> b, int K) {
    constexpr int E = kPiece<T>;
    const int pieces = (K + E - 1) / E;
    const long long na = a.rows * pieces, all = na + b.rows * pieces, step = (long long)gridDim.x * 256;
#pragma unroll 2
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
        const bool first = i < na;
        const long long k = first ? i : i - na, r = k / pieces;
        const int c = (int)(k - r * pieces) * E;
        const T* const from = first ? a.from + r * a.ld + c : b.from + r * b.ld + c;
        *reinterpret_cast<uint4*>((first ? a.to : b.to) + k * E) = load_piece<T>(from, K - c, K);
    }
}

// ------------------------------------------------------------------ dz

// dz = dy act'(z) (null: not wanted), rows padded with zeros to ldd elements, and the
// sums of its columns over a workgroup's rows, [row chunk][N] (null: not wanted): a
// thread's in fp32, the workgroup's over its threads in fp64.  256 threads: `lanes`
// vectors of a row, 256 / lanes rows at a time.
//
// The sums are of the unrounded values; dz itself is rounded to T, as the matrix unit
// takes bf16.  After SiLU or GELU that is half a step at most of every term of dx and dw,
// whose error against fp64 grows from their own rounding's 0.0017 to 0.0023 (rms, 8192 x
// 4096 -> 4096); a second bf16 part of dz would keep it, at twice the products' time.
template <typename T, bool ACT>
__global__ __launch_bounds__(256) void matmul_dz_kernel(MatmulBwdArgs a, T* dz, int ldd, float* sums, int lanes, int chunk) {
    constexpr int V = kPiece<T>;
    __shared__ float part[256][V + 1];
    const int l = threadIdx.x % lanes, group = threadIdx.x / lanes, groups = 256 / lanes;
    const int c = (blockIdx.x * lanes + l) * V;
    const long long m0 = (long long)blockIdx.y * chunk, m1 = m0 + chunk < a.M ? m0 + chunk : a.M;
    float s[V] = {};
    auto row = [&](long long m, float (&v)[V], float (&z)[V]) __attribute__((always_inline)) {
        if constexpr (ACT) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = c + e < a.N ? v[e] * activation_slope(z[e], a.act) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += v[e];
        if (dz) Vec<T, V>::store(dz + m * ldd + c, v);
    };
    const T* const py = static_cast<const T*>(a.dy) + c;
    const T* const pz = static_cast<const T*>(a.z) + (ACT ? c : 0);
    typedef typename Vec<T, V>::raw raw;
    if (c + V <= a.N) {
#pragma unroll 4
        for (long long m = m0 + group; m < m1; m += groups) {
            float v[V], z[V];
            Vec<T, V>::unpack(Vec<T, V>::load(py + m * a.lddy), v);
            if constexpr (ACT) Vec<T, V>::unpack(Vec<T, V>::load(pz + m * a.ldz), z);
            row(m, v, z);
        }
    } else if (c < a.N) {
#pragma unroll 2
        for (long long m = m0 + group; m < m1; m += groups) {
            float v[V], z[V];
            Vec<T, V>::unpack(__builtin_bit_cast(raw, load_piece<T>(py + m * a.lddy, a.N - c, a.N)), v);
            if constexpr (ACT) Vec<T, V>::unpack(__builtin_bit_cast(raw, load_piece<T>(pz + m * a.ldz, a.N - c, a.N)), z);
            row(m, v, z);
        }
    }
    if (!sums) return;
#pragma unroll
    for (int e = 0; e < V; ++e) part[threadIdx.x][e] = s[e];
    __syncthreads();
    for (int i = threadIdx.x; i < lanes * V; i += 256) {
        const int n = blockIdx.x * lanes * V + i;
        double t = 0.0;
        for (int g = 0; g < groups; ++g) t += part[g * lanes + i / V][i % V];
        if (n < a.N) sums[(long long)blockIdx.y * a.N + n] = (float)t;
    }
}

// ------------------------------------------------------------------ host

static_assert(kStageBytes == kStageK, "plans count the tiles' stages");

template <typename T> hipError_t pack(const Packed<T>& a, const Packed<T>& b, int K, hipStream_t st) {
    const long long pieces = (a.rows + b.rows) * (whole_pieces(K, (int)sizeof(T)) / kPiece<T>), blocks = (pieces + 255) / 256;
    matmul_pack_kernel<T><<<(unsigned)(blocks < 8 * kUnits ? blocks : 8 * kUnits), 256, 0, st>>>(a, b, K);
    return hipGetLastError();
}

// Whole 16-byte pieces at aligned addresses; along s too where it is contiguous
// (`padded`: with zeros, up to a whole piece).
bool aligned_operand(const void* p, long long ld, int K, int es, bool strided, bool padded) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && (strided || padded || (long long)K * es % 16 == 0);
}

template <typename T, bool TA, bool TB, Output MODE>
hipError_t tiled(const Product& p, const Plan& q, bool aligned, float* sums, hipStream_t st) {
    const unsigned blocks = (unsigned)(q.tm * q.tn * q.splits);
    if constexpr (MODE != kSums)   // tiles of 256 are enough for the chip and never split
        if (q.b == 256) {
            matmul_tile_kernel<T, 256, 256, 2, 4, TA, TB, MODE><<<blocks, 512, 0, st>>>(p, q.tm, q.tn, q.stages, sums);
            return hipGetLastError();
        }
    if (q.b == 128 && aligned)
        matmul_tile_kernel<T, 128, 128, 2, 2, TA, TB, MODE><<<blocks, 256, 0, st>>>(p, q.tm, q.tn, q.stages, sums);
    else if (q.b == 128)
        matmul_staged_kernel<T, 128, 128, 2, 2, TA, TB, MODE><<<blocks, 256, 0, st>>>(p, q.tm, q.tn, q.stages, sums);
    else if (aligned)
        matmul_tile_kernel<T, 64, 64, 2, 2, TA, TB, MODE><<<blocks, 256, 0, st>>>(p, q.tm, q.tn, q.stages, sums);
    else
        matmul_staged_kernel<T, 64, 64, 2, 2, TA, TB, MODE><<<blocks, 256, 0, st>>>(p, q.tm, q.tn, q.stages, sums);
    return hipGetLastError();
}

// `padded`: contiguous rows end in zeros, up to a whole piece.
template <typename T, bool TA, bool TB> hipError_t product(const Product& p, bool padded, void* ws, hipStream_t st) {
    constexpr int ES = (int)sizeof(T);
    const bool aligned = aligned_operand(p.a, p.lda, p.K, ES, TA, padded) && aligned_operand(p.b, p.ldb, p.K, ES, TB, padded);
    const Plan q = make_plan(p.rows, p.cols, p.K, ES, aligned);
    float* const sums = static_cast<float*>(ws);
    if (q.splits == 1) return tiled<T, TA, TB, TA ? kPlain : kEpilogue>(p, q, aligned, nullptr, st);
    const hipError_t e = tiled<T, TA, TB, kSums>(p, q, aligned, sums, st);
    if (e != hipSuccess) return e;
    const long long pieces = (long long)p.rows * ((p.cols + kPiece<T> - 1) / kPiece<T>);
    int groups = 1;
    while (groups < 32 && groups * 4 <= q.splits) groups *= 2;
    matmul_join_kernel<T><<<(unsigned)((pieces * groups + 255) / 256), 256, 0, st>>>(p, sums, q.splits, groups);
    return hipGetLastError();
}

template <typename T, int MT, int NG, int U> hipError_t skinny_instance(const Product& p, bool aligned, int waves, hipStream_t st) {
    const unsigned blocks = (unsigned)(((long long)p.cols + NG * 16 - 1) / (NG * 16));
    const int lds = waves * NG * MT * 1024;
    if (aligned) matmul_skinny_kernel<T, MT, NG, U, true><<<blocks, waves * 64, lds, st>>>(p);
    else matmul_skinny_kernel<T, MT, NG, U, false><<<blocks, waves * 64, lds, st>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t skinny(const Product& p, const SkinnyShape& k, hipStream_t st) {
    constexpr int ES = (int)sizeof(T);
    const bool aligned = aligned_operand(p.a, p.lda, p.K, ES, false, false) && aligned_operand(p.b, p.ldb, p.K, ES, false, false);
    if (k.two) return k.pairs ? skinny_instance<T, 2, 2, 2>(p, aligned, k.waves, st) : skinny_instance<T, 2, 1, 2>(p, aligned, k.waves, st);
    return k.steps > 2 ? skinny_instance<T, 1, 1, 4>(p, aligned, k.waves, st) : skinny_instance<T, 1, 1, 2>(p, aligned, k.waves, st);
}

template <typename T> size_t forward_workspace(int M, int K, int N) {
    constexpr int ES = (int)sizeof(T);
    if (skinny_shape(M, N, K, ES).fits) return 0;
    const size_t parts = split_bytes(M, N, K, ES);
    return packs_forward(M, K, N, ES) ? round256(parts) + ((size_t)M + N) * whole_pieces(K, ES) * ES : parts;
}

template <typename T> hipError_t forward(Product p, char* ws, hipStream_t st) {
    constexpr int ES = (int)sizeof(T);
    const SkinnyShape k = skinny_shape(p.rows, p.cols, p.K, ES);
    if (k.fits) return skinny<T>(p, k, st);
    if (!packs_forward(p.rows, p.K, p.cols, ES)) return product<T, false, false>(p, false, ws, st);
    const int ld = whole_pieces(p.K, ES);
    T* const a = reinterpret_cast<T*>(ws + round256(split_bytes(p.rows, p.cols, p.K, ES)));
    T* const b = a + (size_t)p.cols * ld;
    const hipError_t e = pack<T>({static_cast<const T*>(p.a), a, p.lda, p.cols}, {static_cast<const T*>(p.b), b, p.ldb, p.rows}, p.K, st);
    if (e != hipSuccess) return e;
    p.a = a;
    p.b = b;
    p.lda = p.ldb = ld;
    return product<T, false, false>(p, true, ws, st);
}

// ---- the backward pass's workspace: dz, the parts of dbias, the parts of dx or dw, and
// x and w in whole pieces

struct BwdSpace {
    size_t dz, sums, parts, x, w;   // offsets; the end
    size_t end;
};

template <typename T> BwdSpace bwd_space(int M, int K, int N) {
    constexpr int ES = (int)sizeof(T);
    const DzShape d = dz_shape(M, N, ES);
    BwdSpace b;
    b.dz = 0;
    b.sums = round256((size_t)M * whole_pieces(N, ES) * ES);
    b.parts = b.sums + round256((size_t)d.chunks * N * 4);
    const size_t u = split_bytes(M, K, N, ES), v = split_bytes(N, K, M, ES);
    const size_t row = packs(M, K, N, ES) ? (size_t)whole_pieces(K, ES) * ES : 0;
    b.x = b.parts + round256(u > v ? u : v);
    b.w = b.x + round256(M * row);
    b.end = b.w + N * row;
    return b;
}

template <typename T> hipError_t gradients(const MatmulBwdArgs& a, char* ws, hipStream_t st) {
    constexpr int ES = (int)sizeof(T);
    const BwdSpace b = bwd_space<T>(a.M, a.K, a.N);
    const DzShape d = dz_shape(a.M, a.N, ES);
    const int ldd = whole_pieces(a.N, ES), ldk = whole_pieces(a.K, ES);
    const bool products = a.dx || a.dw;
    // without an activation dz is dy, read where it lies if it has whole pieces
    const bool copy = a.z || (!aligned_operand(a.dy, a.lddy, a.N, ES, false, false) && worth_copies(a.M, a.K, a.N, ES));
    T* const dz = copy && products ? reinterpret_cast<T*>(ws + b.dz) : nullptr;
    float* const sums = a.dbias ? reinterpret_cast<float*>(ws + b.sums) : nullptr;
    hipError_t e = hipSuccess;
    if (dz || sums) {
        const dim3 grid(d.cols, d.chunks);
        if (a.z) matmul_dz_kernel<T, true><<<grid, 256, 0, st>>>(a, dz, ldd, sums, d.lanes, d.chunk);
        else matmul_dz_kernel<T, false><<<grid, 256, 0, st>>>(a, dz, ldd, sums, d.lanes, d.chunk);
        e = hipGetLastError();
        if (e == hipSuccess && sums) e = launch_join_columns(sums, a.dbias, d.chunks, a.N, st);
        if (e != hipSuccess) return e;
    }
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    long long ldx = a.ldx, ldw = a.ldw;
    if (products && packs(a.M, a.K, a.N, ES)) {
        T* const px = reinterpret_cast<T*>(ws + b.x);
        T* const pw = reinterpret_cast<T*>(ws + b.w);
        e = pack<T>({x, px, ldx, a.dw ? a.M : 0}, {w, pw, ldw, a.dx ? a.N : 0}, a.K, st);
        if (e != hipSuccess) return e;
        x = px;
        w = pw;
        ldx = ldw = ldk;
    }
    Product p = {};
    p.b = dz ? dz : a.dy;
    p.ldb = dz ? ldd : a.lddy;
    if (a.dx) {
        p.a = w; p.lda = ldw; p.rows = a.M; p.cols = a.K; p.K = a.N; p.y = a.dx; p.ldy = a.lddx;
        e = product<T, true, false>(p, dz, ws + b.parts, st);
        if (e != hipSuccess) return e;
    }
    if (a.dw) {
        p.a = x; p.lda = ldx; p.rows = a.N; p.cols = a.K; p.K = a.M; p.y = a.dw; p.ldy = a.lddw;
        e = product<T, true, true>(p, dz, ws + b.parts, st);
    }
    return e;
}

}  // namespace

// A launch counts its threads in 32 bits: 2^24 tiles of 64 x 64 at 256 threads.
bool matmul_supports(int M, int K, int N) {
    auto tiles = [](int v) { return ((long long)v + 63) / 64; };
    constexpr long long most = 1 << 24;
    return tiles(M) * tiles(N) < most && tiles(M) * tiles(K) < most && tiles(N) * tiles(K) < most;
}

size_t matmul_workspace(int M, int K, int N, int dtype) {
    return dtype == 0 /* CONV2D_F32 */ ? forward_workspace<float>(M, K, N) : forward_workspace<bf16_t>(M, K, N);
}

size_t matmul_bwd_workspace(int M, int K, int N, int dtype) {
    return dtype == 0 ? bwd_space<float>(M, K, N).end : bwd_space<bf16_t>(M, K, N).end;
}

hipError_t launch_matmul(const MatmulArgs& a, void* ws, hipStream_t st) {
    Product p = {};
    p.a = a.w; p.b = a.x; p.lda = a.ldw; p.ldb = a.ldx; p.rows = a.M; p.cols = a.N; p.K = a.K;
    p.bias = a.bias; p.residual = a.residual; p.z = a.z; p.y = a.y; p.ldr = a.ldr; p.ldz = a.ldz; p.ldy = a.ldy; p.act = a.act;
    char* const space = static_cast<char*>(ws);
    return a.dtype == 0 /* CONV2D_F32 */ ? forward<float>(p, space, st) : forward<bf16_t>(p, space, st);
}

hipError_t launch_matmul_bwd(const MatmulBwdArgs& a, void* ws, hipStream_t st) {
    return a.dtype == 0 /* CONV2D_F32 */ ? gradients<float>(a, static_cast<char*>(ws), st)
                                         : gradients<bf16_t>(a, static_cast<char*>(ws), st);
}

}  // namespace conv2d
