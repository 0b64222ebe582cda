// int8_matmul.hip -- 8-bit integer products with a scale for every row (a
// token, a pixel) and every output channel, and the quantisation of rows.
//
//   y[m][n] = act( (sum_k q[m][k] * w[n][k]) * (q_scale[m] * w_scale[n]) [+ bias[n]] )
//
// The sums are exact in 32 bits (K <= 131071, so |sum| < 2^31 whatever the
// bytes); everything after them is fp32 and rounded once to the output type.
// Both operands are contiguous along k, which is how the matrix unit takes
// them: 16 bytes of k per lane.
//
// Four kernels:
//   skinny  up to 64 rows: the weights stream from memory straight into the
//           matrix unit's registers, 16 or 32 channels per workgroup, the waves
//           split k and join in LDS.  Bound by reading the weights (one row of
//           4096, 16384 channels: 67 MB in 18.0 us, 3.7 TB/s, from memory, in
//           14.6 where the last-level cache holds them) and, with more rows, by
//           every workgroup reading all of them.
//   tiled   BM rows x BN channels per workgroup, 128 bytes of k per stage,
//           copied from memory into two LDS buffers without passing through
//           registers.  Bound by the matrix unit.
//   stream  many rows with k up to 512: the weights stay in registers, the rows
//           stream past.  Bound by memory.
//   ragged  the same tiles where k or a row stride is no multiple of 16 or a
//           pointer is not aligned: rows are read as aligned words and
//           shifted into place in registers.
// A product with few tiles and a long k is split along k; the pieces' 32-bit
// sums go to the workspace and a second launch adds them.
#include <type_traits>

#include "mfma.hpp"
#include "operators.hpp"
#include "rowvec.hpp"
#include "tiles.hpp"

namespace conv2d {

namespace {

// Descriptor of rows [r0, rows) of a row-major byte matrix, starting at row
// r0: reads past its last byte (rows and k beyond the end) return 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const int8_t* p, long long ld, int r0, int rows, int tile,
                                                            int K) {
    const int n = min(rows - r0, tile);
    return make_rsrc(p + (long long)r0 * ld, (uint32_t)((long long)(n - 1) * ld + K));
}

// ReLU by comparison, so that a NaN (a row or weight that is not finite) stays.
__device__ __forceinline__ float finish(int acc, float scale, float bias, bool relu) {
    const float v = fmaf((float)acc, scale, bias);
    return relu && v < 0.0f ? 0.0f : v;
}

// ------------------------------------------------------------------ skinny

// One workgroup: NG * 16 channels, MT * 16 rows, all of k.  Channels are the
// rows of the 16x16 result, so a lane ends with 4 consecutive channels of one
// row.  128 bytes of k per wave and step, so that a step reads whole lines.  The
// loads of U steps stand before their products; the compiler sinks part of them
// (67 registers at U = 8, where all of them would take 128), so that fewer are in
// flight.
template <int MT, int NG, int U, typename OUT>
__global__ void int8_skinny_kernel(Int8Args a) {
    extern __shared__ i32x4 red[];   // [wave][NG][MT][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * (NG * 16);
    const auto wr = rows_rsrc(a.w, a.ldw, n0, a.N, NG * 16, a.K);
    const auto qr = rows_rsrc(a.q, a.ldq, 0, a.M, 64, a.K);
    const int row = lane & 15, c = lane >> 4;
    int wo[NG], qo[MT];
#pragma unroll
    for (int g = 0; g < NG; ++g)
        wo[g] = n0 + g * 16 + row < a.N ? (int)((g * 16 + row) * a.ldw) + c * 16 : kOOB;
#pragma unroll
    for (int t = 0; t < MT; ++t) qo[t] = t * 16 + row < a.M ? (int)((t * 16 + row) * a.ldq) + c * 16 : kOOB;
    i32x4 acc[NG][MT];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[g][t] = i32x4{0, 0, 0, 0};
    const int stride = waves * 128;
    for (int k0 = wave * 128; k0 < a.K; k0 += stride * U) {
        uint4 wv[U][2][NG], qv[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + u * stride + h * 64;
                const bool in = k + c * 16 < a.K;   // K is a multiple of 16
#pragma unroll
                for (int g = 0; g < NG; ++g) wv[u][h][g] = load16(wr, in && wo[g] != kOOB ? wo[g] + k : kOOB);
#pragma unroll
                for (int t = 0; t < MT; ++t) qv[u][h][t] = load16(qr, in && qo[t] != kOOB ? qo[t] + k : kOOB);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[g][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                            __builtin_bit_cast(i32x4, wv[u][h][g]), __builtin_bit_cast(i32x4, qv[u][h][t]), acc[g][t], 0, 0, 0);
    }
    constexpr int E = NG * MT * 64;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t) red[wave * E + (g * MT + t) * 64 + lane] = acc[g][t];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        i32x4 s = red[e];
        for (int k = 1; k < waves; ++k) s += red[k * E + e];
        const int tile = e >> 6, m = tile % MT * 16 + (e & 15), n = n0 + tile / MT * 16 + ((e & 63) >> 4) * 4;
        if (m >= a.M) continue;
        const float qs = a.q_scale[m];
        OUT* y = static_cast<OUT*>(a.y) + (long long)m * a.ldy;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N)
                store_f32<OUT>(y, n + r, finish(s[r], qs * a.w_scale[n + r], a.bias ? a.bias[n + r] : 0.0f, a.relu));
    }
}

// ------------------------------------------------------------------ tiles

// The matrix products of a 64-byte step of k: TI x TJ blocks of 16 channels x
// 16 rows.  The 16x16x64 form, not 32x32x32: on random bytes the matrix unit
// is held back by power, not by issue, and the small form, which moves half
// the accumulator bytes per product, sustains 3.8 against 3.3 POP/s (registers
// only; on zeros 4.7 against 4.9).  Neighbours share an operand, the turns of
// the order included (1% faster than starting every row of blocks anew).
template <int TI, int TJ>
__device__ __forceinline__ void products(i32x4 (&acc)[TI][TJ], const i32x4 (&w)[TI], const i32x4 (&q)[TJ]) {
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int n = 0; n < TI; ++n) {
            const int i = j & 1 ? TI - 1 - n : n;
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], q[j], acc[i][j], 0, 0, 0);
        }
}

// 16 bytes of results (8 bf16, 4 fp32 or int) to channels n .. of a row, fewer
// at the row's end.  The address is aligned to an element only (a row may have
// any length): one store all the same.
template <typename OUT> __device__ __forceinline__ void store_piece(OUT* row, int n, int N, const uint4& v) {
    constexpr int E = 16 / (int)sizeof(OUT);
    if (n + E <= N) {
        *reinterpret_cast<u32x4_unaligned*>(row + n) = __builtin_bit_cast(u32x4, v);
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (n + e < N)
                row[n + e] = sizeof(OUT) == 4 ? __builtin_bit_cast(OUT, (typename RawBytes<sizeof(OUT)>::type)w[e * (int)sizeof(OUT) / 4])
                                              : __builtin_bit_cast(OUT, (typename RawBytes<sizeof(OUT)>::type)(w[e / 2] >> (16 * (e & 1))));
    }
}

// Four channels of a row: scaled, biased, ReLU.
__device__ __forceinline__ float4 finish4(const Int8Args& a, const i32x4& acc, float qs, const float* sw,
                                          const float* sb) {
    const float4 ws = *reinterpret_cast<const float4*>(sw), bs = *reinterpret_cast<const float4*>(sb);
    return make_float4(finish(acc[0], qs * ws.x, bs.x, a.relu), finish(acc[1], qs * ws.y, bs.y, a.relu),
                       finish(acc[2], qs * ws.z, bs.z, a.relu), finish(acc[3], qs * ws.w, bs.w, a.relu));
}

// Block j of 16 rows of a wave's results, finished, into its piece of LDS (16
// x TI*16 elements).  In the 16x16 result lane l holds, in register r, channel
// 4 (l >> 4) + r of row l & 15.  The 16-byte pieces of a row are permuted with
// the row.  OUT int: the sums themselves.
template <int TI, typename OUT, int TJ>
__device__ __forceinline__ void results_to_lds(const Int8Args& a, const i32x4 (&acc)[TI][TJ], int j, float qs, char* lds,
                                               const float* sw, const float* sb) {
    constexpr int ROW = TI * 16 * (int)sizeof(OUT), PIECES = ROW / 16, MASK = (PIECES < 16 ? PIECES : 16) - 1;
    const int lane = threadIdx.x & 63, r16 = lane & 15;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int c = i * 16 + 4 * (lane >> 4), b = c * (int)sizeof(OUT);
        char* const at = lds + r16 * ROW + ((b / 16) ^ (r16 & MASK)) * 16 + b % 16;
        if constexpr (std::is_same_v<OUT, int>) {
            *reinterpret_cast<i32x4*>(at) = acc[i][j];
        } else {
            const float4 v = finish4(a, acc[i][j], qs, sw + c, sb + c);
            if constexpr (sizeof(OUT) == 4) *reinterpret_cast<float4*>(at) = v;
            else *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
    }
    wave_lds_fence();
}

// Results of a wave's TI*16 channels x TJ*16 rows: block by block of 16 rows
// through the wave's own piece of LDS, so that whole rows are written.  sq, sw,
// sb: the row scales, channel scales and biases in LDS, from the wave's first.
template <int TI, int TJ, typename OUT>
__device__ __forceinline__ void write_results(const Int8Args& a, i32x4 (&acc)[TI][TJ], char* lds, const float* sq,
                                              const float* sw, const float* sb, int m0, int n0, OUT* y, long long ldy) {
    constexpr bool kSums = std::is_same_v<OUT, int>;
    constexpr int ROW = TI * 16 * (int)sizeof(OUT), PIECES = ROW / 16;
    constexpr int MASK = (PIECES < 16 ? PIECES : 16) - 1;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        results_to_lds<TI, OUT>(a, acc, j, kSums ? 0.0f : sq[j * 16 + (lane & 15)], lds, sw, sb);
#pragma unroll
        for (int it = 0; it < 16 * PIECES / 64; ++it) {
            const int e = it * 64 + lane, r = e / PIECES, p = e % PIECES;
            const int m = m0 + j * 16 + r, n = n0 + p * (16 / (int)sizeof(OUT));
            if (m < a.M)
                store_piece<OUT>(y + m * ldy, n, a.N, *reinterpret_cast<const uint4*>(lds + r * ROW + (p ^ (r & MASK)) * 16));
        }
        wave_lds_fence();
    }
}

// The tile's scales and biases, one of each kind per thread: loaded before the
// first copies are issued, put into LDS behind them (zero past the last row
// and channel).
template <int BM, int BN> struct Scales {
    float q, w, b;
    __device__ __forceinline__ void load(const Int8Args& a, int m0, int n0) {
        const int m = m0 + threadIdx.x, n = n0 + threadIdx.x;
        q = w = b = 0.0f;
        if (threadIdx.x < BM && m < a.M) q = a.q_scale[m];
        if (threadIdx.x < BN && n < a.N) {
            w = a.w_scale[n];
            if (a.bias) b = a.bias[n];
        }
    }
    __device__ __forceinline__ void store(float* sq, float* sw, float* sb) const {
        if (threadIdx.x < BM) sq[threadIdx.x] = q;
        if (threadIdx.x < BN) {
            sw[threadIdx.x] = w;
            sb[threadIdx.x] = b;
        }
    }
};

template <typename OUT> __device__ __forceinline__ OUT* out_of(const Int8Args& a, int split) {
    return static_cast<OUT*>(a.y) + (std::is_same_v<OUT, int> ? (long long)split * a.M * a.N : 0);
}

__device__ __forceinline__ void copy_words(__amdgpu_buffer_rsrc_t r, char* dst, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)dst, 4, off, 0, 0, 0);
}

// Aligned operands.  Stage s + 2 is copied into the buffer that stage s has
// just been read from, a whole stage ahead of its use; the reads of a step
// are issued one step before its products, across the stages' border too, so
// there is one barrier per stage.
template <int BM, int BN, int WM, int WN, typename OUT>
__global__ __launch_bounds__(WM * WN * 64) void int8_tile_kernel(Int8Args a, int tm, int tn, int stages) {
    constexpr int NW = WM * WN, TI = BN / WN / 16, TJ = BM / WM / 16;
    constexpr int STAGE = (BM + BN) * kStageK;
    constexpr int CW = BN / 8 / NW, CQ = BM / 8 / NW;   // 1 KB copies per wave and stage
    constexpr bool kScaled = !std::is_same_v<OUT, int>;
    static_assert(BM <= NW * 64 && BN <= NW * 64, "one row and one channel per thread");
    static_assert(CW * 8 * NW == BN && CQ * 8 * NW == BM, "copies split evenly");
    static_assert(NW * 16 * TI * 16 * 4 <= STAGE, "results fit a stage");
    __shared__ uint4 lds0[STAGE / 16], lds1[STAGE / 16];
    __shared__ float sq[BM], sw[BN], sb[BN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const TileAt t = tile_at(tm, tn, BM, BN);
    const int kbase = t.split * stages * kStageK;
    const int nk = min(stages, (a.K - kbase + kStageK - 1) / kStageK);
    const int kend = min(kbase + nk * kStageK, a.K);
    const auto wr = rows_rsrc(a.w, a.ldw, t.n0, a.N, BN, a.K);
    const auto qr = rows_rsrc(a.q, a.ldq, t.m0, a.M, BM, a.K);

    // copy c of a wave: rows (c * NW + wave) * 8 + lane / 8; the lane's LDS
    // slot is fixed (base + 16 lane), so the lane reads the piece that
    // belongs there
    int wo[CW], qo[CQ];
    const int lr = lane >> 3;
    // (c * NW + wave) * 8 is a multiple of 8, so (row >> 1) & 7 takes the
    // row's bits 1..3: bit 3 is the parity of c * NW + wave
#pragma unroll
    for (int c = 0; c < CW; ++c) wo[c] = (int)(((c * NW + wave) * 8 + lr) * a.ldw);
#pragma unroll
    for (int c = 0; c < CQ; ++c) qo[c] = (int)(((c * NW + wave) * 8 + lr) * a.ldq);
    static_assert(NW % 2 == 0, "a wave's copies share their rows' bit 3");
    const int piece = ((lane & 7) ^ (((wave * 8 + lr) >> 1) & 7)) * 16;

    const int wm = wave / WN, wn = wave % WN;
    int ro[2];  // a lane's slot in a 16-row block, for the 2 steps of a stage
#pragma unroll
    for (int j = 0; j < 2; ++j) ro[j] = slot_of(lane & 15, 4 * j + (lane >> 4)) * 16;
    const int wbase = wn * (TI * 16) * kStageK, qbase = BN * kStageK + wm * (TJ * 16) * kStageK;

    i32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    i32x4 fw[2][TI], fq[2][TJ];
    Scales<BM, BN> scales;
    if constexpr (kScaled) scales.load(a, t.m0, t.n0);

#define I8_COPY(DST, S)                                                                                  \
    do {                                                                                                 \
        const int k_ = kbase + (S) * kStageK + piece;                                                    \
        const bool in_ = k_ < kend;                                                                      \
        char* const w_ = (DST) + wave * 1024;                                                            \
        _Pragma("unroll") for (int c = 0; c < CW; ++c) copy_kb(wr, w_ + c * NW * 1024, in_ ? wo[c] + k_ : kOOB); \
        _Pragma("unroll") for (int c = 0; c < CQ; ++c)                                                   \
            copy_kb(qr, w_ + BN * kStageK + c * NW * 1024, in_ ? qo[c] + k_ : kOOB);                     \
    } while (0)
#define I8_READ(SRC, J, SET)                                                                                  \
    do {                                                                                                      \
        _Pragma("unroll") for (int i = 0; i < TI; ++i) fw[SET][i] =                                           \
            *reinterpret_cast<const i32x4*>((SRC) + wbase + ro[J] + i * 16 * kStageK);                        \
        _Pragma("unroll") for (int j = 0; j < TJ; ++j) fq[SET][j] =                                           \
            *reinterpret_cast<const i32x4*>((SRC) + qbase + ro[J] + j * 16 * kStageK);                        \
    } while (0)
// The products of set SET with the reads (and copies) issued before them in
// the source spread between them: the compiler would otherwise sink the reads
// below the products to save registers, and the next step would wait for them.
#define I8_PRODUCTS(SET, COPIES)                                                                \
    do {                                                                                        \
        constexpr int PER = TI * TJ / (TI + TJ) > 0 ? TI * TJ / (TI + TJ) : 1;                  \
        products<TI, TJ>(acc, fw[SET], fq[SET]);                                                \
        _Pragma("unroll") for (int i = 0; i < TI + TJ; ++i) {                                   \
            __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);                                \
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                  \
            if (COPIES) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                      \
        }                                                                                       \
        __builtin_amdgcn_sched_barrier(0);                                                      \
    } while (0)
// One stage from CUR, whose step 0 is in set 0.  At the barrier this wave's
// reads of CUR are complete and its copies of the next stage have landed.
// Past the last stage the copies write zeros and the read is not used.
#define I8_STAGE(CUR, NXT, S)                                                                   \
    do {                                                                                        \
        I8_READ(CUR, 1, 1);                                                                     \
        I8_PRODUCTS(0, false);                                                                  \
        __atomic_signal_fence(__ATOMIC_SEQ_CST);                                                \
        __builtin_amdgcn_s_waitcnt(0x0070); /* vmcnt(0) lgkmcnt(0) */                           \
        __builtin_amdgcn_s_barrier();                                                           \
        __atomic_signal_fence(__ATOMIC_SEQ_CST);                                                \
        I8_READ(NXT, 0, 0);                                                                     \
        I8_COPY(CUR, (S) + 2);                                                                  \
        I8_PRODUCTS(1, true);                                                                   \
    } while (0)

    {
        // every buffer a restrict argument of one function: the compiler then
        // does not make the reads of one wait for the copies into the other
        auto loop = [&](char* __restrict__ b0, char* __restrict__ b1) __attribute__((always_inline)) {
            I8_COPY(b0, 0);
            I8_COPY(b1, 1);
            if constexpr (kScaled) scales.store(sq, sw, sb);
            __builtin_amdgcn_s_waitcnt(0x0070);
            __builtin_amdgcn_s_barrier();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            I8_READ(b0, 0, 0);
            for (int s = 0; s < nk; s += 2) {
                I8_STAGE(b0, b1, s);
                if (s + 1 < nk) I8_STAGE(b1, b0, s + 1);
            }
        };
        loop(reinterpret_cast<char*>(lds0), reinterpret_cast<char*>(lds1));
    }
#undef I8_COPY
#undef I8_READ
#undef I8_PRODUCTS
#undef I8_STAGE
    __builtin_amdgcn_s_waitcnt(0x0070);   // no copy is in flight when the buffers take the results
    __syncthreads();
    write_results<TI, TJ, OUT>(a, acc, reinterpret_cast<char*>(lds0) + wave * (16 * TI * 16 * (int)sizeof(OUT)),
                               sq + wm * TJ * 16, sw + wn * TI * 16, sb + wn * TI * 16, t.m0 + wm * TJ * 16, t.n0 + wn * TI * 16,
                               out_of<OUT>(a, t.split), a.ldy);
}

// ------------------------------------------------------------------ streaming

// Short rows (k up to 512): memory bounds them, so the weights stay in
// registers and the rows stream past.  A workgroup of 8 waves owns BN = WN * 64
// channels, a wave 64 of them and every WM-th group of 16 * TJ rows; row tiles
// of BM rows come through three LDS buffers, two tiles ahead of their use, and
// results leave as whole 128-byte lines while the next tiles arrive.  The tile
// kernel at one or two workgroups per compute unit loads, then stores: 30.7 us
// where this takes 20.3 (100352 x 256 rows, 256 channels, bf16 results).
template <int KS, int WN, int TJ, typename OUT> struct StreamShape {
    static constexpr int WM = 8 / WN, BM = WM * 16 * TJ, BN = WN * 64;
    static constexpr int PR = KS * 4;                 // 16-byte pieces of a row
    static constexpr int ROWS = BM * KS * 64;         // bytes of a tile
    static constexpr int BUF = ROWS + 8 * 64 * 4;     // and of its scales, 64 from every wave
    static constexpr int COPIES = BM * PR / 512;      // of rows, per wave and tile
    static_assert(COPIES * 512 == BM * PR && BM <= 512, "copies split evenly");
};

// Slot of a row's 16-byte piece: 16 rows read at one piece hit all banks.
template <int PR> __device__ __forceinline__ int stream_swizzle(int row) {
    if constexpr (PR >= 16) return row & 15;
    else return (row / (16 / PR)) & (PR - 1);
}

// This wave's LDS operations complete, then the workgroup barrier; copies in
// flight are not waited for.
__device__ __forceinline__ void stream_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

constexpr int vmcnt_of(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0f70; }  // lgkmcnt, expcnt: no wait

// Block j of 16 rows of a wave's results to memory, straight from registers:
// fp32 lanes hold 16 bytes already; bf16 ones hold 8, and the exchange of
// neighbouring groups of 16 lanes between two blocks of channels makes them 16.
// Every store writes 64 contiguous bytes of 16 rows.
template <int TI, typename OUT, int TJ>
__device__ __forceinline__ void store_rows(const Int8Args& a, const i32x4 (&acc)[TI][TJ], int j, float qs,
                                           const float* sw, const float* sb, int m, int n0, bool whole) {
    const int group = (threadIdx.x & 63) >> 4;
    OUT* row = static_cast<OUT*>(a.y) + m * a.ldy;
    // whole: rows are multiples of 16 bytes and written past the cache
    auto put = [&](int n, const uint4& v) {
        if (m >= a.M) return;
        if (!whole) store_piece<OUT>(row, n, a.N, v);
        else if (n < a.N) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(row + n));
    };
    if constexpr (sizeof(OUT) == 4) {
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int c = i * 16 + group * 4;
            put(n0 + c, __builtin_bit_cast(uint4, finish4(a, acc[i][j], qs, sw + c, sb + c)));
        }
    } else {
#pragma unroll
        for (int i = 0; i < TI; i += 2) {
            const int c = i * 16 + group * 4;
            const float4 u = finish4(a, acc[i][j], qs, sw + c, sb + c);
            const float4 v = finish4(a, acc[i + 1][j], qs, sw + 16 + c, sb + 16 + c);
            // groups 0 .. 3 then hold channels 0-7 of block i, 0-7 of i + 1,
            // 8-15 of i, 8-15 of i + 1
            const u32x2_t p = __builtin_amdgcn_permlane16_swap(pack_bf16x2(u.x, u.y), pack_bf16x2(v.x, v.y), false, false);
            const u32x2_t q = __builtin_amdgcn_permlane16_swap(pack_bf16x2(u.z, u.w), pack_bf16x2(v.z, v.w), false, false);
            put(n0 + (i + (group & 1)) * 16 + (group >> 1) * 8, make_uint4(p.x, q.x, p.y, q.y));
        }
    }
}

template <int KS, int WN, int TJ, typename OUT>
__global__ __launch_bounds__(512) void int8_stream_kernel(Int8Args a, int tiles, int cols, bool whole) {
    using S = StreamShape<KS, WN, TJ, OUT>;
    constexpr int TI = 4, D = S::COPIES + 1;
    __shared__ uint4 lds0[S::BUF / 16], lds1[S::BUF / 16], lds2[S::BUF / 16];
    __shared__ float scales[2 * S::BN];   // of the channels, then their biases
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int index = xcd_tile_index(), col = index % cols, first = index / cols, stride = gridDim.x / cols;
    const int n0 = col * S::BN;
    const int count = first < tiles ? (tiles - first - 1) / stride + 1 : 0;

    // the wave's weights: lane l holds channel l & 15 of a block at k 16 (l >> 4)
    i32x4 w[KS][TI];
    {
        const auto wr = rows_rsrc(a.w, a.ldw, n0, a.N, S::BN, a.K);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int c = wn * 64 + i * 16 + (lane & 15);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int k = ks * 64 + (lane >> 4) * 16;
                w[ks][i] = __builtin_bit_cast(i32x4, load16(wr, n0 + c < a.N && k < a.K ? (int)(c * a.ldw) + k : kOOB));
            }
        }
    }
    for (int c = threadIdx.x; c < S::BN; c += 512) {
        scales[c] = n0 + c < a.N ? a.w_scale[n0 + c] : 0.0f;
        scales[S::BN + c] = a.bias && n0 + c < a.N ? a.bias[n0 + c] : 0.0f;
    }
    // before the function below, whose reads of its restrict argument the
    // compiler may move up to its start, past the barriers inside
    __syncthreads();
    int qo[S::COPIES];
#pragma unroll
    for (int c = 0; c < S::COPIES; ++c) {
        const int s = (c * 8 + wave) * 64 + lane, row = s / S::PR, k = (s % S::PR ^ stream_swizzle<S::PR>(row)) * 16;
        qo[c] = k < a.K ? (int)(row * a.ldq) + k : kOOB;
    }
    int ro[KS];   // the lane's slot for each 64 bytes of k, in a block of 16 rows
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        ro[ks] = ((lane & 15) * S::PR + ((ks * 4 + (lane >> 4)) ^ stream_swizzle<S::PR>(lane & 15))) * 16;

// Tile T (of this workgroup's) into DST: the rows, and 64 scales from every
// wave.  Past the last tile it writes zeros: the number of copies in flight
// is always the same.
#define I8_FETCH(DST, T)                                                                                   \
    do {                                                                                                   \
        const int m_ = (T) < count ? (first + (T) * stride) * S::BM : a.M;                                 \
        const int left_ = min(a.M - m_, S::BM);                                                            \
        const auto qr_ = make_rsrc(a.q + (long long)m_ * a.ldq,                                            \
                                   left_ > 0 ? (uint32_t)((long long)(left_ - 1) * a.ldq + a.K) : 0u);     \
        const auto sr_ = make_rsrc(a.q_scale + m_, (uint32_t)max(left_, 0) * 4u);                          \
        _Pragma("unroll") for (int c = 0; c < S::COPIES; ++c)                                              \
            copy_kb(qr_, (DST) + (c * 8 + wave) * 1024, qo[c]);                                            \
        copy_words(sr_, (DST) + S::ROWS + wave * 256, wave * 256 + lane * 4);                              \
    } while (0)
// One tile from CUR, which has landed; the tile after the next goes to DST,
// which the barrier has freed.  Before the tile's stores are issued, all but
// the D youngest operations (the copies of tile T + 2) are waited for: the next
// tile's copies and the last tile's stores, both a whole tile old.
#define I8_TILE(CUR, DST, T)                                                                               \
    do {                                                                                                   \
        stream_barrier();                                                                                  \
        I8_FETCH(DST, (T) + 2);                                                                            \
        i32x4 acc[TI][TJ];                                                                                 \
        _Pragma("unroll") for (int i = 0; i < TI; ++i)                                                     \
            _Pragma("unroll") for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};                  \
        _Pragma("unroll") for (int ks = 0; ks < KS; ++ks) {                                                \
            i32x4 q[TJ];                                                                                   \
            _Pragma("unroll") for (int j = 0; j < TJ; ++j) q[j] = *reinterpret_cast<const i32x4*>(         \
                (CUR) + (wm * TJ + j) * 16 * KS * 64 + ro[ks]);                                            \
            products<TI, TJ>(acc, w[ks], q);                                                               \
        }                                                                                                  \
        const int m_ = (first + (T) * stride) * S::BM;                                                     \
        __atomic_signal_fence(__ATOMIC_SEQ_CST);                                                           \
        __builtin_amdgcn_s_waitcnt(vmcnt_of(D));                                                           \
        __atomic_signal_fence(__ATOMIC_SEQ_CST);                                                           \
        _Pragma("unroll") for (int j = 0; j < TJ; ++j) {                                                   \
            const int row_ = (wm * TJ + j) * 16;                                                           \
            const float qs_ = reinterpret_cast<const float*>((CUR) + S::ROWS)[row_ + (lane & 15)];         \
            store_rows<TI, OUT>(a, acc, j, qs_, sc, sc + S::BN, m_ + row_ + (lane & 15), n0 + wn * 64, whole); \
        }                                                                                                  \
    } while (0)

    // every piece of LDS a restrict argument of one function: the compiler then
    // does not make the reads of one wait for the copies into another
    auto run = [&](char* __restrict__ b0, char* __restrict__ b1, char* __restrict__ b2,
                   const float* __restrict__ sc) __attribute__((always_inline)) {
        I8_FETCH(b0, 0);
        I8_FETCH(b1, 1);
        __builtin_amdgcn_s_waitcnt(vmcnt_of(D));
        for (int t = 0; t < count; t += 3) {
            I8_TILE(b0, b2, t);
            if (t + 1 >= count) break;
            I8_TILE(b1, b0, t + 1);
            if (t + 2 >= count) break;
            I8_TILE(b2, b1, t + 2);
        }
    };
    run(reinterpret_cast<char*>(lds0), reinterpret_cast<char*>(lds1), reinterpret_cast<char*>(lds2),
        scales + wn * 64);
#undef I8_FETCH
#undef I8_TILE
    __builtin_amdgcn_s_waitcnt(0x0070);   // no copy outlives the workgroup's LDS
}

// 16 bytes from any byte offset: two loads of whole words, shifted.  Bytes
// from k on are cleared (`left` of them are inside the row).
struct Unaligned {
    uint4 lo;
    uint32_t hi;
};

__device__ __forceinline__ Unaligned load_words(__amdgpu_buffer_rsrc_t r, int off) {
    Unaligned u;
    u.lo = load16(r, off & ~3);
    u.hi = __builtin_amdgcn_raw_buffer_load_b32(r, (off & ~3) + 16, 0, 0);
    return u;
}

__device__ __forceinline__ uint4 shift_words(const Unaligned& u, int off, int left) {
    const uint32_t w[5] = {u.lo.x, u.lo.y, u.lo.z, u.lo.w, u.hi};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], off & 3);
        const int n = left - 4 * i;
        o[i] = n >= 4 ? o[i] : n <= 0 ? 0u : o[i] & ((1u << (8 * n)) - 1u);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Operands of any alignment: the loads of stage s + 1 are in flight during
// the products of stage s.
template <int BM, int BN, int WM, int WN, typename OUT>
__global__ __launch_bounds__(WM * WN * 64) void int8_ragged_kernel(Int8Args a, int tm, int tn, int stages) {
    constexpr int NT = WM * WN * 64, TI = BN / WN / 16, TJ = BM / WM / 16;
    constexpr int STAGE = (BM + BN) * kStageK, PER = (BM + BN) * 8 / NT;
    constexpr bool kScaled = !std::is_same_v<OUT, int>;
    static_assert(BM <= NT && BN <= NT, "one row and one channel per thread");
    static_assert(BN * 8 % NT == 0 && BM * 8 % NT == 0, "pieces split evenly");
    constexpr int OUTB = WM * WN * 16 * TI * 16 * 4;
    __shared__ uint4 lds[(STAGE > OUTB ? STAGE : OUTB) / 16];
    __shared__ float sq[BM], sw[BN], sb[BN];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const TileAt t = tile_at(tm, tn, BM, BN);
    const int kbase = t.split * stages * kStageK;
    const int nk = min(stages, (a.K - kbase + kStageK - 1) / kStageK);
    // bases down to a whole word, sizes up to one: an aligned word that holds
    // a byte of the matrix is read whole
    const int8_t* wp = a.w + (long long)t.n0 * a.ldw;
    const int8_t* qp = a.q + (long long)t.m0 * a.ldq;
    const int wsh = (int)(reinterpret_cast<uintptr_t>(wp) & 3), qsh = (int)(reinterpret_cast<uintptr_t>(qp) & 3);
    const auto wr = make_rsrc(wp - wsh, (uint32_t)((wsh + (long long)(min(a.N - t.n0, BN) - 1) * a.ldw + a.K + 3) & ~3LL));
    const auto qr = make_rsrc(qp - qsh, (uint32_t)((qsh + (long long)(min(a.M - t.m0, BM) - 1) * a.ldq + a.K + 3) & ~3LL));
    int off[PER], slot[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        const int e = c * NT + tid, row = e >> 3;   // rows of w, then rows of q
        off[c] = row < BN ? wsh + (int)(row * a.ldw) : qsh + (int)((row - BN) * a.ldq);
        slot[c] = slot_of(row, e & 7);
    }
    const int piece = (tid & 7) * 16;
    const int wm = wave / WN, wn = wave % WN;
    i32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    Scales<BM, BN> scales;
    if constexpr (kScaled) {
        scales.load(a, t.m0, t.n0);
        scales.store(sq, sw, sb);
    }
    Unaligned v[PER];
    auto fetch = [&](int s) {
        const int k = kbase + s * kStageK + piece;
#pragma unroll
        for (int c = 0; c < PER; ++c)
            v[c] = load_words(c * NT / 8 < BN ? wr : qr, k < a.K ? off[c] + k : kOOB & ~31);
    };
    fetch(0);
    for (int s = 0; s < nk; ++s) {
        const int k = kbase + s * kStageK + piece;
        __syncthreads();
#pragma unroll
        for (int c = 0; c < PER; ++c) lds[slot[c]] = shift_words(v[c], off[c] + k, a.K - k);
        __syncthreads();
        if (s + 1 < nk) fetch(s + 1);
        const char* base = reinterpret_cast<const char*>(lds);
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            const int ro = slot_of(lane & 15, 4 * step + (lane >> 4)) * 16;
            i32x4 fw[TI], fq[TJ];
#pragma unroll
            for (int i = 0; i < TI; ++i)
                fw[i] = *reinterpret_cast<const i32x4*>(base + (wn * TI + i) * 16 * kStageK + ro);
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                fq[j] = *reinterpret_cast<const i32x4*>(base + BN * kStageK + (wm * TJ + j) * 16 * kStageK + ro);
            products<TI, TJ>(acc, fw, fq);
        }
    }
    __syncthreads();
    write_results<TI, TJ, OUT>(a, acc, reinterpret_cast<char*>(lds) + wave * (16 * TI * 16 * (int)sizeof(OUT)),
                               sq + wm * TJ * 16, sw + wn * TI * 16, sb + wn * TI * 16, t.m0 + wm * TJ * 16, t.n0 + wn * TI * 16,
                               out_of<OUT>(a, t.split), a.ldy);
}

// Adds the pieces of a product that was split along k and finishes it.
template <typename OUT>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Args a, const int* sums, int splits) {
    const int total = a.M * a.N;   // below 256 tiles of 64 x 64
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int m = i / a.N, n = i % a.N;
    int s = 0;
    for (int k = 0; k < splits; ++k) s += sums[(long long)k * total + i];
    store_f32<OUT>(static_cast<OUT*>(a.y) + m * a.ldy, n,
                   finish(s, a.q_scale[m] * a.w_scale[n], a.bias ? a.bias[n] : 0.0f, a.relu));
}

// ------------------------------------------------------------------ rows to 8 bits

// LPP lanes (a power of two) per row, J vectors of a lane in registers.
template <typename T, int V, int J>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int8_t* q, float* scale, int M, int K,
                                                            long long ldx, long long ldq, int LPP) {
    const int l = threadIdx.x % LPP;
    const long long row = (long long)blockIdx.x * (256 / LPP) + threadIdx.x / LPP;
    if (row >= M) return;
    const T* p = x + row * ldx;
    float v[J][V];
    uint32_t top = 0;
    typename Vec<T, V>::raw raw[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * LPP) * V;
        if (c < K) raw[j] = Vec<T, V>::load(p + vector_start<V>(c, K));
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if ((l + j * LPP) * V >= K) break;
        Vec<T, V>::unpack(raw[j], v[j]);
#pragma unroll
        for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(v[j][e]) & 0x7fffffffu);
    }
    const RowScale s = row_scale(lanes_max(top, LPP));
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + j * LPP) * V;
        if (c < K) store_quantised<V>(q + row * ldq + vector_start<V>(c, K), v[j], s.inv);
    }
    if (l == 0) scale[row] = s.scale;
}

// One workgroup per row; the row is read twice (the second time from L2).
template <typename T, int V>
__global__ __launch_bounds__(256) void quantize_long_rows_kernel(const T* x, int8_t* q, float* scale, int K,
                                                                 long long ldx, long long ldq) {
    __shared__ uint32_t tops[4];
    const long long row = blockIdx.x;
    const T* p = x + row * ldx;
    uint32_t top = 0;
#pragma unroll 4
    for (int c = threadIdx.x * V; c < K; c += 256 * V) {
        float v[V];
        Vec<T, V>::unpack(Vec<T, V>::load(p + vector_start<V>(c, K)), v);
#pragma unroll
        for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    top = lanes_max(top, 64);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    const RowScale s = row_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll 4
    for (int c = threadIdx.x * V; c < K; c += 256 * V) {
        float v[V];
        const int at = vector_start<V>(c, K);
        Vec<T, V>::unpack(Vec<T, V>::load(p + at), v);
        store_quantised<V>(q + row * ldq + at, v, s.inv);
    }
    if (threadIdx.x == 0) scale[row] = s.scale;
}

template <typename T, int V>
hipError_t quantize(const void* x, void* q, float* scale, int M, int K, long long ldx, long long ldq, hipStream_t st) {
    const int cv = (K + V - 1) / V;
    int lpp = 1;
    while (lpp < cv && lpp < 64) lpp <<= 1;
    const int j = (cv + lpp - 1) / lpp;
    const int per = j > 4 ? 1 : 256 / lpp;   // rows of a workgroup
    auto k = j == 1 ? quantize_rows_kernel<T, V, 1> : j == 2 ? quantize_rows_kernel<T, V, 2> : quantize_rows_kernel<T, V, 4>;
    // a launch counts its threads in 32 bits: 2^23 workgroups of 256 at a time
    const long long most = (long long)per << 23;
    for (long long m = 0; m < M; m += most) {
        const int rows = (int)(M - m < most ? M - m : most);
        const T* xt = static_cast<const T*>(x) + m * ldx;
        int8_t* qt = static_cast<int8_t*>(q) + m * ldq;
        if (j > 4) quantize_long_rows_kernel<T, V><<<rows, 256, 0, st>>>(xt, qt, scale + m, K, ldx, ldq);
        else k<<<(int)(((long long)rows + per - 1) / per), 256, 0, st>>>(xt, qt, scale + m, rows, K, ldx, ldq, lpp);
    }
    return hipGetLastError();
}

// ------------------------------------------------------------------ host

bool aligned_operands(const Int8Args& a) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    return a.K % 16 == 0 && a.ldq % 16 == 0 && a.ldw % 16 == 0 && al(a.q) && al(a.w);
}

enum { kSkinny, kStream, kTile256, kTile128, kTile64, kRagged128, kRagged64 };

struct Int8Plan {
    int kernel, bm, bn, tm, tn, splits, stages;
};

// Rows up to kSkinnyRows read the weights once whatever the tile, so the
// skinny kernel, which does nothing else, takes them.  Larger products take
// the largest tile that still gives every compute unit one; few tiles of a
// long k are split along it until they do.
constexpr int kSkinnyRows = 64;
constexpr int kUnits = 256;

// The streaming kernel's instance for a K and N: ks of 64 bytes of k, wn of 64
// channels, tj blocks of 16 rows a wave.
constexpr int kStreamK = 512;

struct StreamTile {
    int ks, wn, tj, bm, bn;
};

StreamTile stream_tile(int K, int N) {
    StreamTile t;
    t.ks = K <= 64 ? 1 : K <= 128 ? 2 : K <= 256 ? 4 : 8;
    t.wn = N > 128 ? 4 : N > 64 || t.ks == 8 ? 2 : 1;
    // at least one 16-byte copy per thread and tile, and no more than 32 KB
    t.tj = t.wn == 4 ? (t.ks == 1 ? 4 : t.ks == 8 ? 1 : 2) : t.wn == 2 && t.ks == 1 ? 2 : 1;
    t.bm = 8 / t.wn * 16 * t.tj;
    t.bn = t.wn * 64;
    return t;
}

Int8Plan make_int8_plan(int M, int K, int N, bool aligned) {
    Int8Plan p;
    p.stages = p.splits = 1;
    if (aligned && M > kSkinnyRows && K <= kStreamK) {
        const StreamTile t = stream_tile(K, N);
        p.kernel = kStream;
        p.bm = t.bm;
        p.bn = t.bn;
        p.tm = (M + p.bm - 1) / p.bm;
        p.tn = (N + p.bn - 1) / p.bn;
        // enough tiles for each workgroup to earn the load of its weights:
        // 6 a compute unit up to k = 256 (16384 x 256 -> 1024, 4 each: 15.9 us
        // against 14.3 tiled; 100352 x 256 -> 256, 6 each: 20.3 against 30.7),
        // 16 above, where a tile is half as long (16384 x 512 -> 1024, 8 each:
        // 22.4 against 17.0; 65536 x 512 -> 512, 16 each: 30.4 against 37.6)
        if ((long long)p.tm * p.tn >= (K <= 256 ? 6 : 16) * kUnits && (K <= 256 || N > 64)) return p;
    }
    auto tiles = [&](int b) { return (long long)((M + b - 1) / b) * ((N + b - 1) / b); };
    if (aligned && M <= kSkinnyRows) {
        p.kernel = kSkinny;
        p.bm = kSkinnyRows;
        p.bn = 16;
    } else {
        // no tile wider than the channels: 65536 x 512 -> 64 takes 9.9 us in
        // tiles of 64 and 16.3 in tiles of 256
        const int b = aligned && N > 128 && tiles(256) >= kUnits ? 256 : N > 64 && tiles(128) >= kUnits ? 128 : 64;
        p.kernel = aligned ? (b == 256 ? kTile256 : b == 128 ? kTile128 : kTile64) : b == 128 ? kRagged128 : kRagged64;
        p.bm = p.bn = b;
    }
    p.tm = (M + p.bm - 1) / p.bm;
    p.tn = (N + p.bn - 1) / p.bn;
    const int all = (K + kStageK - 1) / kStageK;
    if (p.kernel != kSkinny) {
        const long long t = (long long)p.tm * p.tn;
        // a piece is at least 4 stages long
        const long long want = t >= kUnits ? 1 : kUnits / t, most = all / 4;
        p.splits = (int)(want < most ? want : most);
        if (p.splits < 1) p.splits = 1;
    }
    p.stages = (all + p.splits - 1) / p.splits;
    p.splits = (all + p.stages - 1) / p.stages;
    return p;
}

template <int MT, int NG, int U, typename OUT> hipError_t skinny_instance(const Int8Args& a, int waves, hipStream_t st) {
    int8_skinny_kernel<MT, NG, U, OUT><<<(a.N + NG * 16 - 1) / (NG * 16), waves * 64, waves * NG * MT * 1024, st>>>(a);
    return hipGetLastError();
}

// Two groups of 16 channels per workgroup use a row's values twice, where half
// the workgroups still fill the chip and the rows are more than 16 (weights from
// memory: 40 rows of 4096, 16384 channels 28.4 us against 38.0; 64 rows of 8192,
// 8192 channels 34.4 against 45.2; but 64 rows of 4096, 4096 channels 18.2 against
// 16.4, and one row of 4096, 16384 channels 22.2 against 18.0).  Waves that split
// k: 4, or up to 16 where that leaves the chip few, of at least 128 bytes of k
// each.  Up to 16 rows the steps whose loads stand together follow what is left
// for a wave: 1 x 4096 -> 16384 takes 18.0 us with 8 and 22.9 with 4, 1 x 2048 ->
// 2048 4.9 with 2 and 5.7 with 4.
template <typename OUT> hipError_t skinny(const Int8Args& a, hipStream_t st) {
    const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const bool pairs = mt > 1 && a.N >= 32 * kUnits;
    const int blocks = (a.N + (pairs ? 31 : 15)) / (pairs ? 32 : 16);
    int waves = 4;   // 8 of 4 x 2 blocks: 64 KB of LDS
    while (waves < (pairs && mt == 4 ? 8 : 16) && blocks * waves < 16 * kUnits && waves * 2 * 128 <= a.K) waves *= 2;
    const int steps = (a.K + waves * 128 - 1) / (waves * 128);
    if (mt == 1)
        return steps > 4   ? skinny_instance<1, 1, 8, OUT>(a, waves, st)
               : steps > 2 ? skinny_instance<1, 1, 4, OUT>(a, waves, st)
                           : skinny_instance<1, 1, 2, OUT>(a, waves, st);
    if (mt == 2) return pairs ? skinny_instance<2, 2, 2, OUT>(a, waves, st) : skinny_instance<2, 1, 2, OUT>(a, waves, st);
    return pairs ? skinny_instance<4, 2, 2, OUT>(a, waves, st) : skinny_instance<4, 1, 2, OUT>(a, waves, st);
}

// Rows of y are whole, aligned 16-byte pieces.
bool vector_stores(const Int8Args& a, int es) {
    return a.ldy * es % 16 == 0 && a.N * (long long)es % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
}

template <int KS, int WN, int TJ, typename OUT>
hipError_t stream_instance(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    constexpr auto kernel = int8_stream_kernel<KS, WN, TJ, OUT>;
    const long long slots = (long long)cu_count(dev) * blocks_per_cu<kernel>(512, dev);
    long long rows = slots / p.tn;   // workgroups per block of channels
    rows = rows < 1 ? 1 : rows > p.tm ? p.tm : rows;
    kernel<<<(unsigned)(rows * p.tn), 512, 0, st>>>(a, p.tm, p.tn, vector_stores(a, (int)sizeof(OUT)));
    return hipGetLastError();
}

template <typename OUT> hipError_t stream(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
    const StreamTile t = stream_tile(a.K, a.N);
    if (t.wn == 4)
        return t.ks == 1 ? stream_instance<1, 4, 4, OUT>(a, p, st) : t.ks == 2 ? stream_instance<2, 4, 2, OUT>(a, p, st)
               : t.ks == 4 ? stream_instance<4, 4, 2, OUT>(a, p, st) : stream_instance<8, 4, 1, OUT>(a, p, st);
    if (t.wn == 2)
        return t.ks == 1 ? stream_instance<1, 2, 2, OUT>(a, p, st) : t.ks == 2 ? stream_instance<2, 2, 1, OUT>(a, p, st)
               : t.ks == 4 ? stream_instance<4, 2, 1, OUT>(a, p, st) : stream_instance<8, 2, 1, OUT>(a, p, st);
    return t.ks == 1 ? stream_instance<1, 1, 1, OUT>(a, p, st) : t.ks == 2 ? stream_instance<2, 1, 1, OUT>(a, p, st)
                                                                           : stream_instance<4, 1, 1, OUT>(a, p, st);
}

template <typename OUT> hipError_t tiled(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
    const int blocks = p.tm * p.tn * p.splits;
    switch (p.kernel) {
    case kTile256: int8_tile_kernel<256, 256, 2, 4, OUT><<<blocks, 512, 0, st>>>(a, p.tm, p.tn, p.stages); break;
    case kTile128: int8_tile_kernel<128, 128, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages); break;
    case kTile64: int8_tile_kernel<64, 64, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages); break;
    case kRagged128: int8_ragged_kernel<128, 128, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages); break;
    default: int8_ragged_kernel<64, 64, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages); break;
    }
    return hipGetLastError();
}

size_t split_bytes(const Int8Plan& p, int M, int N) {
    return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

}  // namespace

// The most rows of one launch (more are taken in equal parts) and the most
// channels: indexes stay below 2^31 past the end of the last tile too.  The
// longest row: sums stay below 2^31.
constexpr int kMostRows = 1 << 29, kMostChannels = 1 << 27, kMostK = 131071;

static int part_rows(int M) {
    const long long parts = ((long long)M + kMostRows - 1) / kMostRows;
    return (int)((M + parts - 1) / parts);
}

// One figure for either alignment.
size_t int8_matmul_workspace(int M, int K, int N) {
    if (K > kMostK || N > kMostChannels) return 0;   // refused
    M = part_rows(M);
    const size_t u = split_bytes(make_int8_plan(M, K, N, false), M, N);
    const size_t v = K % 16 ? 0 : split_bytes(make_int8_plan(M, K, N, true), M, N);
    return u > v ? u : v;
}

bool int8_matmul_supports(int M, int K, int N, long long ldq, long long ldw) {
    // a tile's rows are addressed with 31 bits; a launch counts its threads in 32
    // (the other two kernels have fewer)
    if (K > kMostK || ldq > (1 << 22) || ldw > (1 << 22) || N > kMostChannels) return false;
    for (int al = 0; al < 2; ++al) {
        const Int8Plan p = make_int8_plan(part_rows(M), K, N, al);
        if (p.kernel != kStream && p.kernel != kSkinny &&
            (long long)p.tm * p.tn * p.splits * (p.kernel == kTile256 ? 512 : 256) > 0xffffffffLL)
            return false;
    }
    return true;
}

hipError_t launch_int8_matmul(const Int8Args& a, int out_f32, void* ws, hipStream_t st) {
    if (a.M > kMostRows) {   // parts of 2^28 rows and more are never split along k: they share no workspace
        const int rows = part_rows(a.M);
        for (long long m = 0; m < a.M; m += rows) {
            Int8Args part = a;
            part.M = (int)(a.M - m < rows ? a.M - m : rows);
            part.q += m * a.ldq;
            part.q_scale += m;
            part.y = static_cast<char*>(a.y) + m * a.ldy * (out_f32 ? 4 : 2);
            const hipError_t e = launch_int8_matmul(part, out_f32, ws, st);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const Int8Plan p = make_int8_plan(a.M, a.K, a.N, aligned_operands(a));
    if (p.kernel == kStream) return out_f32 ? stream<float>(a, p, st) : stream<bf16_t>(a, p, st);
    if (p.kernel == kSkinny) return out_f32 ? skinny<float>(a, st) : skinny<bf16_t>(a, st);
    if (p.splits == 1) return out_f32 ? tiled<float>(a, p, st) : tiled<bf16_t>(a, p, st);
    Int8Args part = a;
    part.y = ws;
    part.ldy = a.N;
    hipError_t e = tiled<int>(part, p, st);
    if (e != hipSuccess) return e;
    const unsigned blocks = (unsigned)(((long long)a.M * a.N + 255) / 256);
    if (out_f32) int8_join_kernel<float><<<blocks, 256, 0, st>>>(a, static_cast<const int*>(ws), p.splits);
    else int8_join_kernel<bf16_t><<<blocks, 256, 0, st>>>(a, static_cast<const int*>(ws), p.splits);
    return hipGetLastError();
}

hipError_t launch_quantize_rows(const void* x, void* q, float* scale, int M, int K, long long ldx, long long ldq,
                                int dtype, hipStream_t st) {
    // 16 bytes whatever the alignment, the last vector of a row over part of the
    // one before, unless the row is shorter
    const int es = dtype == 0 /* CONV2D_F32 */ ? 4 : 2;
    int v = 16 / es;
    while (v > K) v >>= 1;
    if (v * es < 16)
        while (K % v) v >>= 1;
    if (es == 4)
        return v == 4 ? quantize<float, 4>(x, q, scale, M, K, ldx, ldq, st)
               : v == 2 ? quantize<float, 2>(x, q, scale, M, K, ldx, ldq, st)
                        : quantize<float, 1>(x, q, scale, M, K, ldx, ldq, st);
    return v == 8 ? quantize<bf16_t, 8>(x, q, scale, M, K, ldx, ldq, st)
           : v == 4 ? quantize<bf16_t, 4>(x, q, scale, M, K, ldx, ldq, st)
           : v == 2 ? quantize<bf16_t, 2>(x, q, scale, M, K, ldx, ldq, st)
                    : quantize<bf16_t, 1>(x, q, scale, M, K, ldx, ldq, st);
}

}  // namespace conv2d
