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
// Three kernels:
//   skinny  up to 64 rows: the weights stream from memory straight into the
//           matrix unit's registers, 16 channels per workgroup, the waves
//           split k and join in LDS.  Bound by reading the weights.
//   tiled   BM rows x BN channels per workgroup, 128 bytes of k per stage,
//           copied from memory into two LDS buffers without passing through
//           registers.  Bound by the matrix unit.
//   ragged  the same tiles where k or a row stride is no multiple of 16 or a
//           pointer is not aligned: rows are read as aligned words and
//           shifted into place in registers.
// A product with few tiles and a long k is split along k; the pieces' 32-bit
// sums go to the workspace and a second launch adds them.
#include <type_traits>

#include "mfma.hpp"
#include "rowvec.hpp"

namespace conv2d {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

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

// One workgroup: 16 channels, MT * 16 rows, all of k.  Channels are the rows
// of the 16x16 result, so a lane ends with 4 consecutive channels of one row.
template <int MT, typename OUT>
__global__ void int8_skinny_kernel(Int8Args a) {
    extern __shared__ i32x4 red[];   // [wave][MT][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * 16;
    const auto wr = rows_rsrc(a.w, a.ldw, n0, a.N, 16, a.K);
    const auto qr = rows_rsrc(a.q, a.ldq, 0, a.M, 64, a.K);
    const int row = lane & 15, c = lane >> 4;
    const int wo = n0 + row < a.N ? (int)(row * a.ldw) + c * 16 : kOOB;
    int qo[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) qo[t] = t * 16 + row < a.M ? (int)((t * 16 + row) * a.ldq) + c * 16 : kOOB;
    i32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    // 128 bytes of k per wave and step, so that a step reads whole lines
    constexpr int U = MT <= 2 ? 4 : 2;
    const int stride = waves * 128;
    for (int k0 = wave * 128; k0 < a.K; k0 += stride * U) {
        uint4 wv[U][2], qv[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + u * stride + h * 64;
                const bool in = k + c * 16 < a.K;   // K is a multiple of 16
                wv[u][h] = load16(wr, in && wo != kOOB ? wo + k : kOOB);
#pragma unroll
                for (int t = 0; t < MT; ++t) qv[u][h][t] = load16(qr, in && qo[t] != kOOB ? qo[t] + k : kOOB);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[u][h]),
                                                                   __builtin_bit_cast(i32x4, qv[u][h][t]), acc[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) red[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * 64; e += blockDim.x) {
        i32x4 s = red[e];
        for (int k = 1; k < waves; ++k) s += red[k * MT * 64 + e];
        const int m = (e >> 6) * 16 + (e & 15), n = n0 + ((e & 63) >> 4) * 4;
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

constexpr int kStageK = 128;  // bytes of k per stage: one line of every row

// 16-byte slot of a stage's (row, 16-byte piece): the pieces of a row are
// permuted so that 16 consecutive rows read at one piece hit all banks.
__device__ __forceinline__ int slot_of(int row, int piece) { return row * 8 + (piece ^ ((row >> 1) & 7)); }

struct TileAt {
    int m0, n0, split;
};

// Block -> tile: every XCD walks a contiguous run (its L2 keeps the shared
// rows), and within it tiles go down groups of 8 row tiles, channel tile by
// channel tile.
__device__ __forceinline__ TileAt tile_at(int tm, int tn, int BM, int BN) {
    const int per = tm * tn;
    int i = xcd_tile_index();
    TileAt t;
    t.split = i / per;
    i %= per;
    constexpr int GM = 8;
    const int group = i / (GM * tn), first = group * GM, rows = min(GM, tm - first);
    i -= group * GM * tn;
    t.m0 = (first + i % rows) * BM;
    t.n0 = (i / rows) * BN;
    return t;
}

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

// Results of a wave's TI*16 channels x TJ*16 rows: block by block of 16 rows
// through the wave's own piece of LDS (16 x TI*16 elements), so that whole
// rows are written.  In the 16x16 result lane l holds, in register r, channel
// 4 (l >> 4) + r of row l & 15.  sw, sb: the tile's channel scales and biases
// in LDS, from the wave's first channel.  OUT int: the sums themselves.
template <int TI, int TJ, typename OUT>
__device__ __forceinline__ void write_results(const Int8Args& a, i32x4 (&acc)[TI][TJ], char* lds, const float* sw,
                                              const float* sb, int m0, int n0, OUT* y, long long ldy, bool vec) {
    constexpr bool kSums = std::is_same_v<OUT, int>;
    constexpr int COLS = TI * 16, ROW = COLS * (int)sizeof(OUT), PIECES = ROW / 16;
    constexpr int MASK = (PIECES < 16 ? PIECES : 16) - 1;
    const int lane = threadIdx.x & 63, r16 = lane & 15;
    char* const row = lds + r16 * ROW;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        float qs = 0.0f;
        if constexpr (!kSums) qs = m0 + j * 16 + r16 < a.M ? a.q_scale[m0 + j * 16 + r16] : 0.0f;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int c = i * 16 + 4 * (lane >> 4), b = c * (int)sizeof(OUT);
            char* const at = row + ((b / 16) ^ (r16 & MASK)) * 16 + b % 16;
            if constexpr (kSums) {
                *reinterpret_cast<i32x4*>(at) = acc[i][j];
            } else {
                const float4 ws = *reinterpret_cast<const float4*>(sw + c);
                const float4 bs = *reinterpret_cast<const float4*>(sb + c);
                const float v0 = finish(acc[i][j][0], qs * ws.x, bs.x, a.relu);
                const float v1 = finish(acc[i][j][1], qs * ws.y, bs.y, a.relu);
                const float v2 = finish(acc[i][j][2], qs * ws.z, bs.z, a.relu);
                const float v3 = finish(acc[i][j][3], qs * ws.w, bs.w, a.relu);
                if constexpr (sizeof(OUT) == 4)
                    *reinterpret_cast<float4*>(at) = make_float4(v0, v1, v2, v3);
                else
                    *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3));
            }
        }
        // the wave's own LDS: its writes are done before its reads
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (vec) {
#pragma unroll
            for (int it = 0; it < 16 * PIECES / 64; ++it) {
                const int e = it * 64 + lane, r = e / PIECES, p = e % PIECES;
                const int m = m0 + j * 16 + r, n = n0 + p * (16 / (int)sizeof(OUT));
                if (m < a.M && n < a.N)
                    *reinterpret_cast<uint4*>(y + m * ldy + n) =
                        *reinterpret_cast<const uint4*>(lds + r * ROW + (p ^ (r & MASK)) * 16);
            }
        } else {
            for (int e = lane; e < 16 * COLS; e += 64) {
                const int r = e / COLS, c = e % COLS, b = c * (int)sizeof(OUT);
                const int m = m0 + j * 16 + r, n = n0 + c;
                if (m < a.M && n < a.N)
                    y[m * ldy + n] = *reinterpret_cast<const OUT*>(lds + r * ROW + ((b / 16) ^ (r & MASK)) * 16 + b % 16);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// The tile's channel scales and biases into LDS (zero past the last channel).
template <int BN> __device__ __forceinline__ void stage_scales(const Int8Args& a, int n0, float* sw, float* sb) {
    for (int c = threadIdx.x; c < BN; c += blockDim.x) {
        sw[c] = n0 + c < a.N ? a.w_scale[n0 + c] : 0.0f;
        sb[c] = a.bias && n0 + c < a.N ? a.bias[n0 + c] : 0.0f;
    }
}

template <typename OUT> __device__ __forceinline__ OUT* out_of(const Int8Args& a, int split) {
    return static_cast<OUT*>(a.y) + (std::is_same_v<OUT, int> ? (long long)split * a.M * a.N : 0);
}

// A wave's copy of 1 KB into LDS, 16 bytes a lane: no registers, no LDS
// instruction; an offset outside the matrix writes zeros.
__device__ __forceinline__ void copy_kb(__amdgpu_buffer_rsrc_t r, char* dst, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)dst, 16, off, 0, 0, 0);
}

// Aligned operands.  Stage s + 2 is copied into the buffer that stage s has
// just been read from, a whole stage ahead of its use; the reads of a step
// are issued one step before its products, across the stages' border too, so
// there is one barrier per stage.
template <int BM, int BN, int WM, int WN, typename OUT>
__global__ __launch_bounds__(WM * WN * 64) void int8_tile_kernel(Int8Args a, int tm, int tn, int stages, bool vec) {
    constexpr int NW = WM * WN, TI = BN / WN / 16, TJ = BM / WM / 16;
    constexpr int STAGE = (BM + BN) * kStageK;
    constexpr int CW = BN / 8 / NW, CQ = BM / 8 / NW;   // 1 KB copies per wave and stage
    static_assert(CW * 8 * NW == BN && CQ * 8 * NW == BM, "copies split evenly");
    static_assert(NW * 16 * TI * 16 * 4 <= STAGE, "results fit a stage");
    __shared__ uint4 lds0[STAGE / 16], lds1[STAGE / 16];
    __shared__ float sw[BN], sb[BN];
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

    stage_scales<BN>(a, t.n0, sw, sb);
    {
        // every buffer a restrict argument of one function: the compiler then
        // does not make the reads of one wait for the copies into the other
        auto loop = [&](char* __restrict__ b0, char* __restrict__ b1) __attribute__((always_inline)) {
            I8_COPY(b0, 0);
            I8_COPY(b1, 1);
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
                               sw + wn * TI * 16, sb + wn * TI * 16, t.m0 + wm * TJ * 16, t.n0 + wn * TI * 16,
                               out_of<OUT>(a, t.split), a.ldy, vec);
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
__global__ __launch_bounds__(WM * WN * 64) void int8_ragged_kernel(Int8Args a, int tm, int tn, int stages, bool vec) {
    constexpr int NT = WM * WN * 64, TI = BN / WN / 16, TJ = BM / WM / 16;
    constexpr int STAGE = (BM + BN) * kStageK, PER = (BM + BN) * 8 / NT;
    static_assert(BN * 8 % NT == 0 && BM * 8 % NT == 0, "pieces split evenly");
    constexpr int OUTB = WM * WN * 16 * TI * 16 * 4;
    __shared__ uint4 lds[(STAGE > OUTB ? STAGE : OUTB) / 16];
    __shared__ float sw[BN], sb[BN];
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
    stage_scales<BN>(a, t.n0, sw, sb);
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
                               sw + wn * TI * 16, sb + wn * TI * 16, t.m0 + wm * TJ * 16, t.n0 + wn * TI * 16,
                               out_of<OUT>(a, t.split), a.ldy, vec);
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
        if (c < K) raw[j] = Vec<T, V>::load(p + c);
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
        if (c < K) store_quantised<V>(q + row * ldq + c, v[j], s.inv);
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
        Vec<T, V>::unpack(Vec<T, V>::load(p + c), v);
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
        Vec<T, V>::unpack(Vec<T, V>::load(p + c), v);
        store_quantised<V>(q + row * ldq + c, v, s.inv);
    }
    if (threadIdx.x == 0) scale[row] = s.scale;
}

template <typename T, int V>
hipError_t quantize(const void* x, void* q, float* scale, int M, int K, long long ldx, long long ldq, hipStream_t st) {
    const int cv = (K + V - 1) / V;
    int lpp = 1;
    while (lpp < cv && lpp < 64) lpp <<= 1;
    const int j = (cv + lpp - 1) / lpp;
    const T* xt = static_cast<const T*>(x);
    int8_t* qt = static_cast<int8_t*>(q);
    if (j > 4) {
        quantize_long_rows_kernel<T, V><<<M, 256, 0, st>>>(xt, qt, scale, K, ldx, ldq);
        return hipGetLastError();
    }
    const int per = 256 / lpp, blocks = (int)(((long long)M + per - 1) / per);
    auto k = j == 1 ? quantize_rows_kernel<T, V, 1> : j == 2 ? quantize_rows_kernel<T, V, 2> : quantize_rows_kernel<T, V, 4>;
    k<<<blocks, 256, 0, st>>>(xt, qt, scale, M, K, ldx, ldq, lpp);
    return hipGetLastError();
}

// ------------------------------------------------------------------ host

bool aligned_operands(const Int8Args& a) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    return a.K % 16 == 0 && a.ldq % 16 == 0 && a.ldw % 16 == 0 && al(a.q) && al(a.w);
}

enum { kSkinny, kTile256, kTile128, kTile64, kRagged128, kRagged64 };

struct Int8Plan {
    int kernel, bm, bn, tm, tn, splits, stages;
};

// Rows up to kSkinnyRows read the weights once whatever the tile, so the
// skinny kernel, which does nothing else, takes them.  Larger products take
// the largest tile that still gives every compute unit one; few tiles of a
// long k are split along it until they do.
constexpr int kSkinnyRows = 64;
constexpr int kUnits = 256;

Int8Plan make_int8_plan(int M, int K, int N, bool aligned) {
    Int8Plan p;
    auto tiles = [&](int b) { return (long long)((M + b - 1) / b) * ((N + b - 1) / b); };
    if (aligned && M <= kSkinnyRows) {
        p.kernel = kSkinny;
        p.bm = kSkinnyRows;
        p.bn = 16;
    } else {
        const int b = aligned && tiles(256) >= kUnits ? 256 : tiles(128) >= kUnits ? 128 : 64;
        p.kernel = aligned ? (b == 256 ? kTile256 : b == 128 ? kTile128 : kTile64) : b == 128 ? kRagged128 : kRagged64;
        p.bm = p.bn = b;
    }
    p.tm = (M + p.bm - 1) / p.bm;
    p.tn = (N + p.bn - 1) / p.bn;
    const int all = (K + kStageK - 1) / kStageK;
    p.splits = 1;
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

template <typename OUT> hipError_t skinny(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
    // waves that split k: 4 where the channels alone fill the chip, else up
    // to 16, of at least 128 bytes of k each
    int waves = 4;
    while (waves < 16 && p.tn * waves < 8 * kUnits && waves * 2 * 128 <= a.K) waves *= 2;
    if (a.M <= 16) int8_skinny_kernel<1, OUT><<<p.tn, waves * 64, waves * 1024, st>>>(a);
    else if (a.M <= 32) int8_skinny_kernel<2, OUT><<<p.tn, waves * 64, waves * 2048, st>>>(a);
    else int8_skinny_kernel<4, OUT><<<p.tn, waves * 64, waves * 4096, st>>>(a);
    return hipGetLastError();
}

template <typename OUT> hipError_t tiled(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
    const int es = (int)sizeof(OUT);
    const bool vec = a.ldy * es % 16 == 0 && a.N * (long long)es % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
    const int blocks = p.tm * p.tn * p.splits;
    switch (p.kernel) {
    case kTile256: int8_tile_kernel<256, 256, 2, 4, OUT><<<blocks, 512, 0, st>>>(a, p.tm, p.tn, p.stages, vec); break;
    case kTile128: int8_tile_kernel<128, 128, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages, vec); break;
    case kTile64: int8_tile_kernel<64, 64, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages, vec); break;
    case kRagged128: int8_ragged_kernel<128, 128, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages, vec); break;
    default: int8_ragged_kernel<64, 64, 2, 2, OUT><<<blocks, 256, 0, st>>>(a, p.tm, p.tn, p.stages, vec); break;
    }
    return hipGetLastError();
}

size_t split_bytes(const Int8Plan& p, int M, int N) {
    return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

}  // namespace

// One figure for either alignment.
size_t int8_matmul_workspace(int M, int K, int N) {
    const size_t u = split_bytes(make_int8_plan(M, K, N, false), M, N);
    const size_t v = K % 16 ? 0 : split_bytes(make_int8_plan(M, K, N, true), M, N);
    return u > v ? u : v;
}

bool int8_matmul_supports(int M, int K, int N, long long ldq, long long ldw) {
    // sums stay below 2^31; a tile's rows are addressed with 31 bits; the grid
    if (K > 131071 || ldq > (1 << 22) || ldw > (1 << 22)) return false;
    for (int al = 0; al < 2; ++al) {
        const Int8Plan p = make_int8_plan(M, K, N, al);
        if ((long long)p.tm * p.tn * p.splits >= 0x7fffffffLL) return false;
    }
    return true;
}

hipError_t launch_int8_matmul(const Int8Args& a, int out_f32, void* ws, hipStream_t st) {
    const Int8Plan p = make_int8_plan(a.M, a.K, a.N, aligned_operands(a));
    if (p.kernel == kSkinny) return out_f32 ? skinny<float>(a, p, st) : skinny<bf16_t>(a, p, st);
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
    const int es = dtype == 0 /* CONV2D_F32 */ ? 4 : 2;
    int v = 16 / es;
    while (v > 1 && !(K % v == 0 && ldx % v == 0 && ldq % v == 0 &&
                      (reinterpret_cast<uintptr_t>(x) & (v * es - 1)) == 0 &&
                      (reinterpret_cast<uintptr_t>(q) & (v - 1)) == 0))
        v >>= 1;
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
