// matmul_plan.hpp -- what the host decides for a product of rows from its sizes: the
// tiles and the parts of the sum, the form for few rows, which operands are copied
// first, and the shape of the pass that makes dz.  Plain C++, no device code.
#pragma once

#include <cstddef>

namespace conv2d {

constexpr int kStageBytes = 128;   // of the summed index, in a stage of the tiles
constexpr int kUnits = 256;        // compute units

struct Plan {
    int b, tm, tn, splits, stages;   // square tiles of b
};

// The largest tile that still gives every compute unit one and that the columns
// fill.  256, of aligned operands only, has the compute unit to itself, so its
// results leave while nothing else is done: two workgroups of 128 are faster where s
// is short (16384 x 1024 -> 4096 bf16 with a residual 185 us against 192, x 128 93
// against 116; but 16384 x 2048 -> 1024 78 against 70).
//
// Few tiles are split along s until every compute unit has two, three of 64 where a
// part is still 16 stages long.  A part of 128 is at least 16 stages: 256 x 4096 -> 4096
// takes 27 us in 8 parts of 128 and 46 in tiles of 64, but 2048 x 1024 -> 1024 18 in parts
// of 8 stages and 11 in tiles of 64.  A part of 64 is at least 4 (dw of 100352 x 256 -> 64:
// 22.7 us with two a unit, 27.7 with one; 64 x 4096 -> 16384: 52 us with one, 41 with two,
// 36 with three; but 1024 x 512 -> 1024, one a unit already, 6.9 whole and 11.2 in two).
constexpr int kLongBytes = 2048;

inline Plan make_plan(int rows, int cols, int K, int es, bool aligned) {
    auto tiles = [&](int b) { return (long long)((rows + b - 1) / b) * ((cols + b - 1) / b); };
    const int all = (int)(((long long)K * es + kStageBytes - 1) / kStageBytes);
    auto parts = [&](int stages) { return all / stages > 1 ? all / stages : 1; };
    Plan p;
    const bool large = aligned && (long long)K * es > kLongBytes && cols > 128 && rows > 128 && tiles(256) >= kUnits;
    p.b = large ? 256 : cols > 64 && rows > 64 && tiles(128) * parts(16) >= kUnits ? 128 : 64;
    p.tm = (rows + p.b - 1) / p.b;
    p.tn = (cols + p.b - 1) / p.b;
    const long long t = (long long)p.tm * p.tn;
    auto split = [&](int units, int stages) { return (int)(units / t < parts(stages) ? units / t : parts(stages)); };
    p.splits = 1;
    if (t < kUnits) p.splits = split(2 * kUnits, p.b == 64 ? 4 : 16);
    if (p.b == 64 && split(3 * kUnits, 16) > p.splits) p.splits = split(3 * kUnits, 16);
    p.stages = (all + p.splits - 1) / p.splits;
    p.splits = (all + p.stages - 1) / p.stages;
    return p;
}

// One figure for either alignment.
inline size_t split_bytes(int rows, int cols, int K, int es) {
    const Plan u = make_plan(rows, cols, K, es, false), v = make_plan(rows, cols, K, es, true);
    const int splits = u.splits > v.splits ? u.splits : v.splits;
    return splits > 1 ? (size_t)splits * rows * cols * 4 : 0;
}

inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Elements of a row in whole 16-byte pieces.
inline int whole_pieces(int n, int es) { return (n + 16 / es - 1) / (16 / es) * (16 / es); }

// Whether a product is large enough for copies of its operands with whole pieces: the
// tiles of aligned operands then save more than the copies take (bf16 with copies and
// without: 4096 x 4095 -> 4096 133 and 230 us, 2048 x 2047 -> 2048 38 and 47, gradients of
// 4096 x 1001 -> 2001 91 and 201; fp32 is bound by its products sooner).
inline bool worth_copies(int M, int K, int N, int es) { return (double)M * N * K * (es == 4 ? 8 : 1) >= 0x1p32; }

// Whether rows of K elements are copied (by K alone: a whole K at other strides or
// addresses is read as it lies): for two products (the gradients), or for one
// that uses an operand's elements often enough (24266 x 2092 -> 367 121 and 97 us).
inline bool packs(int M, int K, int N, int es) { return (long long)K * es % 16 != 0 && worth_copies(M, K, N, es); }
inline bool packs_forward(int M, int K, int N, int es) { return packs(M, K, N, es) && (double)M * N >= 500.0 * ((double)M + N); }

struct DzShape {
    int lanes, chunk, cols, chunks;
};

inline DzShape dz_shape(int M, int N, int es) {
    DzShape d;
    const int vecs = (N + 16 / es - 1) / (16 / es);
    d.lanes = 1;
    while (d.lanes < 64 && d.lanes < vecs) d.lanes <<= 1;
    d.cols = (vecs + d.lanes - 1) / d.lanes;
    // 8 workgroups a compute unit, and up to 512 rows a thread, which sums them in fp32
    const int groups = 256 / d.lanes;
    long long chunks = (8 * kUnits + d.cols - 1) / d.cols, least = ((long long)M + groups * 512 - 1) / (groups * 512);
    const long long most = ((long long)M + groups * 4 - 1) / (groups * 4);
    if (chunks > most) chunks = most;
    if (chunks < least) chunks = least;
    if (chunks > 65535) chunks = 65535;
    d.chunk = (int)(((long long)M + chunks - 1) / chunks);
    d.chunks = (int)(((long long)M + d.chunk - 1) / d.chunk);
    return d;
}

struct SkinnyShape {
    bool fits, two, pairs;   // two blocks of 16 rows; two of 16 columns
    int waves;
    long long steps;         // of 128 bytes of s, for a wave
};

// Up to 32 rows read the weights once whatever the tile.  Waves that split s: 4, or up
// to 16 where that leaves the chip few, of at least 128 bytes each.  Two blocks of
// columns use a row's values twice, where half the workgroups still fill the chip.  Few
// columns with a long s do not: they are split along s over workgroups instead (bf16,
// skinny and tiled: 1 x 8192 -> 1024 11.7 and 10.3 us, 1 x 16384 -> 256 20.3 and 9.8, 20 x
// 4096 -> 1024 11.9 and 9.5; but 1 x 4096 -> 1024 7.4 and 8.9, 1 x 8192 -> 2048 12.2 and
// 13.4, 20 x 1024 -> 1024 5.6 and 8.0).
inline SkinnyShape skinny_shape(int rows, int cols, int K, int es) {
    SkinnyShape k;
    k.two = rows > 16;
    k.pairs = k.two && cols >= 32 * kUnits;
    const int blocks = (int)(((long long)cols + (k.pairs ? 31 : 15)) / (k.pairs ? 32 : 16));
    const long long bytes = (long long)K * es;
    k.waves = 4;
    while (k.waves < 16 && (long long)blocks * k.waves < 16 * kUnits && k.waves * 2 * kStageBytes <= bytes) k.waves *= 2;
    k.steps = (bytes + k.waves * kStageBytes - 1) / (k.waves * kStageBytes);
    // (a launch counts its threads in 32 bits)
    k.fits = rows <= 32 && cols <= 1 << 27 && !(blocks <= (rows > 8 ? 128 : 64) && k.steps >= (k.two ? 4 : 8));
    return k;
}

}  // namespace conv2d
