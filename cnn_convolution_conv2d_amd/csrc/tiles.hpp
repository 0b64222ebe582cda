// tiles.hpp -- device helpers shared by the tiled products (8-bit integers, bf16
// and fp32): the stages' layout in LDS, copies into it and the order of the tiles.
#pragma once

#include "mfma.hpp"
#include "rowvec.hpp"

namespace conv2d {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_unaligned __attribute__((aligned(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

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

// The wave's accesses to its own piece of LDS before this are done before
// those after it.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's copy of 1 KB into LDS, 16 bytes a lane: no registers, no LDS
// instruction; an offset outside the matrix writes zeros.
__device__ __forceinline__ void copy_kb(__amdgpu_buffer_rsrc_t r, char* dst, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)dst, 16, off, 0, 0, 0);
}

}  // namespace conv2d
