// rowvec.hpp -- device helpers shared by the group-norm and the int8 kernels:
// vector loads of V fp32 or bf16 elements, the activations and the
// quantisation of a row to 8 bits.
#pragma once

#include "common.hpp"

namespace conv2d {

// V consecutive elements of T in one load or store of V * sizeof(T) bytes
// (2, 4, 8 or 16), aligned to one element at least.
template <int BYTES> struct RawBytes;
template <> struct RawBytes<16> { typedef uint4 type; };
template <> struct RawBytes<8> { typedef uint2 type; };
template <> struct RawBytes<4> { typedef uint32_t type; };
template <> struct RawBytes<2> { typedef uint16_t type; };
template <> struct RawBytes<1> { typedef uint8_t type; };

template <typename T, int V> struct Vec;

// One access of any alignment.
template <int BYTES> __device__ __forceinline__ typename RawBytes<BYTES>::type load_bytes(const void* p) {
    typename RawBytes<BYTES>::type v;
    __builtin_memcpy(&v, p, BYTES);
    return v;
}
template <int BYTES> __device__ __forceinline__ void store_bytes(void* p, const typename RawBytes<BYTES>::type& v) {
    __builtin_memcpy(p, &v, BYTES);
}

// Where the vector of a row of C elements from element c on starts: the last one of a row
// that is no multiple of V ends with the row and covers part of the one before
// (whoever writes both writes the same values twice).
template <int V> __device__ __forceinline__ int vector_start(int c, int C) { return min(c, C - V); }

template <int V> struct Vec<float, V> {
    typedef typename RawBytes<4 * V>::type raw;
    static __device__ __forceinline__ raw load(const float* p) { return load_bytes<4 * V>(p); }
    static __device__ __forceinline__ void unpack(const raw& r, float (&v)[V]) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = __uint_as_float(w[j]);
    }
    static __device__ __forceinline__ raw pack(const float (&v)[V]) {
        raw r;
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = __float_as_uint(v[j]);
        return r;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[V]) { store_bytes<4 * V>(p, pack(v)); }
};

template <int V> struct Vec<bf16_t, V> {
    typedef typename RawBytes<2 * V>::type raw;
    static __device__ __forceinline__ raw load(const bf16_t* p) { return load_bytes<2 * V>(p); }
    static __device__ __forceinline__ void unpack(const raw& r, float (&v)[V]) {
        if constexpr (V == 1) {
            v[0] = bf16_to_f32(r);
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
    // one rounding, to nearest even
    static __device__ __forceinline__ raw pack(const float (&v)[V]) {
        if constexpr (V == 1) {
            return f32_to_bf16(v[0]);
        } else {
            raw r;
            uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
            return r;
        }
    }
    static __device__ __forceinline__ void store(bf16_t* p, const float (&v)[V]) { store_bytes<2 * V>(p, pack(v)); }
};

// 1 / (1 + exp(-z)) from the hardware's exp2 and reciprocal (1 ulp each).
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

enum { kActNone = 0, kActRelu = 1, kActSilu = 2 };

// ReLU by comparison: a NaN stays a NaN.
template <int ACT> __device__ __forceinline__ float activate(float z) {
    if (ACT == kActRelu) return z < 0.0f ? 0.0f : z;
    if (ACT == kActSilu) return z * sigmoid(z);
    return z;
}

// One step of a reduction over neighbouring lanes: the value of a lane of the
// other half of a group of 2, 4, 8, 16, 32 or 64 lanes, where both halves
// already hold one value each (so a mirrored lane serves as well as the
// exchanged one).  Register moves only; no LDS.
template <int STEP> __device__ __forceinline__ uint32_t other_half(uint32_t v) {
    if constexpr (STEP == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, false);        // quad_perm 1 0 3 2
    else if constexpr (STEP == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, false);   // quad_perm 2 3 0 1
    else if constexpr (STEP == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, false);  // row_half_mirror
    else return __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, false);                           // row_mirror
}
// The last two steps exchange whole rows of 16 (or halves of 32) lanes: both
// sides come back, in the order (lower, upper) on every lane.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2_t rows_of_16(uint32_t v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); }
__device__ __forceinline__ u32x2_t halves_of_32(uint32_t v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); }

// Sum (or unsigned maximum) over L consecutive lanes, L a power of two <= 64
// and the same on every lane; every lane gets the result.
template <typename OP> __device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, int L, OP op) {
    if (L > 1) v = op(v, other_half<1>(v));
    if (L > 2) v = op(v, other_half<2>(v));
    if (L > 4) v = op(v, other_half<4>(v));
    if (L > 8) v = op(v, other_half<8>(v));
    if (L > 16) {
        const u32x2_t p = rows_of_16(v);
        v = op(p.x, p.y);
    }
    if (L > 32) {
        const u32x2_t p = halves_of_32(v);
        v = op(p.x, p.y);
    }
    return v;
}
__device__ __forceinline__ float lanes_sum(float v, int L) {
    return __uint_as_float(lanes_reduce(__float_as_uint(v), L, [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
// The same in fp64, for L on every lane of the wave: the two halves of a value
// move side by side.
__device__ __forceinline__ double lanes_sum(double v, int L) {
    const auto join = [](uint32_t lo, uint32_t hi) {
        return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
    };
    const auto lo = [&] { return (uint32_t)__builtin_bit_cast(unsigned long long, v); };
    const auto hi = [&] { return (uint32_t)(__builtin_bit_cast(unsigned long long, v) >> 32); };
    if (L > 1) v += join(other_half<1>(lo()), other_half<1>(hi()));
    if (L > 2) v += join(other_half<2>(lo()), other_half<2>(hi()));
    if (L > 4) v += join(other_half<4>(lo()), other_half<4>(hi()));
    if (L > 8) v += join(other_half<8>(lo()), other_half<8>(hi()));
    if (L > 16) {
        const u32x2_t p = rows_of_16(lo()), q = rows_of_16(hi());
        v = join(p.x, q.x) + join(p.y, q.y);
    }
    if (L > 32) {
        const u32x2_t p = halves_of_32(lo()), q = halves_of_32(hi());
        v = join(p.x, q.x) + join(p.y, q.y);
    }
    return v;
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int L) {
    return lanes_reduce(v, L, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// ---- a row in 8 bits: a = max(max |v|, 2^-100), q = round(v * (127 / a)),
// scale = a / 127.  The maximum is taken over the bit patterns of |v|, whose
// order is that of the values with infinities and NaN above all: a row that
// holds one of them gets scale NaN and q = 0, so that every product with it
// is NaN.
constexpr uint32_t kInfBits = 0x7f800000u;

struct RowScale {
    float inv;    // 127 / a (0: the row is not finite)
    float scale;  // a / 127
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
    if (amax_bits >= kInfBits) return {0.0f, __uint_as_float(0x7fc00000u)};
    const float a = fmaxf(__uint_as_float(amax_bits), 0x1p-100f);
    return {127.0f / a, a / 127.0f};
}

// The rounded value's low byte, by adding 1.5 * 2^23: the product is rounded
// to fp32 first (no fused multiply-add), then the sum's rounding to integers
// is to nearest even.  In a row that is not finite (inv = 0) the product may
// be NaN: store_quantised writes 0 there.
__device__ __forceinline__ uint32_t quant_bits(float v, float inv) {
#pragma clang fp contract(off)
    const float p = v * inv;
    return __float_as_uint(p + 12582912.0f);
}

template <int V>
__device__ __forceinline__ void store_quantised(int8_t* q, const float (&v)[V], float inv) {
    typedef typename RawBytes<V>::type raw;
    uint32_t b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = quant_bits(v[j], inv);
    raw r;
    if constexpr (V >= 4) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const uint32_t lo = __builtin_amdgcn_perm(b[4 * j + 1], b[4 * j], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[4 * j + 3], b[4 * j + 2], 0x04000c0cu);
            w[j] = inv == 0.0f ? 0u : (lo | hi);
        }
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) w |= (b[j] & 0xffu) << (8 * j);
        r = (raw)(inv == 0.0f ? 0u : w);
    }
    store_bytes<V>(q, r);
}

}  // namespace conv2d
