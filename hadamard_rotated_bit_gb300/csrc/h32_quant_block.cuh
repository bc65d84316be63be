// One 32-block of activations in a thread's registers (sm_103a): loading, rotating,
// rounding to integer codes and packing them, as the activation quantizers do it.  The
// norm that quantizes its output holds half a block a lane and has its own forms of
// these steps, with the same bits; it shares the rotate argument, the codes of
// degenerate blocks and the byte packing.
#pragma once

#include <stdint.h>

#include "h32_tcform.cuh"

namespace h32 {

// ----------------------------------------------------------------------------
// loading one block as 32 fp32 values
// ----------------------------------------------------------------------------
__device__ __forceinline__ void load_block_bf16(const uint16_t *__restrict__ p, float (&v)[32]) {
    const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 u = __ldg(q + c);
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * c + 2 * i] = __uint_as_float(w[i] << 16);
            v[8 * c + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ void load_block_f32(const float *__restrict__ p, float (&v)[32]) {
    const float4 *q = reinterpret_cast<const float4 *>(p);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float4 f = __ldg(q + c);
        v[4 * c] = f.x;
        v[4 * c + 1] = f.y;
        v[4 * c + 2] = f.z;
        v[4 * c + 3] = f.w;
    }
}

// ----------------------------------------------------------------------------
// the rotation: butterfly with strides 1, 2, 4, 8, 16, then the 1/sqrt(32) scale
// ----------------------------------------------------------------------------
// The kRot-point rotation (0 = none, 32, 64, 128) of the thread's 32-block,
// which is 32-block `pos` (0 .. kRot/32 - 1) of its kRot-block.  The other
// 32-blocks of the kRot-block are held by the lanes that differ from this one
// in the low bits pos covers (lane ^ 1, lane ^ 2); those lanes are in `mask`.
// Strides 32 and 64 pair element i of two blocks: the lower block takes
// a + c, the upper a - c (a the lower block's value), as in strides 1..16.
template <int kRot>
__device__ __forceinline__ void rotate_block(float (&v)[32], uint32_t pos, unsigned mask) {
    if constexpr (kRot == 32) {
        rotate32(v);
    } else if constexpr (kRot > 32) {
        butterfly32(v);
#pragma unroll
        for (int hb = 1; hb < kRot / 32; hb <<= 1) {
            const bool lower = (pos & hb) == 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float c = __shfl_xor_sync(mask, v[i], hb);
                v[i] = lower ? __fadd_rn(v[i], c) : __fsub_rn(c, v[i]);
            }
        }
        const float sc = (kRot == 64) ? 0.125f : kInvSqrt128;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(v[i], sc);
    }
}

// the rotate argument of the entry points: 0 = none, 1 or 32, 64, 128 points
// (-1 = not supported)
inline int rot_points(int rotate) {
    return rotate == 0 ? 0 : rotate == 1 || rotate == 32 ? 32 : rotate == 64 ? 64
         : rotate == 128 ? 128 : -1;
}

// low byte of each of four words -> one word
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __byte_perm(a, b, 0x0040);
    const uint32_t cd = __byte_perm(c, d, 0x0040);
    return __byte_perm(ab, cd, 0x5410);
}

// ----------------------------------------------------------------------------
// rounding a block to codes
// ----------------------------------------------------------------------------
// d = amax / qmax (IEEE divide); bits[i] holds the code round-half-even(v * fl(1/d))
// plus 1.5 * 2^23 as a float, for kN of the block's values.  With a finite amax and
// a finite 1/d every product lies in [-qmax, qmax] up to rounding; when 1/d
// overflowed (a block of subnormal size) or the rotation itself overflowed to
// +-inf, the code is the clamped v / d instead.  Returns d.
template <int kBits, int kN>
__device__ __forceinline__ float quant_bits(const float (&v)[kN], float amax, uint32_t (&bits)[kN]) {
    constexpr float kQmax = (kBits == 4) ? 7.0f : 127.0f;
    constexpr float kQmin = (kBits == 4) ? -8.0f : -127.0f;
    const float d = __fdiv_rn(amax, kQmax);
    const float id = (d != 0.0f) ? __frcp_rn(d) : 0.0f;
    if (!(amax < INFINITY) || isinf(id)) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            bits[i] = __float_as_uint(__fadd_rn(degenerate_code(v[i], d, kQmin, kQmax),
                                                kRoundMagic));
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            bits[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], id), kRoundMagic));
    }
    return d;
}

// the whole block of one thread
template <int kBits>
__device__ __forceinline__ float quant_block_bits(const float (&v)[32], uint32_t (&bits)[32]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
    return quant_bits<kBits>(v, amax, bits);
}

// 4-bit codes in Q4_0 nibble order: byte j = element j (low) | element j + 16 (high)
__device__ __forceinline__ void pack_q4(const uint32_t (&bits)[32], uint32_t (&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo =
            pack_low_bytes(bits[4 * k], bits[4 * k + 1], bits[4 * k + 2], bits[4 * k + 3]);
        const uint32_t hi = pack_low_bytes(bits[16 + 4 * k], bits[17 + 4 * k], bits[18 + 4 * k],
                                           bits[19 + 4 * k]);
        w[k] = (lo & 0x0F0F0F0Fu) | ((hi << 4) & 0xF0F0F0F0u);
    }
}

// 8-bit codes in element order
__device__ __forceinline__ void pack_q8(const uint32_t (&bits)[32], uint32_t (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        w[k] = pack_low_bytes(bits[4 * k], bits[4 * k + 1], bits[4 * k + 2], bits[4 * k + 3]);
}

// 8-bit codes in tensor-core form: the bytes of 16 h, and the bytes of l
// (integer byte arithmetic: measured faster than converting floats)
__device__ __forceinline__ void pack_q8_tc(const uint32_t (&bits)[32], uint32_t (&wh)[8],
                                           uint32_t (&wl)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        tc_bytes_q8(pack_low_bytes(bits[4 * k], bits[4 * k + 1], bits[4 * k + 2], bits[4 * k + 3]),
                    wh[k], wl[k]);
}

}  // namespace h32
