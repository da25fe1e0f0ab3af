// mfma_tiles.h -- the bf16 matrix instruction (16 x 16 x 32) and its operands: values split into
// bf16 parts, LDS tiles in 16-byte pieces, reads along rows and transposing reads down rows.
//
// Layouts: A lane (row li, k 8 g4 ..), B lane (column li, k 8 g4 ..), result lane (column li, rows
// 4 g4 ..), li = lane % 16, g4 = lane / 16.  A result whose rows are the next product's contraction
// is that product's operand as it stands, with k running 4 g4 + e over one 16-row tile and
// 16 + 4 g4 + e over the next ("token order" below).
#pragma once

#include "internal.h"

namespace ssm {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4any __attribute__((ext_vector_type(4), aligned(2)));  // any bf16 address
typedef uint32_t u2any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4 mfma(bf8 a, bf8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// v = sum of its parts in bf16, each the rounded rest: PARTS = 3 leaves nothing of 24 bits
template <int PARTS>
__device__ __forceinline__ void split(const float (&v)[8], bf8 (&part)[PARTS]) {
    u4 w[PARTS];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            const uint32_t q = pack_bf16x2(a, b);
            w[k][i] = q;
            if (k + 1 < PARTS) {
                a -= __uint_as_float(q << 16);
                b -= __uint_as_float(q & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k) part[k] = __builtin_bit_cast(bf8, w[k]);
}

// LDS tiles of bf16: rows of RB bytes in 16-byte pieces, the piece index XORed with sw(row), so
// that over the 64 banks (256 bytes) fall apart: the equal pieces of 16 rows (operand reads along
// rows), and the neighbouring pairs of pieces of the 8 rows that two 16-lane groups of a
// transposing read take (0-7 and 8-15 in token order, 0-3 with 8-11 and 4-7 with 12-15 else).
template <int RB>
__device__ __forceinline__ int sw(int row) {
    const int b0 = row & 1, b1 = (row >> 1) & 1, b2 = (row >> 2) & 1, b3 = (row >> 3) & 1;
    if (RB == 128) return b1 << 2 | (b2 ^ b3) << 1 | b3;  // neighbouring rows lie 128 bytes apart
    return b0 << 3 | b1 << 2 | (b2 ^ b3) << 1 | b3;
}
template <int RB>
__device__ __forceinline__ int piece(int row, int q) { return row * RB + ((q ^ sw<RB>(row)) << 4); }

template <class T>
__device__ __forceinline__ T lds(const uint8_t* p) { return *reinterpret_cast<const T*>(p); }

// operand read along rows: row r0 + li, k = 32 kk + 8 g4 ..
template <int RB>
__device__ __forceinline__ bf8 along(const uint8_t* tile, int lane_off, int r0, int kk) {
    return lds<bf8>(tile + r0 * RB + (lane_off ^ (kk << 6)));
}
template <int RB>
__device__ __forceinline__ int along_off(int li, int g4) { return piece<RB>(li, g4); }

__device__ __forceinline__ s4 tr_read(const uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s4*)const_cast<uint8_t*>(p));
}
// lane offset of a transposing read of rows r .. r + 3 (r = 4 x group) and columns 0 .. 15
template <int RB>
__device__ __forceinline__ int down_off(int r, int li) {
    const int row = r + (li >> 2);
    return piece<RB>(row, (li & 3) >> 1) + 8 * (li & 1);
}
__device__ __forceinline__ bf8 join(s4 a, s4 b) {
    const u2 x = __builtin_bit_cast(u2, a), y = __builtin_bit_cast(u2, b);
    return __builtin_bit_cast(bf8, u4{x[0], x[1], y[0], y[1]});
}
// operand read down rows in token order: rows r0 + 4 g4 .. and r0 + 16 + 4 g4 .. (r0 = 32 x), of
// columns 16 c ..
template <int RB>
__device__ __forceinline__ bf8 down(const uint8_t* tile, int lane_off, int r0, int c) {
    const uint8_t* p = tile + r0 * RB + (lane_off ^ (c << 5));
    return join(tr_read(p), tr_read(p + 16 * RB));
}

// Sums over the 16 lanes that share g4, of four values at once: lane li holds that of v[li % 4].
__device__ __forceinline__ float row_sums(const float (&v)[4], int li) {
    const float k01 = li & 1 ? v[1] : v[0], s01 = li & 1 ? v[0] : v[1];
    const float k23 = li & 1 ? v[3] : v[2], s23 = li & 1 ? v[2] : v[3];
    const float a = k01 + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s01), 0xB1, 0xf, 0xf, true));
    const float b = k23 + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s23), 0xB1, 0xf, 0xf, true));
    const float k = li & 2 ? b : a, o = li & 2 ? a : b;
    float r = k + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(o), 0x4E, 0xf, 0xf, true));
    r += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(r), 0x124, 0xf, 0xf, true));         // rotated by 4
    return r + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(r), 0x128, 0xf, 0xf, true));   // by 8
}
// Makes an offset opaque: what is derived from it is computed where it is used instead of being
// kept in registers over the whole loop over the heads.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

}  // namespace
}  // namespace ssm
