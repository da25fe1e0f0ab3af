// scan_bwd_mfma.hip -- the complete backward of the selective scan on the bf16 matrix cores:
// bf16 activations, headdim 64, dstate 64 or 128 (the formulas stand in scan_bwd.hip).
//
// Chunks of Q = 128 tokens: the states before the chunks and the gradients after them are 8 N
// bytes a channel and chunk, written once and read once, and are the larger part of the
// traffic; twice the chunk halves them and costs only more pairs within the chunk.
//
//   sbf_decay   one pass over dt: for each head and chunk the sums of log2 a in double, kept as
//               hi + lo floats, f_t, e_t, dt_t and f_last
//   sbf_states  S and G, one block a row, head and direction walking over the chunks with the
//               state in accumulators (or, where those are too few blocks, one block a chunk,
//               joined along the row by sbf_pass)
//   sbf_dc      one block a chunk, group and range of its heads: dy against S, dC's part from
//               before the chunk in accumulators over the heads, and u
//   sbf_grad    one block a chunk, group and range of its heads: everything else.  B and the
//               pairs' C B^T stay in LDS for all heads; the sums over heads of L dt (dy x^T),
//               from which dB and dC take their pairs, stay in registers, and dB in accumulators:
//               the heads are summed without traffic.  Ranges of heads are joined by sbf_join.
//   sbf_anchor  f_last <G, S> of every eighth chunk; sb_ddt has the others from
//               f<G, S> of c = f<G, S> of c + 1 + sum of u of c + 1 - sum of v of c
//               (both sides plus sum of v are <G_c, S_{c+1}>), so S and G are not read a second
//               time; the rounding errors of eight chunks at most add up, and where f <G, S> is
//               far below u and v, |G| |S| f bounds it and with it the error
// One kernel for dC and the rest together read S, G and dy once, but held 300 registers a lane:
// at two wavefronts a SIMD (LDS) it spilled, and took 2318 us at 4 x 8192 tokens x 64 heads,
// dstate 128, where the two take 168 + 515 us.
//
// Operands: x, dy, B and C are exact in bf16.  Every fp32 operand (S, G, the scaled x and dy of
// sbf_states, the pairs of dx, the heads' summed pairs of dB and dC) is taken in three bf16 parts: 24
// bits, nothing lost.  Two parts (2^-17 of the operand) for those that only bf16 outputs depend on
// put 16 times as many of dx, dB and dC on the neighbour of the bf16 value that fp32 products give
// (1.5 in a thousand at 4 x 8192 tokens x 64 heads, now 0.1), and took 1043 us where this takes 1081.
//
// Layouts of the 16 x 16 x 32 instruction: A lane (row li, k 8 g4 ..), B lane (column li, k
// 8 g4 ..), result lane (column li, rows 4 g4 ..), li = lane % 16, g4 = lane / 16.  A result
// whose rows are the next product's contraction is that product's operand as it stands, with
// k running 4 g4 + e over one 16-row tile and 16 + 4 g4 + e over the next ("token order"
// below); the transposing LDS read (4 rows of 16 columns a 16-lane group) gives the other
// operand in the same order.  So pairs never pass through LDS.
#include <type_traits>

#include "internal.h"

namespace ssm {
namespace {

constexpr int kFQ = 128;
constexpr int kFP = 64;

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

__device__ __forceinline__ float lane_sum16(float v) {  // over the 16 lanes that share g4
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));   // i ^ 1
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));   // i ^ 2
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));  // half mirror
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));  // mirror
    return v;
}
__device__ __forceinline__ float group_sum4(float v) {  // over the four lanes that share li
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Sums over the four lanes that share li, of four values at once: rows of 16 lanes 0, 1, 2, 3 of
// the result hold the sums of a, c, b, d.
__device__ __forceinline__ float group_sums(float a, float b, float c, float d) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(c), __float_as_uint(d), false, false);
    const float ab = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const float cd = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(ab), __float_as_uint(cd), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ int group_of_row(int row) { return row == 1 ? 2 : row == 2 ? 1 : row; }
// Of the tile's W on rows 4 g4 + e, column li (0 on and above the diagonal): the column's sums
// from row 4 g4 + e on where that lies below the diagonal.  Summed over the columns they are the W
// that span a token, without a difference of row and column sums: that kept the rounding of every
// pair for all 16 tokens, eight times what dA of a fast head is made of.
__device__ __forceinline__ void spanning(float (&w)[4], int li, int g4) {
    const int d = li - 4 * g4;
    w[2] += w[3];
    w[1] += w[2];
    w[0] += w[1];
    const uint32_t t = __float_as_uint(w[0]);
    const auto p = __builtin_amdgcn_permlane16_swap(t, t, false, false);  // rows 0 0 2 2 and 1 1 3 3
    const float even = __uint_as_float(p[0]), odd = __uint_as_float(p[1]);
    const uint32_t two = __float_as_uint(even + odd);
    const auto q = __builtin_amdgcn_permlane32_swap(two, two, false, false);
    const float later = (g4 & 1 ? 0.0f : odd) + (g4 & 2 ? 0.0f : __uint_as_float(q[1]));
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = e > d ? w[e] + later : 0.0f;
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
// Sum of squares of a lane's 16 values, times 4^kNormExp, and never below it: a square of what is under
// 2^-95 may be rounded to 0 (each by less than 2^-126), which the rest makes up for.  The gradients
// are linear in dy, so a bound on their sums must not depend on how small they are.
struct SquareSum {
    float sum = 0.0f, most = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float q = v * static_cast<float>(uint64_t{1} << kNormExp);
        sum += q * q;
        most = __builtin_fmaxf(most, __builtin_fabsf(v));
    }
    __device__ __forceinline__ float bound() const { return sum + (most > 0.0f ? 0x1p-121f : 0.0f); }
};
// Makes an offset opaque: what is derived from it is computed where it is used instead of being
// kept in registers over the whole loop over the heads.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
// keeps a sum where it is computed (moved to the loop's end it would keep its terms in registers)
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void settle(f4& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(v[e]));
}

// ---------------------------------------------------------------------------------------
// decays
// ---------------------------------------------------------------------------------------
// Block: one row, chunk and 16 heads; dt is turned over in LDS, then a wavefront does four heads,
// two tokens a lane.
__global__ void __launch_bounds__(256) sbf_decay_kernel(ScanBwdArgs a) {
    __shared__ float dts[16][kFQ + 1];
    const int64_t hb = (a.H + 15) / 16;
    const int64_t h0 = blockIdx.x % hb * 16, c = blockIdx.x / hb % a.chunks, b = blockIdx.x / hb / a.chunks;
    const int64_t t0 = c * kFQ;
    const int nv = a.L - t0 < kFQ ? static_cast<int>(a.L - t0) : kFQ;
    for (int i = threadIdx.x; i < 16 * kFQ; i += 256) {
        const int h = i & 15, t = i >> 4;
        dts[h][t] = t < nv && h0 + h < a.H ? a.dt[(b * a.L + t0 + t) * a.H + h0 + h] : 0.0f;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63;
    const int32_t* seq = a.seq ? a.seq + b * a.L + t0 : nullptr;
    int start[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int t = lane + 64 * k;
        if (seq && t < nv && t0 + t > 0) start[k] = seq[t] != seq[t - 1];
    }
    int r0 = start[0], r1 = start[1];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u0 = __shfl_up(r0, o), u1 = __shfl_up(r1, o);
        if (lane >= o) {
            r0 += u0;
            r1 += u1;
        }
    }
    r1 += __shfl(r0, 63);
    const int rend = __shfl(r1, 63);
    if (h0 == 0 && threadIdx.x < 64) {
        a.starts[(b * a.chunks + c) * kFQ + lane] = r0;
        a.starts[(b * a.chunks + c) * kFQ + 64 + lane] = r1;
        // (every lane counts: the ballots are the wavefront's)
        const int head = __popcll(__ballot(r0 == 0)) + __popcll(__ballot(r1 == 0));
        const int tail = __popcll(__ballot(r0 != rend)) + __popcll(__ballot(r1 != rend));
        if (lane == 0) a.bounds[b * a.chunks + c] = int2{head, tail};
    }
    for (int j = 0; j < 4; ++j) {
        const int h = (threadIdx.x >> 6) + 4 * j;
        if (h0 + h >= a.H) break;
        const double A2 = static_cast<double>(a.A[h0 + h]) * 1.4426950408889634;
        const float d0 = dts[h][lane], d1 = dts[h][64 + lane];
        double s0 = d0 * A2, s1 = d1 * A2;
        // a = 0 in fp32 by far: the sums keep what follows
        if (s0 < -1500.0) s0 = -1500.0;
        if (s1 < -1500.0) s1 = -1500.0;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double u0 = __shfl_up(s0, o), u1 = __shfl_up(s1, o);
            if (lane >= o) {
                s0 += u0;
                s1 += u1;
            }
        }
        s1 += __shfl(s0, 63);
        const double end = __shfl(s1, 63);
        const int64_t bh = b * a.H + h0 + h;
        float* rec = a.decay + (bh * a.chunks + c) * 5 * kFQ;
        auto put = [&](int t, double s, int r, float d) {
            const float hi = static_cast<float>(s);
            rec[t] = hi;
            rec[kFQ + t] = static_cast<float>(s - hi);
            rec[2 * kFQ + t] = r == 0 ? exp2_of(s) : 0.0f;
            rec[3 * kFQ + t] = r == rend ? exp2_of(end - s) : 0.0f;
            rec[4 * kFQ + t] = d;
        };
        put(lane, s0, r0, d0);
        put(64 + lane, s1, r1, d1);
        if (lane == 63) a.through[bh * a.chunks + c] = r1 == 0 ? exp2_of(s1) : 0.0f;
    }
}

// ---------------------------------------------------------------------------------------
// states before the chunks (forward) and gradients after them (reverse)
// ---------------------------------------------------------------------------------------
// Block: row, head, direction; wavefront w holds channels 16 w .. of the state as result tiles
// [p][n].  Stored as the tiles lie, [n tile][p tile][lane][4]: a store is 1024 consecutive bytes, and
// the gradient kernels' operands (a state dimension, eight channels) are two 16-byte pieces of it.
// SEQ: the chunks in turn; else one chunk's own share.
template <int N, bool SEQ>
__global__ void __launch_bounds__(256, 2) sbf_states_kernel(ScanBwdArgs a) {
    constexpr int TH = 256, NT = N / 16, RB = 2 * N, BP = N / 8;  // n tiles, row bytes and pieces of B
    constexpr int BL = kFQ * BP / TH, XL = kFQ * 8 / TH, XR = TH / 8, BR = TH / BP;  // loads a thread, rows apart
    __shared__ __attribute__((aligned(16))) uint8_t sb[kFQ * RB];
    __shared__ __attribute__((aligned(16))) uint8_t sx[kFQ * 128];
    __shared__ __attribute__((aligned(16))) float scale[kFQ];
    const bool rev = blockIdx.y != 0;
    const int64_t per = SEQ ? 1 : a.chunks;
    const int64_t bh = blockIdx.x / per, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t x_row = rev ? a.dy_row : a.x_row, b_row = rev ? a.c_row : a.b_row;
    const uint16_t* xs = static_cast<const uint16_t*>(rev ? a.dy : a.x) + b * a.L * x_row + h * kFP;
    const uint16_t* bs = static_cast<const uint16_t*>(rev ? a.C : a.Bm) + b * a.L * b_row + g * N;
    float* out = (rev ? a.grads : a.states) + bh * a.chunks * N * kFP;
    // lane offsets of the loads and of the stores, the same for every chunk
    const uint32_t vx = static_cast<uint32_t>((tid >> 3) * x_row * 2 + 16 * (tid & 7));
    const uint32_t vb = static_cast<uint32_t>((tid / BP) * b_row * 2 + 16 * (tid % BP));
    const uint32_t vo = static_cast<uint32_t>(w * 1024 + lane * 16);

    // The next chunk's loads, none of them under a branch or used here: a use would wait for all
    // of them, and behind a branch around some the wait for one is a wait for all.  Rows past the
    // row's end are its last, set to 0 when they are staged.
    u4 rb[BL], rx[XL];
    float rs0, rs1, rth;
    int2 rbound;
    int nv;
    auto load = [&](int64_t c) __attribute__((always_inline)) {
        const int64_t t0 = c * kFQ;
        nv = a.L - t0 < kFQ ? static_cast<int>(a.L - t0) : kFQ;
        const float* rec = a.decay + (bh * a.chunks + c) * 5 * kFQ + (tid & (kFQ - 1));
        rs0 = rec[rev ? 2 * kFQ : 3 * kFQ];
        rs1 = rec[4 * kFQ];
        rth = a.through[bh * a.chunks + c];
        rbound = a.bounds[b * a.chunks + c];
        const char* xp = reinterpret_cast<const char*>(xs + t0 * x_row);
        const char* bp = reinterpret_cast<const char*>(bs + t0 * b_row);
        if (nv == kFQ) {
            const uint32_t ox = here(vx), ob = here(vb);
#pragma unroll
            for (int i = 0; i < XL; ++i) rx[i] = *reinterpret_cast<const u4any*>(xp + i * (2 * XR) * x_row + ox);
#pragma unroll
            for (int i = 0; i < BL; ++i) rb[i] = *reinterpret_cast<const u4any*>(bp + i * (2 * BR) * b_row + ob);
            asm volatile("");  // not merged with the other path
        } else {
            const int id = here(tid);
#pragma unroll
            for (int i = 0; i < XL; ++i) {
                const int r = (id >> 3) + XR * i < nv ? (id >> 3) + XR * i : nv - 1;
                rx[i] = *reinterpret_cast<const u4any*>(xp + 2 * r * x_row + 16 * (id & 7));
            }
#pragma unroll
            for (int i = 0; i < BL; ++i) {
                const int r = id / BP + BR * i < nv ? id / BP + BR * i : nv - 1;
                rb[i] = *reinterpret_cast<const u4any*>(bp + 2 * r * b_row + 16 * (id % BP));
            }
        }
    };
    const int64_t steps = SEQ ? a.chunks : 1;
    const int64_t c0 = SEQ ? (rev ? a.chunks - 1 : 0) : blockIdx.x % per, dc = rev ? -1 : 1;
    load(c0);
    f4 acc[NT];
    const float* from = SEQ ? (rev ? a.dhT : a.h0) : nullptr;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[n][e] = from ? from[(bh * kFP + 16 * w + 4 * g4 + e) * N + 16 * n + li] : 0.0f;
    auto store = [&](int64_t c) __attribute__((always_inline)) {
        char* o = reinterpret_cast<char*>(out + c * N * kFP);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            __builtin_nontemporal_store(acc[n], reinterpret_cast<f4*>(o + vo + n * 4096));
    };
    const int xo = down_off<128>(4 * g4, li) ^ (w << 5), bo = down_off<RB>(4 * g4, li);
    for (int64_t i = 0; i < steps; ++i) {
        const int64_t c = c0 + i * dc;
        // tokens that hand nothing on: past the row's end, and across a start (forward those before
        // the chunk's last start, in reverse those from its first on).  Their factor is 0, and so are
        // both operands here: a NaN or infinity of a sequence that ends in this chunk, times 0, would
        // reach the chunks behind it
        const int lo = rev ? 0 : rbound.y, hi = rev && rbound.x < nv ? rbound.x : nv;
        if (lo > 0 || hi < kFQ) {
#pragma unroll
            for (int j = 0; j < XL; ++j) {
                const int t = (tid >> 3) + XR * j;
                if (t < lo || t >= hi) rx[j] = u4{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < BL; ++j) {
                const int t = tid / BP + BR * j;
                if (t < lo || t >= hi) rb[j] = u4{0, 0, 0, 0};
            }
        }
        const float th = rth;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < XL; ++j)
            *reinterpret_cast<u4*>(sx + piece<128>(tid >> 3, tid & 7) + j * XR * 128) = rx[j];
#pragma unroll
        for (int j = 0; j < BL; ++j)
            *reinterpret_cast<u4*>(sb + piece<RB>(tid / BP, tid % BP) + j * BR * RB) = rb[j];
        if (tid < kFQ) scale[tid] = rev ? rs0 : rs0 * rs1;
        __syncthreads();
        if (SEQ) load(i + 1 < steps ? c + dc : c);  // the last once more, not used
        if (SEQ) {
            store(c);
            if (th == 0.0f) {  // nothing passes a start, whatever the state was
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = f4{0, 0, 0, 0};
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] *= th;
            }
        }
#pragma unroll
        for (int k = 0; k < kFQ / 32; ++k) {
            const u4 raw = __builtin_bit_cast(u4, down<128>(sx, xo, 32 * k, 0));
            const f4 s0 = *reinterpret_cast<const f4*>(scale + 32 * k + 4 * g4);
            const f4 s1 = *reinterpret_cast<const f4*>(scale + 32 * k + 16 + 4 * g4);
            bf8 q[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) q[n] = down<RB>(sb, bo, 32 * k, n);
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(raw[e] << 16) * (e < 2 ? s0[2 * e] : s1[2 * e - 4]);
                v[2 * e + 1] = __uint_as_float(raw[e] & 0xFFFF0000u) * (e < 2 ? s0[2 * e + 1] : s1[2 * e - 3]);
            }
            bf8 p[3];
            split(v, p);
#pragma unroll
            for (int j = 2; j >= 0; --j)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = mfma(p[j], q[n], acc[n]);
        }
        if (!SEQ) store(c);
    }
    if (SEQ && rev && a.dh0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.dh0[(bh * kFP + 16 * w + 4 * g4 + e) * N + 16 * n + li] = acc[n][e];
    }
}

// The chunks' shares summed along the row, in place (states stored as tiles, the caller's [p][n])
__global__ void __launch_bounds__(256) sbf_pass_kernel(ScanBwdArgs a) {
    const int64_t PN = kFP * a.N, per = PN / 256;
    const int64_t bh = blockIdx.x / per, i = blockIdx.x % per * 256 + threadIdx.x;
    const int64_t j = (16 * (i / 256 % 4) + 4 * (i / 64 % 4) + i % 4) * a.N + 16 * (i / 1024) + i / 4 % 16;
    const bool rev = blockIdx.y != 0;
    float* s = (rev ? a.grads : a.states) + bh * a.chunks * PN + i;
    const float* f = a.through + bh * a.chunks;
    const float* from = rev ? a.dhT : a.h0;
    float v = from ? from[bh * PN + j] : 0.0f;
    for (int64_t k0 = 0; k0 < a.chunks; k0 += 8) {
        float own[8], th[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t m = k0 + k < a.chunks ? k0 + k : a.chunks - 1;
            const int64_t c = rev ? a.chunks - 1 - m : m;
            own[k] = s[c * PN];
            th[k] = f[c];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k0 + k >= a.chunks) break;
            const int64_t c = rev ? a.chunks - 1 - (k0 + k) : k0 + k;
            s[c * PN] = v;
            v = th[k] == 0.0f ? own[k] : th[k] * v + own[k];
        }
    }
    if (rev && a.dh0) a.dh0[bh * PN + j] = v;
}

// ---------------------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------------------
template <int N>
struct GradLds {
    static constexpr int B = 0;                        // [128 s][N] bf16
    static constexpr int CB = B + kFQ * N * 2;         // C B^T, 36 tiles as results lie (at first and last: C)
    static constexpr int X = CB + 36 * 1024;           // [128 s][64] bf16
    static constexpr int DY = X + kFQ * 128;           // [128 t][64] bf16
    static constexpr int G = DY + kFQ * 128;           // three parts of [N][64] bf16
    static constexpr int ROW = G + 3 * N * 128;        // row sums of W by s tile [8][128]
    static constexpr int V = ROW + 8 * kFQ * 4;        // v by n tile [8][128]
    static constexpr int DEC = V + 8 * kFQ * 4;        // decays [5][128]
    static constexpr int START = DEC + 5 * kFQ * 4;    // [128] int
    static constexpr int LW = CB + kFQ * N * 2;        // at the end, behind C: three parts of [128 t][128 s] bf16
    static constexpr int TOTAL = START + kFQ * 4 > LW + 3 * kFQ * 256 ? START + kFQ * 4 : LW + 3 * kFQ * 256;
};
static_assert(GradLds<128>::TOTAL <= 160 * 1024, "LDS");

// Joins one head's sums over wavefronts and writes them out for the ddt kernel: threads 0-127 v,
// 128-255 the row sums, 256-319 the row sums' sums by tile.
template <int N>
__device__ __forceinline__ void head_sums(const uint8_t* sm, float* out, int tid) {
    using O = GradLds<N>;
    const int t = tid & 127, which = tid >> 7;
    const float* row = reinterpret_cast<const float*>(sm + O::ROW);
    if (which == 0) {
        const float* p = reinterpret_cast<const float*>(sm + O::V) + t;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < N / 16; ++i) v += p[i * kFQ];
        out[kSumV * kFQ + t] = v;
    } else if (which == 1) {
        float off = 0.0f;
        const int j = t >> 4;
        for (int i = 0; i < j; ++i) off += row[i * kFQ + t];
        out[kSumRowOff * kFQ + t] = off;
        out[kSumRowDiag * kFQ + t] = row[j * kFQ + t];
    } else if (which == 2 && t < 64) {
        const int j = t >> 3, i = t & 7;
        float r = 0.0f;
        if (i < j) {
            const f4* p = reinterpret_cast<const f4*>(row + i * kFQ + 16 * j);
            const f4 q = (p[0] + p[1]) + (p[2] + p[3]);
            r = (q[0] + q[1]) + (q[2] + q[3]);
        }
        out[kSums * kFQ + t] = r;
    }
}

// dC from before the chunk, summed over the heads of a range, and u
template <int N>
__global__ void __launch_bounds__(512, 4) sbf_dc_kernel(ScanBwdArgs a) {
    constexpr int NT = N / 16, RB = 2 * N, BP = N / 8;
    constexpr int TT = NT;  // t tiles a wavefront does: all 8, or half of them
    __shared__ __attribute__((aligned(16))) uint8_t sc[kFQ * RB];
    __shared__ __attribute__((aligned(16))) uint8_t sdy[2][kFQ * 128];
    __shared__ float su[2][8][kFQ];
    __shared__ float sf[2][kFQ];
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t hs = blockIdx.x % a.dc_splits, g = blockIdx.x / a.dc_splits % a.G;
    const int64_t c = blockIdx.x / a.dc_splits / a.G % a.chunks, b = blockIdx.x / a.dc_splits / a.G / a.chunks;
    const int64_t k_heads = a.H / a.G;
    const int64_t hfirst = g * k_heads + hs * a.dc_heads;
    const int64_t hend = hs * a.dc_heads + a.dc_heads < k_heads ? hfirst + a.dc_heads : (g + 1) * k_heads;
    const int64_t t0 = c * kFQ, tok = b * a.L + t0;
    const int nv = a.L - t0 < kFQ ? static_cast<int>(a.L - t0) : kFQ;
    const int nt = wave % NT, th0 = NT == 8 ? 0 : (wave / NT) * TT;
    const bool fresh = a.bounds[b * a.chunks + c].x == 0;  // a start on its first token: S is another sequence's
    const int row = tid >> 3;
    const uint32_t vdy = static_cast<uint32_t>(row * a.dy_row * 2 + 16 * (tid & 7));
    const uint32_t vs = static_cast<uint32_t>(nt * 4096 + (g4 >> 1) * 1024 + (g4 & 1) * 512 + li * 16);
    u4 rdy[2];
    f4 rS[4];
    float rf = 0.0f;
    auto load = [&](int64_t h) __attribute__((always_inline)) {
        const char* db = reinterpret_cast<const char*>(static_cast<const uint16_t*>(a.dy) + tok * a.dy_row + h * kFP);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rdy[i] = u4{0, 0, 0, 0};
            if (row + 64 * i < nv) rdy[i] = *reinterpret_cast<const u4any*>(db + i * 128 * a.dy_row + vdy);
        }
        const char* sp = reinterpret_cast<const char*>(a.states + ((b * a.H + h) * a.chunks + c) * N * kFP);
#pragma unroll
        for (int i = 0; i < 4; ++i) rS[i] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(sp + 2048 * (i >> 1) + 256 * (i & 1) + vs));
        if (tid < kFQ) rf = a.decay[(((b * a.H + h) * a.chunks + c) * 5 + 2) * kFQ + tid];
    };
    load(hfirst);
    {
        const uint16_t* cg = static_cast<const uint16_t*>(a.C) + tok * a.c_row + g * N;
        for (int q = tid; q < kFQ * BP; q += 512) {
            const int r = q / BP;
            u4 u{0, 0, 0, 0};
            if (r < nv) u = *reinterpret_cast<const u4any*>(cg + r * a.c_row + 8 * (q % BP));
            *reinterpret_cast<u4*>(sc + piece<RB>(r, q % BP)) = u;
        }
    }
    f4 acc[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[j] = f4{0, 0, 0, 0};
    const int64_t sum_step = a.chunks * (kSums * kFQ + kSumTail);
    float* sums = a.sums + ((b * a.H + hfirst) * a.chunks + c) * (kSums * kFQ + kSumTail) + kSumU * kFQ;
    auto put_u = [&](int par) __attribute__((always_inline)) {  // of the head before
        if (tid < kFQ) {
            float u = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i) u += su[par][i][tid];
            (sums - sum_step)[tid] = u;
        }
    };
    const int xo = along_off<128>(li, g4) + 16 * th0 * 128;
    const int cw = piece<RB>(li, 2 * nt + (g4 >> 1)) + 8 * (g4 & 1) + 16 * th0 * RB;
    for (int64_t h = hfirst; h < hend; ++h) {
        const int par = static_cast<int>(h - hfirst) & 1;
        bf8 Sp[2][3];
        SquareSum squares;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = fresh ? 0.0f : rS[2 * kk + (e >> 2)][e & 3];
                squares.add(v[e]);
            }
            split(v, Sp[kk]);
        }
        const float norm = group_sum4(lane_sum16(squares.bound()));
        if (lane == 0 && wave < NT) sums[(kSums - kSumU) * kFQ + 64 + nt] = norm;
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<u4*>(sdy[par] + piece<128>(row, tid & 7) + i * 64 * 128) = rdy[i];
        if (tid < kFQ) sf[par][tid] = rf;
        // one barrier a head: what is written above was last read two heads ago
        __syncthreads();
        if (h > hfirst) put_u(par ^ 1);
        if (h + 1 < hend) load(h + 1);
        const uint8_t* dp = sdy[par] + here(xo);
        const uint8_t* dq = sdy[par] + here(xo ^ 64);
        const uint8_t* fp = reinterpret_cast<const uint8_t*>(sf[par]) + here(64 * th0 + 4 * li);
        float* up = su[par][nt] + here(16 * (th0 + group_of_row(g4)) + li);
        float u[4];
#pragma unroll
        for (int jj = 0; jj < TT; ++jj) {
            const bf8 d0 = lds<bf8>(dp + 16 * jj * 128), d1 = lds<bf8>(dq + 16 * jj * 128);
            f4 o{0, 0, 0, 0};
#pragma unroll
            for (int k = 2; k >= 0; --k) {
                o = mfma(Sp[0][k], d0, o);
                o = mfma(Sp[1][k], d1, o);
            }
            const float ft = lds<float>(fp + 64 * jj);
            const u2 cv = lds<u2>(sc + cw + 16 * jj * RB);
            float w = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w += __uint_as_float(e & 1 ? cv[e >> 1] & 0xFFFF0000u : cv[e >> 1] << 16) * o[e];
                acc[jj][e] += ft * o[e];
            }
            settle(acc[jj]);
            settle(w);
            u[jj & 3] = ft == 0.0f ? 0.0f : w * ft;  // of another sequence's dy, say, if it is no number
            if ((jj & 3) == 3) up[16 * (jj - 3)] = group_sums(u[0], u[1], u[2], u[3]);
        }
        sums += sum_step;
    }
    __syncthreads();
    put_u(static_cast<int>(hend - 1 - hfirst) & 1);
#pragma unroll
    for (int jj = 0; jj < TT; ++jj) {
        const int t = 16 * (th0 + jj) + li;
        if (t < nv)
            *reinterpret_cast<f4*>(a.dC_head + (hs * a.B * a.L + tok + t) * a.G * N + g * N + 16 * nt + 4 * g4) = acc[jj];
    }
}

// f_last <G, S> of the last chunk of every kAnchor (one block each)
__global__ void __launch_bounds__(256) sbf_anchor_kernel(ScanBwdArgs a) {
    __shared__ float sum[4];
    const int64_t n = (a.chunks + kAnchor - 1) / kAnchor;
    const int64_t bh = blockIdx.x / n, i = blockIdx.x % n;
    const int64_t c = (i + 1) * kAnchor < a.chunks ? (i + 1) * kAnchor - 1 : a.chunks - 1;
    const int64_t at = bh * a.chunks + c, PN = a.P * a.N;
    const float th = a.through[at];
    float d = 0.0f;
    if (th != 0.0f)
        for (int64_t k = threadIdx.x * 4; k < PN; k += 1024) {
            const f4 x = *reinterpret_cast<const f4*>(a.states + at * PN + k);
            const f4 y = *reinterpret_cast<const f4*>(a.grads + at * PN + k);
            d += (x[0] * y[0] + x[1] * y[1]) + (x[2] * y[2] + x[3] * y[3]);
        }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) d += __shfl_xor(d, o);
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = d;
    __syncthreads();
    if (threadIdx.x == 0) a.anchor[bh * n + i] = th * ((sum[0] + sum[1]) + (sum[2] + sum[3]));
}

// 16 wavefronts, four a SIMD, in two roles that meet at the two barriers of a head and otherwise
// run beside each other:
//   0-7   s tile st (1, 2, .. and 7, 6, .. on one SIMD: nine pair tiles each): the pairs, W's sums, dx
//   8-15  n tile nt: G's parts, dB from behind the chunk and v; between the barriers the head
//         before's sums
// LDS holds one block a CU, so the roles are what hides one's LDS waits behind the other's
// products: as eight wavefronts that did both in turn it took 541 us where the roles took 478 (227
// and 190 us at one row of 32768 tokens, 24 heads, dstate 64), with two parts for the pairs and for
// G of dx; with three of each it takes 515 and 212.  The third part of G fills the 160 KB, so the
// heads' sums have one place, not two in turn, and are written out between the barriers.  The t
// tiles are taken in pairs from an even one on, so that the bodies a wavefront may start in are few
// and keep within 128 registers: from any one on they were 8, and 510 us where these took 478.
template <int N>
__global__ void __launch_bounds__(1024) sbf_grad_kernel(ScanBwdArgs a) {
    using O = GradLds<N>;
    constexpr int NT = N / 16, RB = 2 * N, BP = N / 8;
    constexpr int TT = NT;       // s tiles a wavefront does for dB: all 8, or half of them
    constexpr int PL = N * 128;  // bytes of one part of G
    constexpr int LR = kFQ * 4;  // bytes of one float a token
    __shared__ __attribute__((aligned(16))) uint8_t sm[O::TOTAL];
    const int tid = threadIdx.x & 511, lane = tid & 63, li = lane & 15, g4 = lane >> 4;
    const bool pairs = __builtin_amdgcn_readfirstlane(threadIdx.x >> 9) == 0;  // the role
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t hs = blockIdx.x % a.splits, g = blockIdx.x / a.splits % a.G;
    const int64_t c = blockIdx.x / a.splits / a.G % a.chunks, b = blockIdx.x / a.splits / a.G / a.chunks;
    const int64_t k_heads = a.H / a.G;
    const int64_t hfirst = g * k_heads + hs * a.split_heads;
    const int heads = static_cast<int>(hs * a.split_heads + a.split_heads < k_heads ? a.split_heads : k_heads - hs * a.split_heads);
    const int64_t t0 = c * kFQ, tok = b * a.L + t0;
    const int nv = a.L - t0 < kFQ ? static_cast<int>(a.L - t0) : kFQ;
    const int nt = wave % NT, th0 = NT == 8 ? 0 : (wave / NT) * TT;  // n tile and first s tile for dB
    const int st = wave < 4 ? wave : 11 - wave;
    int* starts = reinterpret_cast<int*>(sm + O::START);

    // loads of one head: uniform bases that move with the head, 32-bit lane offsets that do not
    // (128 token rows are under 2^32 bytes).  The pairs' role stages dy, the other x, G and decays.
    const int64_t xrow = pairs ? a.dy_row : a.x_row;
    const char* xb = reinterpret_cast<const char*>(static_cast<const uint16_t*>(pairs ? a.dy : a.x) + tok * xrow + hfirst * kFP);
    const int xpart = pairs ? O::DY : O::X;
    u4 rx[2];
    auto load_x = [&]() __attribute__((always_inline)) {
        const int id = here(tid), row = id >> 3;  // and row + 64
        const uint32_t vx = static_cast<uint32_t>(row) * static_cast<uint32_t>(xrow * 2) + 16 * (id & 7);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rx[i] = u4{0, 0, 0, 0};
            if (row + 64 * i < nv) rx[i] = *reinterpret_cast<const u4any*>(xb + i * 128 * xrow + vx);
        }
        xb += kFP * 2;
    };
    auto stage_x = [&]() __attribute__((always_inline)) {  // rows row and row + 64 share the swizzle
        const int id = here(tid), xpiece = xpart + piece<128>(id >> 3, id & 7);
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<u4*>(sm + xpiece + i * 64 * 128) = rx[i];
    };
    {
        const uint16_t* bg = static_cast<const uint16_t*>(pairs ? a.Bm : a.C) + tok * (pairs ? a.b_row : a.c_row) + g * N;
        const int64_t brow = pairs ? a.b_row : a.c_row;
        for (int q = tid; q < kFQ * BP; q += 512) {
            const int r = q / BP;
            u4 v{0, 0, 0, 0};
            if (r < nv) v = *reinterpret_cast<const u4any*>(bg + r * brow + 8 * (q % BP));
            *reinterpret_cast<u4*>(sm + (pairs ? O::B : O::CB) + piece<RB>(r, q % BP)) = v;
        }
        if (threadIdx.x < kFQ) starts[threadIdx.x] = a.starts[(b * a.chunks + c) * kFQ + threadIdx.x];
    }
    const int64_t sum_step = a.chunks * (kSums * kFQ + kSumTail);
    float* sums = a.sums + ((b * a.H + hfirst) * a.chunks + c) * (kSums * kFQ + kSumTail);
    __syncthreads();

    if (pairs) {
        const bool masked = __builtin_amdgcn_readfirstlane(starts[kFQ - 1]) != 0;
        // C B^T of this wavefront's s tile and t tiles st .. 7, then in place of C
        const int cbt = O::CB + (st * (17 - st) / 2) * 1024 - st * 1024;  // t tile j at + 1024 j
        {
            f4 cb[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cb[j] = f4{0, 0, 0, 0};
                if (j >= st) {
#pragma unroll
                    for (int kk = 0; kk < N / 32; ++kk)
                        cb[j] = mfma(lds<bf8>(sm + O::CB + 16 * j * RB + (along_off<RB>(li, g4) ^ (kk << 6))),
                                     lds<bf8>(sm + O::B + 16 * st * RB + (along_off<RB>(li, g4) ^ (kk << 6))), cb[j]);
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= st) *reinterpret_cast<f4*>(sm + cbt + 16 * lane + 1024 * j) = cb[j];
        }
        load_x();
        // sums over the heads of L dt (dy x^T) with s tile st: the even t tile and its neighbour that
        // hold the diagonal, and tiles 2 m, 2 m + 1 behind them
        f4 lwd[2] = {}, lw[3][2] = {};
        char* dxp = reinterpret_cast<char*>(static_cast<uint16_t*>(a.dx) + tok * a.dx_row + hfirst * kFP);
        for (int h = 0; h < heads; ++h) {
            __syncthreads();  // the previous head's x, dy and G have been read
            stage_x();
            __syncthreads();
            // all that depends on the lane is computed anew for each head: registers are short
            const int ln = here(lane), li = ln & 15, g4 = ln >> 4, s = 16 * st + li;
            const int rs = masked ? starts[s] : 0;
            // LDS offsets of this head's reads
            const int xo = here(O::X + along_off<128>(li, g4));              // x, dy along rows
            const int yo = here(O::DY + down_off<128>(4 * g4, li));          // dy down rows
            const int tl = here(O::DEC + 4 * li);                            // decays of token li of a tile
            const int t4 = here(O::DEC + 16 * g4);                           // decays of tokens 4 g4 ..
            const int rt = here(O::ROW + st * LR + 16 * g4 + 4 * (li & 3));  // row sums
            const int ct = here(cbt + 16 * ln);                              // C B^T

            // ---- pairs s <= t: W's sums, the pairs' part of dx ----
            f4 dxa[4] = {};
            const float hi_s = lds<float>(sm + tl + 64 * st), lo_s = lds<float>(sm + tl + LR + 64 * st);
            const float dts = lds<float>(sm + tl + 4 * LR + 64 * st);
            float below = 0.0f, bdiag = 0.0f, diag = 0.0f;  // column sums of W / dt_s
            u4 pw[3];  // three parts of the pairs of two t tiles, in token order
            // the pairs of t tile j with s tile st, in half i of that operand
            auto tile = [&](int j, int i, f4& sum, auto on_diagonal) __attribute__((always_inline)) {
                constexpr bool DIAG = decltype(on_diagonal)::value;
                const uint8_t* dp = sm + xo + (O::DY - O::X) + j * 2048;
                const uint8_t* dq = sm + (xo ^ 64) + (O::DY - O::X) + j * 2048;
                f4 yx = mfma(lds<bf8>(dp), lds<bf8>(sm + xo + 2048 * st), f4{0, 0, 0, 0});
                yx = mfma(lds<bf8>(dq), lds<bf8>(sm + (xo ^ 64) + 2048 * st), yx);
                const f4 ht = lds<f4>(sm + t4 + 64 * j), lt = lds<f4>(sm + t4 + LR + 64 * j);
                f4 l;
#pragma unroll
                for (int e = 0; e < 4; ++e) l[e] = __builtin_amdgcn_exp2f((ht[e] - hi_s) + (lt[e] - lo_s));
                if (masked) {
                    const int4 r = *reinterpret_cast<const int4*>(starts + 16 * j + 4 * g4);
                    l = f4{r.x == rs ? l[0] : 0.0f, r.y == rs ? l[1] : 0.0f, r.z == rs ? l[2] : 0.0f, r.w == rs ? l[3] : 0.0f};
                }
                const f4 cb = lds<f4>(sm + ct + 1024 * j);
                const int d = li - 4 * g4;  // t - s = e - d on the diagonal
                float pv[4], rw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (DIAG) l[e] = e >= d ? l[e] : 0.0f;
                    pv[e] = l[e] * cb[e];
                    const float yd = yx[e] * dts;
                    sum[e] += l[e] * yd;
                    rw[e] = pv[e] * yd;
                    if (DIAG) {
                        const float w = pv[e] * yx[e];
                        diag += e == d ? w : 0.0f;
                        bdiag += e == d ? 0.0f : w;
                        rw[e] = e == d ? 0.0f : rw[e];
                    } else {
                        below += pv[e] * yx[e];
                    }
                }
                settle(sum);
                if (DIAG) spanning(rw, li, g4);
                *reinterpret_cast<float*>(sm + rt + 64 * j) = row_sums(rw, li);  // the same from four lanes
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint32_t q0 = pack_bf16x2(pv[0], pv[1]), q1 = pack_bf16x2(pv[2], pv[3]);
                    pw[k][2 * i] = q0;
                    pw[k][2 * i + 1] = q1;
                    pv[0] -= __uint_as_float(q0 << 16);
                    pv[1] -= __uint_as_float(q0 & 0xFFFF0000u);
                    pv[2] -= __uint_as_float(q1 << 16);
                    pv[3] -= __uint_as_float(q1 & 0xFFFF0000u);
                }
                __builtin_amdgcn_sched_barrier(0);  // the registers of one tile at a time
            };
            // their part of dx, from t tile j on (even)
            auto to_dx = [&](int j) __attribute__((always_inline)) {
#pragma unroll
                for (int p0 = 0; p0 < 4; p0 += 2) {
                    bf8 y[2];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint8_t* q = sm + (yo ^ ((p0 + p) << 5)) + j * 2048;
                        y[p] = join(tr_read(q), tr_read(q + 16 * 128));
                    }
#pragma unroll
                    for (int k = 2; k >= 0; --k)
#pragma unroll
                        for (int p = 0; p < 2; ++p) dxa[p0 + p] = mfma(y[p], __builtin_bit_cast(bf8, pw[k]), dxa[p0 + p]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            if (st & 1) {
                pw[0] = pw[1] = pw[2] = u4{0, 0, 0, 0};
            } else {
                tile(st, 0, lwd[0], std::true_type{});
            }
            if (st & 1) tile(st, 1, lwd[1], std::true_type{});
            else tile(st + 1, 1, lwd[1], std::false_type{});
            to_dx(st & 6);
#pragma unroll
            for (int m = 1; m < 4; ++m)
                if (m > (st >> 1)) {
                    tile(2 * m, 0, lw[m - 1][0], std::false_type{});
                    tile(2 * m + 1, 1, lw[m - 1][1], std::false_type{});
                    to_dx(2 * m);
                }
            if (h + 1 < heads) load_x();
            {  // rows of lanes 0, 1, 2: kSumColOff, kSumColDiag, kSumDiag
                const float v = group_sums(below, diag, bdiag, 0.0f);
                if (g4 < 3) sums[(kSumColOff + g4) * kFQ + s] = v;
            }
            sums += sum_step;

            // ---- dx: G B, then with the pairs ----
            const float es = lds<float>(sm + tl + 3 * LR + 64 * st);
            const int bst = here(along_off<RB>(li, g4) + 16 * st * RB);  // B, rows of s tile st
            const int go0 = here(O::G + down_off<128>(8 * g4, li)), go1 = here(O::G + down_off<128>(8 * g4 + 4, li));
            f4 gb[4] = {};
#pragma unroll
            for (int kk = 0; kk < N / 32; ++kk) {
                const bf8 bf = lds<bf8>(sm + (bst ^ (kk << 6)));
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int o = k * PL + 32 * kk * 128;
                        gb[p] = mfma(join(tr_read(sm + (go0 ^ (p << 5)) + o), tr_read(sm + (go1 ^ (p << 5)) + o)), bf, gb[p]);
                    }
            }
            const uint32_t vdx = static_cast<uint32_t>(s) * static_cast<uint32_t>(a.dx_row * 2) + 8 * g4;
            if (s < nv) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    f4 r;
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = dts * (dxa[p][e] + es * gb[p][e]);
                    *reinterpret_cast<u2any*>(dxp + vdx + 32 * p) = u2{pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3])};
                }
            }
            dxp += kFP * 2;
        }
        __syncthreads();
        __syncthreads();  // the last head's sums have been read
        // ---- the heads' summed pairs: three parts of [t][s] in LDS (zero above the diagonal) ----
        const int s = 16 * st + li;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = j >> 1 == st >> 1 ? lwd[j & 1][e] : j > st ? lw[(j >> 1) > 0 ? (j >> 1) - 1 : 0][j & 1][e] : 0.0f;
                const int t = 16 * j + 4 * g4 + e;
                const int o = piece<256>(t, s >> 3) + 2 * (s & 7);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint16_t part = f32_to_bf16(v);
                    *reinterpret_cast<uint16_t*>(sm + O::LW + k * kFQ * 256 + o) = part;
                    v -= bf16_to_f32(part);
                }
            }
        __syncthreads();
        // ---- dC of n tile nt: sbf_dc's part (where this block alone has the pairs), then the pairs ----
        const int b0 = down_off<RB>(8 * g4, li) ^ (nt << 5), b1 = down_off<RB>(8 * g4 + 4, li) ^ (nt << 5);
        const int lo_ = along_off<256>(li, g4);
#pragma unroll
        for (int jj = 0; jj < TT; ++jj) {
            const int j = th0 + jj, t = 16 * j + li;
            const int64_t col = g * N + 16 * nt + 4 * g4, slab = a.B * a.L * a.G * N;
            const int64_t at = (tok + t) * a.G * N + col;
            f4 acc{0, 0, 0, 0};
            if (a.splits == 1 && t < nv)
                for (int64_t i = 0; i < a.dc_splits; ++i) acc += *reinterpret_cast<const f4*>(a.dC_head + i * slab + at);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (2 * k <= j) {  // s tiles 2 k, 2 k + 1
                    const uint8_t* p = sm + O::B + 32 * k * RB;
                    const bf8 f = join(tr_read(p + b0), tr_read(p + b1));
#pragma unroll
                    for (int i = 2; i >= 0; --i) acc = mfma(f, along<256>(sm + O::LW + i * kFQ * 256, lo_, 16 * j, k), acc);
                }
            if (t >= nv) continue;
            if (a.splits == 1)
                *reinterpret_cast<u2any*>(static_cast<uint16_t*>(a.dC) + (tok + t) * a.dc_row + col) =
                    u2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
            else
                *reinterpret_cast<f4*>(a.dC_head + (a.dc_splits + hs) * slab + at) = acc;
        }
    } else {
        const char* gp = reinterpret_cast<const char*>(a.grads + ((b * a.H + hfirst) * a.chunks + c) * N * kFP);
        const float* rec = a.decay + ((b * a.H + hfirst) * a.chunks + c) * 5 * kFQ;
        f4 rG[4];
        float rd[2];
        auto load_g = [&]() __attribute__((always_inline)) {
            const int ln = here(lane);
            const uint32_t vs = static_cast<uint32_t>(nt * 4096 + (ln >> 5) * 1024 + (ln >> 4 & 1) * 512 + (ln & 15) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rG[i] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(gp + 2048 * (i >> 1) + 256 * (i & 1) + vs));
            gp += a.chunks * N * kFP * 4;
            const int id = here(tid);
            rd[0] = rec[id];
            if (id < kFQ) rd[1] = rec[4 * kFQ + id];
            rec += a.chunks * 5 * kFQ;
        };
        load_g();
        load_x();
        __syncthreads();  // the other role's of C B^T
        f4 acc[TT] = {};
        for (int h = 0; h < heads; ++h) {
            const int id = here(tid), ln = id & 63, li = ln & 15, g4 = ln >> 4;
            bf8 Gp[2][3];
            SquareSum squares;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = rG[2 * kk + (e >> 2)][e & 3];
                    squares.add(v[e]);
                }
                split(v, Gp[kk]);
            }
            const float norm = group_sum4(lane_sum16(squares.bound()));
            if (ln == 0 && wave < NT) sums[kSums * kFQ + 72 + nt] = norm;
            __syncthreads();  // the previous head's x, dy and G have been read
            stage_x();
            if (wave < NT) {
                const int q = here(O::G + 16 * nt * 128 + along_off<128>(li, g4));
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int k = 0; k < 3; ++k) *reinterpret_cast<bf8*>(sm + k * PL + (q ^ (kk << 6))) = Gp[kk][k];
            }
            {
                float* dec = reinterpret_cast<float*>(sm + O::DEC);
                dec[id] = rd[0];
                if (id < kFQ) dec[4 * kFQ + id] = rd[1];
            }
            if (h > 0) head_sums<N>(sm, sums - sum_step, here(id));
            __syncthreads();
            if (h + 1 < heads) load_x();
            sums += sum_step;
            const int xo = here(O::X + along_off<128>(li, g4));                      // x along rows
            const int cw = here(piece<RB>(li, 2 * nt + (g4 >> 1)) + 8 * (g4 & 1));   // B elements (n 4 g4 .., s li)
            const int tl = here(O::DEC + 4 * li);                                    // decays of token li of a tile
            const int vt = here(O::V + nt * LR + 64 * group_of_row(g4) + 4 * li);  // v of n tile nt, four s tiles
            float v[4];
#pragma unroll
            for (int jj = 0; jj < TT; ++jj) {
                const int j = th0 + jj;
                const bf8 x0 = lds<bf8>(sm + xo + 16 * j * 128), x1 = lds<bf8>(sm + (xo ^ 64) + 16 * j * 128);
                f4 o{0, 0, 0, 0};
#pragma unroll
                for (int k = 2; k >= 0; --k) {
                    o = mfma(Gp[0][k], x0, o);
                    o = mfma(Gp[1][k], x1, o);
                }
                const float es = lds<float>(sm + tl + 3 * LR + 64 * j), ed = es * lds<float>(sm + tl + 4 * LR + 64 * j);
                const u2 bv = lds<u2>(sm + cw + O::B + 16 * j * RB);
                float w = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w += __uint_as_float(e & 1 ? bv[e >> 1] & 0xFFFF0000u : bv[e >> 1] << 16) * o[e];
                    acc[jj][e] += ed * o[e];
                }
                settle(acc[jj]);
                settle(w);
                if (jj == TT / 2 - 1 && h + 1 < heads) load_g();
                v[jj & 3] = es == 0.0f ? 0.0f : w * es;
                if ((jj & 3) == 3) *reinterpret_cast<float*>(sm + vt + 64 * (j - 3)) = group_sums(v[0], v[1], v[2], v[3]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
        head_sums<N>(sm, sums - sum_step, tid);
        __syncthreads();
        {  // C again, in place of C B^T
            const uint16_t* cg = static_cast<const uint16_t*>(a.C) + tok * a.c_row + g * N;
            for (int q = tid; q < kFQ * BP; q += 512) {
                const int r = q / BP;
                u4 u{0, 0, 0, 0};
                if (r < nv) u = *reinterpret_cast<const u4any*>(cg + r * a.c_row + 8 * (q % BP));
                *reinterpret_cast<u4*>(sm + O::CB + piece<RB>(r, q % BP)) = u;
            }
        }
        __syncthreads();
        // ---- dB of n tile nt: the pairs ----
        const int bo = down_off<RB>(4 * g4, li) ^ (nt << 5), ld = down_off<256>(4 * g4, li);
#pragma unroll
        for (int jj = 0; jj < TT; ++jj) {
            const int j = th0 + jj, t = 16 * j + li;
            const int64_t col = g * N + 16 * nt + 4 * g4;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (2 * k + 1 >= j) {  // t tiles 2 k, 2 k + 1
                    const bf8 f = down<RB>(sm + O::CB, bo, 32 * k, 0);
#pragma unroll
                    for (int i = 2; i >= 0; --i) acc[jj] = mfma(f, down<256>(sm + O::LW + i * kFQ * 256, ld, 32 * k, j), acc[jj]);
                }
            if (t >= nv) continue;
            if (a.splits == 1)
                *reinterpret_cast<u2any*>(static_cast<uint16_t*>(a.dB) + (tok + t) * a.db_row + col) =
                    u2{pack_bf16x2(acc[jj][0], acc[jj][1]), pack_bf16x2(acc[jj][2], acc[jj][3])};
            else
                *reinterpret_cast<f4*>(a.dB_head + ((hs * a.B * a.L + tok + t) * a.G) * N + col) = acc[jj];
        }
    }
}

// dB, dC of several ranges of heads, added in order and rounded once (blockIdx.y: dB, dC)
__global__ void __launch_bounds__(256) sbf_join_kernel(ScanBwdArgs a) {
    const int64_t GN = a.G * a.N, n = a.B * a.L * GN;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const float* p = (blockIdx.y ? a.dC_head : a.dB_head) + i;
    f4 s = *reinterpret_cast<const f4*>(p);
    const int64_t slabs = a.splits + (blockIdx.y ? a.dc_splits : 0);
#pragma unroll 8
    for (int64_t j = 1; j < slabs; ++j) s += *reinterpret_cast<const f4*>(p + j * n);
    uint16_t* o = blockIdx.y ? static_cast<uint16_t*>(a.dC) + i / GN * a.dc_row
                             : static_cast<uint16_t*>(a.dB) + i / GN * a.db_row;
    *reinterpret_cast<u2any*>(o + i % GN) = u2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
}

size_t r256(size_t n) { return (n + 255) / 256 * 256; }

// Ranges of heads a chunk and group: one block runs on a unit at a time (LDS), so the time is
// the rounds of blocks over the 256 units times what a block does: its heads, and about two
// heads' worth of B, C and the pairs' end.  Against one range, dstate 128: 1 x 8192 x 64 heads
// 406 for 625 us, 2 x 8192 x 48 581 for 689, 2 x 2048 x 64 190 for 480.
void cut_heads(ScanBwdArgs& a) {
    const int64_t blocks = a.B * a.chunks * a.G, k = a.H / a.G;
    int64_t best = -1;
    for (int64_t n = 1; n <= k && n <= 256; ++n) {
        const int64_t heads = (k + n - 1) / n;
        if ((k + heads - 1) / heads != n) continue;
        const int64_t cost = (blocks * n + 255) / 256 * (heads + 2);
        if (best < 0 || cost < best) {
            best = cost;
            a.splits = n;
            a.split_heads = heads;
        }
    }
    // sbf_dc: two blocks run on a unit
    const int64_t n = blocks >= 512 ? 1 : (512 + blocks - 1) / blocks < k ? (512 + blocks - 1) / blocks : k;
    a.dc_heads = (k + n - 1) / n;
    a.dc_splits = (k + a.dc_heads - 1) / a.dc_heads;
}

size_t lay_out(ScanBwdArgs& a, uint8_t* base) {
    size_t at = 0;
    auto part = [&](auto*& p, size_t n) {
        p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at);
        at += r256(n * sizeof(*p));
    };
    const size_t bhc = static_cast<size_t>(a.B * a.H * a.chunks);
    part(a.dA_part, bhc);
    part(a.through, bhc);
    part(a.decay, bhc * 5 * kFQ);
    part(a.starts, static_cast<size_t>(a.B * a.chunks) * kFQ);
    part(a.bounds, static_cast<size_t>(a.B * a.chunks));
    part(a.sums, bhc * (kSums * kFQ + kSumTail));
    part(a.states, bhc * a.P * a.N);
    part(a.grads, bhc * a.P * a.N);
    part(a.anchor, static_cast<size_t>(a.B * a.H * ((a.chunks + kAnchor - 1) / kAnchor)));
    const size_t slab = static_cast<size_t>(a.B * a.L * a.G * a.N), slabs = a.splits > 1 ? a.splits : 0;
    part(a.dB_head, slabs * slab);
    part(a.dC_head, (slabs + a.dc_splits) * slab);
    return at;
}

void set_up(ScanBwdArgs& a) {
    a.chunks = (a.L + kFQ - 1) / kFQ;
    cut_heads(a);
}

template <int N>
hipError_t launch_typed(const ScanBwdArgs& a, hipStream_t s) {
    const int64_t bh = a.B * a.H;
    sbf_decay_kernel<<<static_cast<uint32_t>(a.B * a.chunks * ((a.H + 15) / 16)), 256, 0, s>>>(a);
    // Walking over the chunks reads nothing twice but runs 2 B H blocks; else one block a chunk
    // and a pass over their shares (us of the whole call, walking / by chunk, dstate 128):
    // 4 x 8192 x 64 heads 1074 / 1462; 2 x 8192 x 48 525 / 582; 1 x 8192 x 64 419 / 404;
    // 1 x 8192 x 32 320 / 233; 1 x 32768 x 24, dstate 64, 806 / 383
    if (2 * bh >= 192 || a.chunks == 1) {
        sbf_states_kernel<N, true><<<dim3(static_cast<uint32_t>(bh), 2), 256, 0, s>>>(a);
    } else {
        sbf_states_kernel<N, false><<<dim3(static_cast<uint32_t>(bh * a.chunks), 2), 256, 0, s>>>(a);
        sbf_pass_kernel<<<dim3(static_cast<uint32_t>(bh * (kFP * N / 256)), 2), 256, 0, s>>>(a);
    }
    sbf_anchor_kernel<<<static_cast<uint32_t>(bh * ((a.chunks + kAnchor - 1) / kAnchor)), 256, 0, s>>>(a);
    sbf_dc_kernel<N><<<static_cast<uint32_t>(a.B * a.chunks * a.G * a.dc_splits), 512, 0, s>>>(a);
    sbf_grad_kernel<N><<<static_cast<uint32_t>(a.B * a.chunks * a.G * a.splits), 1024, 0, s>>>(a);
    if (a.splits > 1)
        sbf_join_kernel<<<dim3(static_cast<uint32_t>((a.B * a.L * a.G * N / 4 + 255) / 256), 2), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// 128 rows of tokens within 2^32 bytes: the lanes' offsets into a chunk have 32 bits
bool scan_bwd_mfma_supported(int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype) {
    const int64_t most = int64_t{1} << 23;
    return dtype == SSM_BF16 && P == kFP && (N == 64 || N == 128) && H <= most / P && G <= most / N;
}

size_t scan_bwd_mfma_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N) {
    ScanBwdArgs a{};
    a.B = B; a.L = L; a.H = H; a.P = P; a.G = G; a.N = N;
    set_up(a);
    return lay_out(a, nullptr);
}

hipError_t launch_scan_bwd_mfma(ScanBwdArgs a, void* workspace, hipStream_t s) {
    set_up(a);
    lay_out(a, static_cast<uint8_t*>(workspace));
    const hipError_t e = a.N == 128 ? launch_typed<128>(a, s) : launch_typed<64>(a, s);
    return e == hipSuccess ? launch_scan_bwd_ddt(a, kFQ, s) : e;
}

}  // namespace ssm
