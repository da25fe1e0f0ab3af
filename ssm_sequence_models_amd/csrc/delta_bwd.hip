// delta_bwd.hip -- the gated delta rule's backward.  With the chunk's quantities of delta.h, dh the
// gradient of the state after the chunk and dY' = scale dY:
//     dU = M^T dY + e^{G_Q - G} K dh^T,   dZ = T^T (b dU),   dV = dZ
//     dh_0 = e^{G_Q} dh + (e^G dY')^T Q - (e^G dZ)^T K
//     X_ts = r_ts scale (dY_t . U_s) (s <= t),   F_ts = -r_ts b_s (dZ_t . E_s) (s < t)
//     dQ = e^G dY' h_0 + X K
//     dK = e^{G_Q - G} U dh - e^G dZ h_0 + X^T Q + F^T K + F K
//     db_s = dU_s . E_s - sum_t r_ts (k_t . k_s) (dZ_t . E_s)
//     dgate_t: every product whose factor e^(..) spans token t, times itself: pairs s < t <= t',
//              h_0 to t' >= t, s < t to the chunk's end, h_0 to the end
//
//   delta_walk   (delta.hip) along the rows again: the state before every chunk, and E
//   delta_back   from the last chunk to the first: dh before every chunk, dZ, and of the channels'
//                sums dU . E and e^{G_Q - G} (K dh^T) . U; laid out as the walk
//   delta_grad   one block a chunk and key head (and range of its heads): dQ, dK, and of dbeta and dgate
//                what the pairs and the states give
//   delta_gate   a wavefront a chunk and head: dbeta, and dgate's sums along the chunk
#include <type_traits>

#include "delta.h"

namespace ssm {
namespace {

using namespace delta;

constexpr int kGradWaves = 8;

struct Buffers {
    DeltaSaved saved;
    float* grads;  // [B, H, chunks, P, N]: the gradient of the state after each chunk
    float* dz;     // [B, L, H, P]
    float* part;   // [B, H, chunks, 16-channel tiles, 2, Q]
    float* gate;   // [B, H, chunks, 4, Q]: for dgate and dbeta, what delta_gate sums over a chunk's tokens
    float* dqk;    // [2, splits, B, L, G, N] where the heads of a key head are split
    int64_t splits, heads;  // ranges of a key head's heads, and heads in each
};

__device__ __forceinline__ float sum_groups(float v) {  // over the four lanes that share li
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ f4 row4(const float* p) { return lds<f4>(reinterpret_cast<const uint8_t*>(p)); }

// Laid out as the walk (delta.hip), from the last chunk to the first; E comes and dZ goes by the wavefronts
// that use them (LDS is full).
// Bound by the chain of a chunk's products with one such wavefront a SIMD (matrix instructions busy 24 % of it,
// vector ones 32 %) and by the 3.4 GB that it moves, dh and dZ out, E and the images of T and M in, at 4.2 TB/s:
// 4 x 8192 x 32 heads x 128 x 128, bf16, 800 to 840 us for 128 chunks.
template <class MM, int NT>
struct BackLds {
    static constexpr int W = 16 * NT, HALVES = NT <= 8 ? 2 : 1;
    static constexpr int V = 0, K = V + staged_bytes<MM, 64>(), T = K + staged_bytes<MM, W>(), F = T + image_bytes<MM>(MM::TP),
                         Qq = F + 1024, M = Qq + staged_bytes<MM, W>(), HALF = M + image_bytes<MM>(MM::TP);
};

// SPAN: a segment from zero, only the gradient of the state before it
template <class MM, int NT, bool SPAN, bool DIRECT>
__global__ __launch_bounds__(320) void delta_back_kernel(DeltaArgs a, Buffers u) {
    using S = typename MM::S;
    using O = BackLds<MM, NT>;
    constexpr int Q = MM::Q, RT = Q / 16, KT = Q / MM::KB, W = 16 * NT, KN = W / MM::KB, TP = MM::TP;
    __shared__ __attribute__((aligned(1024))) uint8_t sm[O::HALVES * O::HALF];
    const int lane = threadIdx.x & 63, li = lane & 15, g4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int H = static_cast<int>(a.H), P = static_cast<int>(a.P), N = static_cast<int>(a.N);
    const int pblocks = (P + 63) / 64, ptiles = (P + 15) / 16;
    const int unit = xcd_order(blockIdx.x, gridDim.x);
    const int segs = static_cast<int>(a.segs), pb = unit % pblocks, seg = unit / pblocks % segs, bh = unit / pblocks / segs;
    const int h = bh % H, b = bh / H, g = h / (H / static_cast<int>(a.G));
    const int chunks = static_cast<int>(a.chunks), c0 = seg * static_cast<int>(a.seg_chunks);
    const int c1 = c0 + static_cast<int>(a.seg_chunks) < chunks ? c0 + static_cast<int>(a.seg_chunks) : chunks;
    const auto rows_of = [&](int c) {
        const int64_t left = a.L - static_cast<int64_t>(c) * Q;
        return static_cast<int>(left < Q ? left : Q);
    };
    const auto half_of = [&](int c) { return sm + (O::HALVES == 2 ? (c & 1) * O::HALF : 0); };
    const auto marks_of = [&](const uint8_t* half) {
        return __builtin_amdgcn_readfirstlane(static_cast<int>(reinterpret_cast<const float*>(half + O::F)[4 * Q - 1]));
    };

    if (w == 4) {
        const int64_t col = static_cast<int64_t>(h) * P + 64 * pb;
        const int width = P - 64 * pb < 64 ? P - 64 * pb : 64;
        const auto fetch = [&](int c) {
            uint8_t* const half = half_of(c);
            const int64_t t0 = b * a.L + static_cast<int64_t>(c) * Q, image = static_cast<int64_t>(bh) * chunks + c;
            const int valid = rows_of(c);
            if (DIRECT) {
                direct_rows<MM, W, true>(half + O::K, token_buffer<S>(a.k, t0, a.k_row, g * N, valid, N), static_cast<int>(a.k_row), N, lane);
                direct_rows<MM, W, true>(half + O::Qq, token_buffer<S>(a.q, t0, a.q_row, g * N, valid, N), static_cast<int>(a.q_row), N, lane);
                direct_rows<MM, 64, false>(half + O::V, token_buffer<S>(a.dy, t0, a.dy_row, col, valid, width), static_cast<int>(a.dy_row), width, lane);
            } else {
                stage_rows<MM, W, 64, true>(half + O::K, static_cast<const S*>(a.k) + t0 * a.k_row + g * N, a.k_row, valid, N);
                stage_rows<MM, W, 64, true>(half + O::Qq, static_cast<const S*>(a.q) + t0 * a.q_row + g * N, a.q_row, valid, N);
                stage_elements<MM, 64>(half + O::V, static_cast<const S*>(a.dy) + t0 * a.dy_row + col, a.dy_row, valid, width);
            }
            direct_image<image_bytes<MM>(MM::TP)>(half + O::T, a.Tt + image * image_bytes<MM>(MM::TP), lane);
            direct_image<image_bytes<MM>(MM::TP)>(half + O::M, a.M + image * image_bytes<MM>(MM::TP), lane);
            direct_image<kFactors * Q * 4>(half + O::F, reinterpret_cast<const uint8_t*>(a.factors + image * kFactors * Q), lane);
        };
        if (O::HALVES == 2) fetch(c1 - 1);
        for (int c = c1 - 1; c >= c0; --c) {
            if (O::HALVES == 1) {
                __syncthreads();
                fetch(c);
            }
            wait_loads();
            __syncthreads();
            if (O::HALVES == 2 && c > c0) fetch(c - 1);
            if (marks_of(half_of(c)) >= static_cast<int>(kNotFinite)) {
                __syncthreads();
                __syncthreads();
            }
        }
        return;
    }

    const int p0 = 64 * pb + 16 * w, p = p0 + li;
    const bool mine = p0 < P, have = p < P;
    const int64_t erow = static_cast<int64_t>(H) * P, bhs = static_cast<int64_t>(bh) * segs + seg;
    const float* const from = SPAN ? nullptr : segs > 1 ? a.entry + (bhs * P + p) * N : a.dhT ? a.dhT + (static_cast<int64_t>(bh) * P + p) * N : nullptr;
    float* const dest = SPAN ? a.gain + (bhs * P + p) * N : a.dh0 && seg == 0 ? a.dh0 + (static_cast<int64_t>(bh) * P + p) * N : nullptr;
    const uint32_t eat = have ? 4 * g4 * static_cast<uint32_t>(erow) * 4 + p * 4 : kOutside;
    float en[RT][4];  // the next chunk's E
    const auto fetch_e = [&](int c) {
        const int64_t t0 = b * a.L + static_cast<int64_t>(c) * Q;
        const int valid = rows_of(c);
        const Buffer re = token_buffer<float>(u.saved.e, t0, erow, static_cast<int64_t>(h) * P, DIRECT ? valid : 1, P);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 16 * i + 4 * g4 + e;
                if (DIRECT) en[i][e] = load_at<float>(re, eat + (16 * i + e) * static_cast<uint32_t>(erow) * 4);
                else en[i][e] = have && t < valid ? u.saved.e[(t0 + t) * erow + static_cast<int64_t>(h) * P + p] : 0.0f;
            }
    };
    f4 dh[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = MM::state_row(i, g4);
        dh[i] = have && n < N && from ? *reinterpret_cast<const f4*>(from + n) : f4{0, 0, 0, 0};
    }
    if (!SPAN) fetch_e(c1 - 1);
    for (int c = c1 - 1; c >= c0; --c) {
        const int64_t t0 = b * a.L + static_cast<int64_t>(c) * Q, image = static_cast<int64_t>(bh) * chunks + c;
        const int valid = rows_of(c);
        uint8_t* const half = half_of(c);
        if (O::HALVES == 1) __syncthreads();
        __syncthreads();
        f4 ev[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) ev[i][e] = SPAN ? 0.0f : en[i][e];
        if (!SPAN && c > c0) fetch_e(c - 1);
        if (!SPAN && have) {
            float* to = u.grads + image * P * N + static_cast<int64_t>(p) * N;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int n = MM::state_row(i, g4);
                if (n < N) *reinterpret_cast<f4*>(to + n) = dh[i];
            }
        }
        uint8_t* const sk = half + O::K;
        uint8_t* const sq = half + O::Qq;
        const float* const sf = reinterpret_cast<const float*>(half + O::F);
        const int marks = marks_of(half);
        const bool clean = marks < static_cast<int>(kNotFinite);
        if (clean && !mine) continue;
        const auto chunk = [&](auto with_starts) __attribute__((always_inline)) {
            constexpr bool STARTS = decltype(with_starts)::value;
            f4 du[RT], dz[RT], dy[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                du[i] = dz[i] = f4{0, 0, 0, 0};
                dy[i] = MM::template four_rows<64>(half + O::V, 16 * i, w, li, g4);
            }
            // e^{G_Q - G} K dh^T, and its products with U
#pragma unroll
            for (int kk = 0; kk < KN; ++kk) {
                const auto s = MM::template of_state<3>(dh, kk, g4);
#pragma unroll
                for (int i = 0; i < RT; ++i) MM::template mac<1, 3>(du[i], MM::template state_rows<W>(sk, 16 * i, kk, li, g4), s);
            }
            float* part = u.part + (image * ptiles + p0 / 16) * 2 * Q + 4 * g4 + li;
            scale_rows<STARTS>(du, sf + Q, 1.0f, g4);
#pragma unroll
            for (int i = 0; i < (SPAN ? 0 : RT); ++i) {
                const f4 v = du[i] * ev[i] * row4(sf + 2 * Q + 16 * i + 4 * g4);
                const float s = row_sums({v[0], v[1], v[2], v[3]}, li);
                if (mine && li < 4) part[Q + 16 * i] = s;
            }
            // dU += M^T dY
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const auto s = finite_tiles<MM, 1, STARTS>(dy, kk);
#pragma unroll
                for (int i = 0; i < (kk + 1) * MM::KB / 16; ++i)
                    MM::template mac<TP, 1>(du[i], frag<MM, TP>(half + O::M, frag_at<MM>(i, kk, true), lane), s);
            }
            mark_sequences<STARTS, Q>(du, dy, sf + 3 * Q, lane);
#pragma unroll
            for (int i = 0; i < (SPAN ? 0 : RT); ++i) {
                const f4 v = du[i] * ev[i];
                const float s = row_sums({v[0], v[1], v[2], v[3]}, li);
                if (mine && li < 4) part[16 * i] = s;
            }
            // dZ = T^T (b dU)
            scale_rows<false>(du, sf + 2 * Q, 1.0f, g4);
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const auto s = finite_tiles<MM, 3, STARTS>(du, kk);
#pragma unroll
                for (int i = 0; i < (kk + 1) * MM::KB / 16; ++i)
                    MM::template mac<TP, 3>(dz[i], frag<MM, TP>(half + O::T, frag_at<MM>(i, kk, true), lane), s);
            }
            mark_sequences<STARTS, Q>(dz, du, sf + 3 * Q, lane);
            const Buffer rz = token_buffer<float>(u.dz, t0, erow, static_cast<int64_t>(h) * P, DIRECT ? valid : 1, P);
#pragma unroll
            for (int i = 0; i < (SPAN ? 0 : RT); ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * i + 4 * g4 + e;
                    if (DIRECT) store_at<float>(rz, eat + (16 * i + e) * static_cast<uint32_t>(erow) * 4, dz[i][e]);
                    else if (have && t < valid) u.dz[(t0 + t) * erow + static_cast<int64_t>(h) * P + p] = dz[i][e];
                }
            // the gradient of the state before the chunk
            if (STARTS && !clean) {
                __syncthreads();
                clear_rows<MM, W>(sk, sf);
                clear_rows<MM, W>(sq, sf);
                __syncthreads();
            }
            scale_state<STARTS>(dh, sf[Q - 1]);
            scale_rows<STARTS>(dy, sf, a.scale, g4);
            scale_rows<STARTS>(dz, sf, -1.0f, g4);
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const auto sy = MM::template of_tiles<3>(dy, kk);
                const auto sz = MM::template of_tiles<3>(dz, kk);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    MM::template mac<1, 3>(dh[i], MM::template state_columns<W>(sq, kk * MM::KB, i, li, g4), sy);
                    MM::template mac<1, 3>(dh[i], MM::template state_columns<W>(sk, kk * MM::KB, i, li, g4), sz);
                }
            }
        };
        if (marks != 0) chunk(std::true_type{});
        else chunk(std::false_type{});
    }
    if (dest && have) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = MM::state_row(i, g4);
            if (n < N) *reinterpret_cast<f4*>(dest + n) = dh[i];
        }
    }
}

// ---------------------------------------------------------------------------------------
// delta_grad: eight wavefronts a block; a wavefront owns columns of dQ and dK (state dimensions) and
// reads of h_0 and dh each element once, and takes tiles of the pairs in turn.  dY, dZ and E pass
// through LDS in blocks of 64 channels; dQ and dK are summed over the heads of a key head in
// accumulators.
// fp32 operands go in three bf16 parts, which hold all of their 24 bits, or whole.
// Bound by its waits and vector work: 1370 to 1470 us at 4 x 8192 x 32 heads of 16 key heads x 128 x 128, bf16 (matrix
// instructions busy 25 %, vector ones 46 %; it moves 4.3 GB, h_0, dh, E and dZ the most of them, at 3.0 TB/s).  With
// X, F, E and dh of dk in two parts, which lose what bf16's rounding does not hide where terms cancel, 1250 to 1400.
// Four wavefronts a block: 1.3 times slower.  LDS addresses are formed where they are used (`here`): kept over the
// loops they cost as much again in spilled registers.
// ---------------------------------------------------------------------------------------
template <class MM>
__device__ __forceinline__ void store_values(typename MM::S* p, int n, const float (&v)[MM::R]) {
    if (n >= MM::R) {
        if constexpr (MM::R == 8)
            *reinterpret_cast<u4any*>(p) = u4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        else
            *reinterpret_cast<u4any4*>(p) = __builtin_bit_cast(u4, f4{v[0], v[1], v[2], v[3]});
    } else {
#pragma unroll
        for (int j = 0; j < MM::R; ++j)
            if (j < n) MM::store(p, j, v[j]);
    }
}
// R values into PARTS tiles
template <class MM, int W, int PARTS>
__device__ __forceinline__ void put_parts(uint8_t* tiles, int bytes, int row, int q, const float (&v)[MM::R]) {
    if constexpr (MM::TP == 1) {
        *reinterpret_cast<f4*>(tiles + MM::template piece_at<W>(row, q)) = f4{v[0], v[1], v[2], v[3]};
    } else {
        const auto f = MM::template parts<PARTS>(v);
#pragma unroll
        for (int i = 0; i < PARTS; ++i) *reinterpret_cast<bf8*>(tiles + i * bytes + MM::template piece_at<W>(row, q)) = f.p[i];
    }
}
// one value of a pair into PARTS tiles
template <class MM, int PARTS>
__device__ __forceinline__ void put_pair(uint8_t* tiles, int bytes, int row, int col, float v) {
    if constexpr (MM::TP == 1) {
        *reinterpret_cast<float*>(tiles + (row * (MM::Q + 4) + col) * 4) = v;
    } else {
        const int at = piece<2 * MM::Q>(row, col >> 3) + 2 * (col & 7);
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            const uint16_t h = f32_to_bf16(v);
            *reinterpret_cast<uint16_t*>(tiles + i * bytes + at) = h;
            v -= bf16_to_f32(h);
        }
    }
}

template <class MM, int NT, bool DIRECT>
__global__ __launch_bounds__(64 * kGradWaves) void delta_grad_kernel(DeltaArgs a, Buffers u) {
    using S = typename MM::S;
    constexpr int Q = MM::Q, RT = Q / 16, KT = Q / MM::KB, W = 16 * NT, KN = W / MM::KB, KP = 64 / MM::KB, R = MM::R;
    constexpr int WV = kGradWaves, CG = NT < WV ? NT : WV, RG = WV / CG;  // column and row groups of wavefronts
    constexpr int CT = NT / CG, RW = RT / RG;           // a wavefront's column and row tiles
    constexpr int TILES = RT * (RT + 1) / 2, MINE = (TILES + WV - 1) / WV;
    constexpr int TP = MM::TP;
    constexpr int QN = staged_bytes<MM, W>(), QP = MM::template tile_bytes<64>(Q), QQ = MM::template tile_bytes<Q>(Q);
    constexpr int LOADS = (1 + 2 * TP) * QP, PAIRS = 3 * TP * QQ;
    __shared__ __attribute__((aligned(16))) uint8_t sk[QN];
    __shared__ __attribute__((aligned(16))) uint8_t sq[QN];
    __shared__ __attribute__((aligned(16))) uint8_t pool[LOADS > PAIRS ? LOADS : PAIRS];
    __shared__ __attribute__((aligned(16))) float sf[kFactors * Q];  // plane 3: sequences begun
    __shared__ double sg[Q];
    __shared__ float sdb[RT][Q];    // sums over t of pairs, by row tiles
    __shared__ float sc[CG][Q];     // products with h_0, by column groups
    __shared__ float sspan[Q];
    __shared__ float sdot[WV];
    uint8_t* const ty = pool;                   // dY
    uint8_t* const tz = pool + QP;              // dZ
    uint8_t* const te = pool + (1 + TP) * QP;   // E
    uint8_t* const tx = pool;                   // X
    uint8_t* const tf = pool + TP * QQ;         // F
    uint8_t* const tw = pool + 2 * TP * QQ;     // the pairs' products themselves
    const int tid = threadIdx.x, lane = tid & 63, li_ = lane & 15, g4_ = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), cg = w % CG, rg = RG == 1 ? 0 : w / CG;
    int64_t unit = xcd_order(blockIdx.x, gridDim.x);
    const int64_t split = unit % u.splits;
    unit /= u.splits;
    const int64_t g = unit % a.G;
    unit /= a.G;
    const int64_t c = unit % a.chunks, b = unit / a.chunks;
    const int64_t rep = a.H / a.G;
    const int64_t h1 = g * rep + (rep < (split + 1) * u.heads ? rep : (split + 1) * u.heads);
    const int valid = static_cast<int>(a.L - c * Q < Q ? a.L - c * Q : Q);
    const int N = static_cast<int>(a.N), P = static_cast<int>(a.P);
    const int64_t t0 = b * a.L + c * Q;

    if (DIRECT) {  // on their way while the first loads below are issued; waited for at the head's first barrier
        direct_rows<MM, W, false, WV>(sk, token_buffer<S>(a.k, t0, a.k_row, g * a.N, valid, N), static_cast<int>(a.k_row), N, lane, w);
        direct_rows<MM, W, false, WV>(sq, token_buffer<S>(a.q, t0, a.q_row, g * a.N, valid, N), static_cast<int>(a.q_row), N, lane, w);
    } else {
        stage_rows<MM, W, 64 * WV, false>(sk, static_cast<const S*>(a.k) + t0 * a.k_row + g * a.N, a.k_row, valid, N);
        stage_rows<MM, W, 64 * WV, false>(sq, static_cast<const S*>(a.q) + t0 * a.q_row + g * a.N, a.q_row, valid, N);
    }
    f4 dq[RW][CT], dk[RW][CT];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) dq[i][j] = dk[i][j] = f4{0, 0, 0, 0};

    // what a thread stages of 64 channels of a head, and what a lane takes of h_0 and dh, are loaded
    // one block of channels ahead
    constexpr int PT = Q * 64 / R / (64 * WV);  // pieces of the tokens' tiles a thread
    const int sq8 = tid % (64 / R);
    const auto srow = [&](int i) { return (tid + 64 * WV * i) / (64 / R); };
    u4 ny[PT];
    f4 nz[PT][R / 4], ne[PT][R / 4];
    float ns[KP][CT][R], nd[KP][CT][R];
    const auto load_tokens = [&](int64_t h, int p0) {
        const int p = p0 + R * sq8;
        const Buffer ry = token_buffer<S>(a.dy, t0, a.dy_row, h * a.P, DIRECT ? valid : 1, a.P);
        const Buffer rz = token_buffer<float>(u.dz, t0, a.H * a.P, h * a.P, DIRECT ? valid : 1, a.P);
        const Buffer re = token_buffer<float>(u.saved.e, t0, a.H * a.P, h * a.P, DIRECT ? valid : 1, a.P);
#pragma unroll
        for (int x = 0; x < PT; ++x) {
            const int row = srow(x);
            if constexpr (DIRECT) {
                const uint32_t ya = p < P ? (row * static_cast<uint32_t>(a.dy_row) + p) * sizeof(S) : kOutside;
                const uint32_t za = p < P ? (row * static_cast<uint32_t>(a.H * a.P) + p) * 4 : kOutside;
                ny[x] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(ry, ya, 0, 0));
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    nz[x][i] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rz, za + 16 * i, 0, 0));
                    ne[x][i] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(re, za + 16 * i, 0, 0));
                }
            } else {
                const int left = row < valid ? P - p : 0;
                const int64_t at = ((t0 + row) * a.H + h) * a.P + p;
                const S* y = static_cast<const S*>(a.dy) + (t0 + row) * a.dy_row + h * a.P + p;
                S v[R];
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    v[j] = j < left ? y[j] : S{0};
                    nz[x][j >> 2][j & 3] = j < left ? u.dz[at + j] : 0.0f;
                    ne[x][j >> 2][j & 3] = j < left ? u.saved.e[at + j] : 0.0f;
                }
                __builtin_memcpy(&ny[x], v, 16);
            }
        }
    };
    const auto load_states = [&](int64_t h, int p0) {
        const int li = here(li_), g4 = here(g4_);
        const int64_t image = (b * a.H + h) * a.chunks + c;
        const Buffer rs = buffer(u.saved.states + image * P * N, static_cast<int64_t>(P) * N * 4);
        const Buffer rd = buffer(u.grads + image * P * N, static_cast<int64_t>(P) * N * 4);
#pragma unroll
        for (int kk = 0; kk < KP; ++kk)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int n = 16 * (cg * CT + j) + li;
                const uint32_t at = n < N ? ((p0 + MM::KB * kk + R * g4) * N + n) * 4 : kOutside;
#pragma unroll
                for (int m = 0; m < R; ++m) {
                    ns[kk][j][m] = load_at<float>(rs, at + m * N * 4);
                    nd[kk][j][m] = load_at<float>(rd, at + m * N * 4);
                }
            }
    };
    float nf = 0.0f;
    double ng = 0.0;
    const auto load_factors = [&](int64_t h) {
        const int64_t image = (b * a.H + h) * a.chunks + c;
        if (tid < kFactors * Q) nf = a.factors[image * kFactors * Q + tid];
        if (tid < Q) ng = a.gates[image * Q + tid];
    };
    int trow[MINE], tcol[MINE];  // this wavefront's tiles of the pairs, row tiles from the first on
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
        tcol[m] = w + WV * m;
        trow[m] = 0;
        while (tcol[m] > trow[m]) tcol[m] -= ++trow[m];
    }
    const int64_t h0 = g * rep + split * u.heads;
    load_factors(h0);
    load_tokens(h0, 0);
    load_states(h0, 0);
    if (DIRECT) wait_loads();
    for (int64_t h = h0; h < h1; ++h) {
        const int64_t image = (b * a.H + h) * a.chunks + c;
        f4 qo[RW][CT], ko[RW][CT], ke[RW][CT], dm[MINE], db[MINE];
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) qo[i][j] = ko[i][j] = ke[i][j] = f4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < MINE; ++i) dm[i] = db[i] = f4{0, 0, 0, 0};
        float dot = 0.0f;
        for (int p0 = 0; p0 < P; p0 += 64) {
            __syncthreads();
            if (p0 == 0) {
                if (tid < kFactors * Q) sf[tid] = nf;
                if (tid < Q) sg[tid] = ng;
            }
#pragma unroll
            for (int x = 0; x < PT; ++x) {
                const int row = srow(x);
                *reinterpret_cast<u4*>(ty + MM::template piece_at<64>(row, sq8)) = ny[x];
                float z[R], e[R];
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    z[j] = nz[x][j >> 2][j & 3];
                    e[j] = ne[x][j >> 2][j & 3];
                }
                put_parts<MM, 64, TP>(tz, QP, row, sq8, z);
                put_parts<MM, 64, TP>(te, QP, row, sq8, e);
                if (DIRECT) {
                    if (row < valid && p0 + R * sq8 < P) store_values<MM>(static_cast<S*>(a.dv) + (t0 + row) * a.dv_row + h * a.P + p0 + R * sq8, R, z);
                } else {
                    store_values<MM>(static_cast<S*>(a.dv) + (t0 + row) * a.dv_row + h * a.P + p0 + R * sq8, row < valid ? P - p0 - R * sq8 : 0, z);
                }
            }
            const bool same = p0 + 64 < P;
            const int64_t hn = same ? h : h + 1;
            if (hn < h1) {
                load_tokens(hn, same ? p0 + 64 : 0);
                if (!same) load_factors(hn);
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < KP; ++kk) {
                const int li = here(li_), g4 = here(g4_);
                typename MM::template Frag<3> fs[CT];
                typename MM::template Frag<3> fd[CT];
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    if (rg == 0) {
#pragma unroll
                        for (int m = 0; m < R; ++m) dot += ns[kk][j][m] * nd[kk][j][m];
                    }
                    fs[j] = MM::template parts<3>(ns[kk][j]);
                    fd[j] = MM::template parts<3>(nd[kk][j]);
                }
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const int r0 = 16 * (rg * RW + i);
                    const auto y = MM::template along<64>(ty, r0, kk, li, g4);
                    const auto z = of_parts<MM, TP>([&](int q) { return MM::template along<64>(tz + q * QP, r0, kk, li, g4); });
                    const auto e = of_parts<MM, TP>([&](int q) { return MM::template along<64>(te + q * QP, r0, kk, li, g4); });
#pragma unroll
                    for (int j = 0; j < CT; ++j) {
                        MM::template mac<1, 3>(qo[i][j], y, fs[j]);
                        MM::template mac<TP, 3>(ko[i][j], z, fs[j]);
                        MM::template mac<TP, 3>(ke[i][j], e, fd[j]);
                    }
                }
            }
            if (hn < h1) load_states(hn, same ? p0 + 64 : 0);
#pragma unroll
            for (int m = 0; m < MINE; ++m) {
                if (w + WV * m >= TILES) continue;
                const int tile = tcol[m], rt = trow[m];
                const int li = here(li_), g4 = here(g4_);
#pragma unroll
                for (int kk = 0; kk < KP; ++kk) {
                    const auto e = of_parts<MM, TP>([&](int q) { return MM::template along<64>(te + q * QP, 16 * tile, kk, li, g4); });
                    MM::template mac<1, TP>(dm[m], MM::template along<64>(ty, 16 * rt, kk, li, g4), e);
                    const auto z = of_parts<MM, TP>([&](int q) { return MM::template along<64>(tz + q * QP, 16 * rt, kk, li, g4); });
                    MM::template mac<TP, TP>(db[m], z, e);
                }
            }
        }
        __syncthreads();  // the loads' tiles become the pairs'
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
            if (w + WV * m >= TILES) continue;
            const int tile = tcol[m], rt = trow[m];
            const int li = here(li_), g4 = here(g4_);
            f4 kk{0, 0, 0, 0}, qk{0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < KN; ++x) {
                const auto s = MM::template along<W>(sk, 16 * tile, x, li, g4);
                MM::template mac<1, 1>(kk, MM::template along<W>(sk, 16 * rt, x, li, g4), s);
                MM::template mac<1, 1>(qk, MM::template along<W>(sq, 16 * rt, x, li, g4), s);
            }
            const int s = 16 * tile + li;
            const float be = sf[2 * Q + s];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 16 * rt + 4 * g4 + e;
                const bool one = sf[3 * Q + s] == sf[3 * Q + t], on = one && s <= t, below = one && s < t;
                const float r = exp_of(sg[t] - sg[s]);
                const float x = on ? r * a.scale * be * dm[m][e] : 0.0f;
                const float f = below ? -r * db[m][e] : 0.0f;
                const float pair = below ? x * qk[e] + f * be * kk[e] : 0.0f;
                sum += below ? f * kk[e] : 0.0f;
                put_pair<MM, TP>(tx, QQ, t, s, x);
                put_pair<MM, TP>(tf, QQ, t, s, f * be);
                put_pair<MM, TP>(tw, QQ, t, s, pair);
                if (MM::KB == 32 && (rt & 1) && tile == rt - 1) {  // above the diagonal, in its contraction block
                    put_pair<MM, TP>(tx, QQ, t - 16, s + 16, 0.0f);
                    put_pair<MM, TP>(tf, QQ, t - 16, s + 16, 0.0f);
                    put_pair<MM, TP>(tw, QQ, t - 16, s + 16, 0.0f);
                }
            }
            sum = sum_groups(sum);
            if (g4 == 0) sdb[rt][s] = sum;
        }
        // products with h_0, for dgate
        const bool several = sf[4 * Q - 1] != 0.0f;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int li = here(li_), g4 = here(g4_);
            const int r0 = 16 * (rg * RW + i) + 4 * g4;
            const f4 f = row4(sf + r0);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                qo[i][j] *= f * a.scale;
                ko[i][j] *= -f;
                if (several) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        qo[i][j][e] = f[e] != 0.0f ? qo[i][j][e] : 0.0f;
                        ko[i][j][e] = f[e] != 0.0f ? ko[i][j][e] : 0.0f;
                    }
                }
                const f4 q4 = MM::template four_rows<W>(sq, 16 * (rg * RW + i), cg * CT + j, li, g4);
                const f4 k4 = MM::template four_rows<W>(sk, 16 * (rg * RW + i), cg * CT + j, li, g4);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += qo[i][j][e] * q4[e] + ko[i][j][e] * k4[e];
            }
            const float sum = row_sums(v, li);
            if (li < 4) sc[cg][r0 + li] = sum;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
        if (lane == 0) sdot[w] = dot;
        __syncthreads();
        if (w < RT) {  // pairs that span token t = 16 w + li
            const int li = here(li_), g4 = here(g4_);
            float span = 0.0f;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if (rt < w) continue;
                f4 v{0, 0, 0, 0};
#pragma unroll
                for (int kk = 0; kk < KT; ++kk) {
                    if (kk * MM::KB > 16 * w) continue;
                    float one[R];
#pragma unroll
                    for (int j = 0; j < R; ++j)
                        one[j] = MM::KB * kk + (j >> 2) * 16 + 4 * g4 + (j & 3) < 16 * w + li ? 1.0f : 0.0f;
                    const auto l = of_parts<MM, TP>([&](int q) { return MM::template rows<Q>(tw + q * QQ, 16 * rt, kk, li, g4); });
                    MM::template mac<TP, 1>(v, l, MM::template parts<1>(one));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) span += 16 * rt + 4 * g4 + e >= 16 * w + li ? v[e] : 0.0f;
            }
            span = sum_groups(span);
            if (g4 == 0) sspan[16 * w + li] = span;
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int li = here(li_), g4 = here(g4_);
            const int rt = rg * RW + i;
            const f4 f = row4(sf + Q + 16 * rt + 4 * g4) * row4(sf + 2 * Q + 16 * rt + 4 * g4);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int ct = cg * CT + j;
                dq[i][j] += qo[i][j];
#pragma unroll
                for (int e = 0; e < 4; ++e) dk[i][j][e] += ko[i][j][e] + (several && f[e] == 0.0f ? 0.0f : f[e] * ke[i][j][e]);
#pragma unroll
                for (int kk = 0; kk < KT; ++kk) {
                    const auto fk = MM::template columns<W>(sk, kk * MM::KB, ct, li, g4);
                    const auto fq = MM::template columns<W>(sq, kk * MM::KB, ct, li, g4);
                    if (kk * MM::KB <= 16 * rt) {
                        const auto x = of_parts<MM, TP>([&](int q) { return MM::template rows<Q>(tx + q * QQ, 16 * rt, kk, li, g4); });
                        MM::template mac<TP, 1>(dq[i][j], x, fk);
                        const auto y = of_parts<MM, TP>([&](int q) { return MM::template rows<Q>(tf + q * QQ, 16 * rt, kk, li, g4); });
                        MM::template mac<TP, 1>(dk[i][j], y, fk);
                    }
                    if ((kk + 1) * MM::KB > 16 * rt) {
                        const auto x = of_parts<MM, TP>([&](int q) { return MM::template columns<Q>(tx + q * QQ, kk * MM::KB, rt, li, g4); });
                        MM::template mac<TP, 1>(dk[i][j], x, fq);
                        const auto y = of_parts<MM, TP>([&](int q) { return MM::template columns<Q>(tf + q * QQ, kk * MM::KB, rt, li, g4); });
                        MM::template mac<TP, 1>(dk[i][j], y, fk);
                    }
                }
            }
        }
        __syncthreads();
        if (tid < Q) {
            float from = 0.0f, be = 0.0f, all = 0.0f;
#pragma unroll
            for (int i = 0; i < CG; ++i) from += sc[i][tid];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) be += rt >= tid / 16 ? sdb[rt][tid] : 0.0f;
#pragma unroll
            for (int i = 0; i < WV; ++i) all += sdot[i];
            const float through = sf[Q - 1];
            float* to = u.gate + image * 4 * Q + tid;
            to[0] = from;
            to[Q] = sspan[tid];
            to[2 * Q] = be;
            to[3 * Q] = through != 0.0f ? through * all : 0.0f;
        }
    }
    const int li = li_, g4 = g4_;
    if (u.splits == 1) {
        const Buffer rq = token_buffer<S>(a.dq, t0, a.dq_row, g * a.N, DIRECT ? valid : 1, a.N);
        const Buffer rk = token_buffer<S>(a.dk, t0, a.dk_row, g * a.N, DIRECT ? valid : 1, a.N);
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int n = 16 * (cg * CT + j) + li;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * (rg * RW + i) + 4 * g4 + e;
                    if (DIRECT) {
                        store_at<S>(rq, n < N ? (t * static_cast<uint32_t>(a.dq_row) + n) * sizeof(S) : kOutside, dq[i][j][e]);
                        store_at<S>(rk, n < N ? (t * static_cast<uint32_t>(a.dk_row) + n) * sizeof(S) : kOutside, dk[i][j][e]);
                    } else if (t < valid && n < N) {
                        MM::store(static_cast<S*>(a.dq) + (t0 + t) * a.dq_row + g * a.N, n, dq[i][j][e]);
                        MM::store(static_cast<S*>(a.dk) + (t0 + t) * a.dk_row + g * a.N, n, dk[i][j][e]);
                    }
                }
            }
    } else {
        const int64_t part = a.B * a.L * a.G * a.N;
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int n = 16 * (cg * CT + j) + li;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * (rg * RW + i) + 4 * g4 + e;
                    if (t >= valid || n >= N) continue;
                    float* to = u.dqk + split * part + ((t0 + t) * a.G + g) * a.N + n;
                    to[0] = dq[i][j][e];
                    to[u.splits * part] = dk[i][j][e];
                }
            }
    }
}

// dbeta, and dgate_t = sum of the products with h_0 of t and later tokens + the pairs that span t + sum of
// the products with dh of tokens before t + the states' own product
template <int Q>
__global__ __launch_bounds__(256) void delta_gate_kernel(DeltaArgs a, Buffers u) {
    const int lane = threadIdx.x & 63;
    const int64_t image = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (image >= a.B * a.H * a.chunks) return;
    const int64_t c = image % a.chunks, bh = image / a.chunks, h = bh % a.H, b = bh / a.H;
    const int64_t t = c * Q + lane, ptiles = (a.P + 15) / 16;
    const bool have = lane < Q && t < a.L;
    double from = 0.0, end = 0.0;
    float be = 0.0f, rest = 0.0f;
    if (have) {
        const float* part = u.part + image * ptiles * 2 * Q + lane;
        const float* g = u.gate + image * 4 * Q + lane;
        from = g[0];
        rest = g[Q] + g[3 * Q];
        be = g[2 * Q];
#pragma unroll 8
        for (int i = 0; i < ptiles; ++i) {
            be += part[i * 2 * Q];
            end += part[i * 2 * Q + Q];
        }
    }
    const double own = end;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_down(from, d), e = __shfl_up(end, d);
        if (lane + d < 64) from += o;
        if (lane >= d) end += e;
    }
    if (have) {
        const int64_t at = (b * a.L + t) * a.H + h;
        a.dbeta[at] = be;
        if (a.dgate) a.dgate[at] = static_cast<float>(from + (end - own) + rest);
    }
}

// dQ and dK of key heads whose heads were split
template <class MM>
__global__ __launch_bounds__(256) void delta_join_kernel(DeltaArgs a, Buffers u) {
    using S = typename MM::S;
    const int64_t width = a.G * a.N, n = a.B * a.L * width;
    for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < 2 * n; i += gridDim.x * int64_t{256}) {
        const bool k = i >= n;
        const int64_t at = k ? i - n : i, row = at / width, col = at % width;
        const float* from = u.dqk + (k ? u.splits * n : 0) + at;
        float sum = 0.0f;
        for (int64_t s = 0; s < u.splits; ++s) sum += from[s * n];
        if (k) MM::store(static_cast<S*>(a.dk) + row * a.dk_row, col, sum);
        else MM::store(static_cast<S*>(a.dq) + row * a.dq_row, col, sum);
    }
}

// Ranges of a key head's heads where key heads and chunks alone leave CUs idle; they cost a pass over their partial
// sums.  The whole backward, with the pairs in two parts: 256 tokens of 16 heads of one key head x 64 x 64 64 us
// (unsplit 185), 1024 of 32 heads of 8 x 128 x 128 202 (unsplit 215; in blocks for twice the CUs 218), 2 x 4096 of 8 of
// 2 x 64 x 128, 256 blocks unsplit, 277 (split 301).
void split_heads(const DeltaArgs& a, Buffers& u) {
    const int64_t rep = a.H / a.G, blocks = a.B * a.chunks * a.G;
    int64_t splits = (256 + blocks - 1) / blocks;
    if (splits > rep) splits = rep;
    u.heads = (rep + splits - 1) / splits;
    u.splits = (rep + u.heads - 1) / u.heads;
}

template <class MM>
size_t place(DeltaArgs& a, Buffers& u, uint8_t* ws) {
    size_t at = place_chunks<MM>(a, ws, true);
    const auto take = [&](int64_t floats) {
        float* p = reinterpret_cast<float*>(ws + at);
        at += static_cast<size_t>((floats + 63) / 64 * 64) * 4;
        return p;
    };
    split_heads(a, u);
    const int64_t units = a.B * a.H * a.chunks, rows = a.B * a.L * a.H * a.P;
    u.saved.states = take(units * a.P * a.N);
    u.grads = take(units * a.P * a.N);
    u.saved.e = take(rows);
    u.dz = take(rows);
    u.part = take(units * ((a.P + 15) / 16) * 2 * MM::Q);
    u.gate = take(units * 4 * MM::Q);
    u.dqk = take(u.splits > 1 ? 2 * u.splits * a.B * a.L * a.G * a.N : 0);
    return at;
}

template <class MM, int NT, bool SPAN>
hipError_t back_of(const DeltaArgs& a, const Buffers& u, hipStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(a.B * a.H * a.segs * ((a.P + 63) / 64));
    if (a.direct) delta_back_kernel<MM, NT, SPAN, true><<<blocks, 320, 0, stream>>>(a, u);
    else delta_back_kernel<MM, NT, SPAN, false><<<blocks, 320, 0, stream>>>(a, u);
    return hipGetLastError();
}
template <class MM, int NT>
hipError_t kernels_of(const DeltaArgs& a, const Buffers& u, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.segs > 1) {
        e = back_of<MM, NT, true>(a, u, stream);
        if (e == hipSuccess) e = launch_delta_join_back(a, MM::TP == 1 ? SSM_F32 : SSM_BF16, stream);
    }
    if (e == hipSuccess) e = back_of<MM, NT, false>(a, u, stream);
    if (e != hipSuccess) return e;
    const unsigned grads = static_cast<unsigned>(a.B * a.chunks * a.G * u.splits);
    if (a.direct) delta_grad_kernel<MM, NT, true><<<grads, 64 * kGradWaves, 0, stream>>>(a, u);
    else delta_grad_kernel<MM, NT, false><<<grads, 64 * kGradWaves, 0, stream>>>(a, u);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    delta_gate_kernel<MM::Q><<<static_cast<unsigned>((a.B * a.H * a.chunks + 3) / 4), 256, 0, stream>>>(a, u);
    e = hipGetLastError();
    if (e != hipSuccess || u.splits == 1) return e;
    delta_join_kernel<MM><<<1024, 256, 0, stream>>>(a, u);
    return hipGetLastError();
}
template <class MM>
hipError_t bwd_of(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream) {
    Buffers u{};
    place<MM>(a, u, static_cast<uint8_t*>(workspace));
    constexpr size_t es = sizeof(typename MM::S);
    const int64_t keys = a.G * a.N, values = a.H * a.P;
    a.direct = a.N % (16 / es) == 0 && a.P % (16 / es) == 0 && direct_rows_fit(a.q, a.q_row, keys, es) &&
               direct_rows_fit(a.k, a.k_row, keys, es) && direct_rows_fit(a.v, a.v_row, values, es) &&
               direct_rows_fit(a.dy, a.dy_row, values, es) && direct_rows_fit(a.dq, a.dq_row, keys, es) &&
               direct_rows_fit(a.dk, a.dk_row, keys, es) && direct_rows_fit(nullptr, values, values, 4);
    const hipError_t e = launch_delta_walk_saved(a, u.saved, dtype, stream);
    if (e != hipSuccess) return e;
    if (a.N <= 64) return kernels_of<MM, 4>(a, u, stream);
    if (a.N <= 128) return kernels_of<MM, 8>(a, u, stream);
    return kernels_of<MM, 16>(a, u, stream);
}

}  // namespace

size_t delta_bwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype) {
    DeltaArgs a{};
    a.B = B;
    a.L = L;
    a.H = H;
    a.P = P;
    a.G = G;
    a.N = N;
    Buffers u{};
    return dtype == SSM_BF16 ? place<ByBf16>(a, u, nullptr) : place<ByF32>(a, u, nullptr);
}

hipError_t launch_delta_bwd(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? bwd_of<ByBf16>(a, workspace, dtype, stream) : bwd_of<ByF32>(a, workspace, dtype, stream);
}

}  // namespace ssm
