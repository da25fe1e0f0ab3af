// scan_bwd.hip -- the complete backward of the selective scan (ssm_scan_bwd), general shapes.
//
// Forward (length-generalization reading notes, Sec. 2.1 Eq. (1), Sec. 2.5 Eq. (4)), per head:
//     h_t = a_t h_{t-1} + dt_t x_t B_t^T,  y_t = h_t C_t,  a_t = exp(dt_t A),
// a_t counting as 0 where a packed sequence starts.  With g_t = dL/dh_t,
//     g_t = dy_t C_t^T + a_{t+1} g_{t+1},  g past the end = d(final state),
//     dx_t = dt_t g_t B_t,  dB_t = dt_t g_t^T x_t,  dC_t = h_t^T dy_t  (summed over the group's heads),
//     ddt_t = x_t . (g_t B_t) + A q_t,  dA = sum_t dt_t q_t,  q_t = <g_t, a_t h_{t-1}> = dL/d log a_t.
//
// Chunked: tokens in chunks of Q = 64, L_ts = a_{s+1} .. a_t for s <= t of one sequence (else
// 0), S the state before the chunk, G the gradient of the state after it, f_t = a_first .. a_t
// (from the chunk's start), e_s = a_{s+1} .. a_last (to its end), both 0 across a start:
//     S' = f_last S + sum_s (dt_s e_s x_s) B_s^T        (the next chunk's S)
//     G' = f_last G + sum_t (f_t dy_t) C_t^T            (the previous chunk's G)
//     dx_s = dt_s ( sum_t L_ts (C_t.B_s) dy_t  +  e_s G B_s )
//     dC_t = sum_s L_ts dt_s (dy_t.x_s) B_s  +  f_t S^T dy_t
//     dB_s = dt_s ( sum_t L_ts (dy_t.x_s) C_t  +  e_s G^T x_s )
// and q_t is the sum of every product whose factor spans t: with
//     W_ts = L_ts (C_t.B_s) (dy_t.x_s) dt_s,  u_t = f_t dy_t.(S C_t),  v_s = dt_s e_s x_s.(G B_s),
//     q_tau = sum_{s < tau <= t} W_ts + sum_{t >= tau} u_t + sum_{s < tau} v_s + f_last <G, S>.
// The W that span tau are not taken as the difference of all row sums and column sums from tau
// on: those are far larger where the decay is fast, and dA, a sum over the whole batch, would
// keep their rounding errors.  With 16-token tiles they are the row sums over earlier tiles
// from tau to its tile's end, the column sums over later tiles from its tile's start to tau, the
// tile pairs around its tile, all sums of what spans tau only, and the pairs within the one tile
// (here as a difference in double, on the bf16 matrix cores summed directly).  The part of ddt that does not pass through a_t is sum_t W_ts / dt_s + v_s / dt_s,
// formed without the division.
//
// Decays: log a_t is summed in double over the chunk and each factor is the exponential of a sum
// or of a difference of two: f, e and f_last are within two steps of fp32 however fast the decay,
// and here L too; on the bf16 matrix cores, where L's exponent is a difference of fp32 pairs, L is
// within (2 + 1.4 |log2 L|) 2^-24 of itself (36 half-steps where it has fallen to 2^-24).
// log2 a below -1500 (a = 0 in fp32 by far) counts as -1500: the sums keep what follows.
//
// This file: any headdim and dstate that the forward takes, fp32 or bf16 activations, products
// on the fp32 matrix instruction (16 x 16 x 4).  Three steps: the chunks' own shares of S and G
// (one block a chunk and head), their sums along the row (one thread a state element), the
// gradients (one block a chunk and head; dB and dC a head, which a last kernel adds over the
// heads of a group in order, with the chunks' dA).  4 x 8192 tokens x 64 heads x 64 x 128, fp32:
// 1.33 + 0.96 + 5.92 ms and 0.6 ms for the rest, about 190 GFLOP of products at 33 TFLOP/s of the
// 153 that a large fp32 matrix product reaches: bound by the operands' loads, one to four for
// four products.  One head of 64 tokens x 4 x 4: 35 us in six launches, the dependent steps of
// one block (17 us in the gradients).
//
// dA is one number a head: what it is summed from (the pairs' sums, u, v, <G, S>) is formed in
// double from the fp32 dot products and kept as two floats, so that what cancels in it is the
// dot products' rounding alone.
#include "internal.h"

namespace ssm {
namespace {

constexpr int kQ = 64;

typedef float f4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4 mfma4(const f4& a, const f4& b, f4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// The chunk's decays, by the block's first wavefront (lane = token).
struct ChunkDecay {
    double cs[kQ];   // sum of log2 a over the chunk's tokens 0 .. t
    int starts[kQ];  // sequence starts among tokens 0 .. t
    int head, tail;  // tokens before the first start, and before the last
    float f[kQ];     // f_t
    float e[kQ];     // e_t
    float dt[kQ];    // dt_t (0 past the row's end)
    float through;   // f_last
};

__device__ __forceinline__ void chunk_decay(ChunkDecay& cd, const float* dt, int64_t dt_stride,
                                            float A, const int32_t* seq, int64_t t0, int nv) {
    const int t = threadIdx.x;
    if (t < kQ) {
        const float d = t < nv ? dt[t * dt_stride] : 0.0f;
        double s = static_cast<double>(d) * (static_cast<double>(A) * 1.4426950408889634);
        if (s < -1500.0) s = -1500.0;
        int r = 0;
        if (seq && t < nv && t0 + t > 0) r = seq[t0 + t] != seq[t0 + t - 1];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double so = __shfl_up(s, o);
            const int ro = __shfl_up(r, o);
            if (t >= o) {
                s += so;
                r += ro;
            }
        }
        const double end = __shfl(s, 63);
        const int rend = __shfl(r, 63);
        cd.cs[t] = s;
        cd.starts[t] = r;
        cd.f[t] = r == 0 ? exp2_of(s) : 0.0f;
        cd.e[t] = r == rend ? exp2_of(end - s) : 0.0f;
        cd.dt[t] = d;
        if (t == 63) cd.through = cd.f[63];
        const int head = __popcll(__ballot(r == 0)), tail = __popcll(__ballot(r != rend));
        if (t == 0) {
            cd.head = head;
            cd.tail = tail;
        }
    }
    __syncthreads();
}

// block -> (row, head, chunk)
struct Where {
    int64_t b, h, c, g, t0;
    int nv;
};
__device__ __forceinline__ Where where(const ScanBwdArgs& a, int64_t blk) {
    Where w;
    w.c = blk % a.chunks;
    w.h = blk / a.chunks % a.H;
    w.b = blk / a.chunks / a.H;
    w.g = w.h / (a.H / a.G);
    w.t0 = w.c * kQ;
    w.nv = a.L - w.t0 < kQ ? static_cast<int>(a.L - w.t0) : kQ;
    return w;
}

// four consecutive elements at any element's alignment
__device__ __forceinline__ f4 load4(const float* p) {
    typedef float f4any __attribute__((ext_vector_type(4), aligned(4)));
    return *reinterpret_cast<const f4any*>(p);
}
__device__ __forceinline__ f4 load4(const uint16_t* p) {
    typedef uint32_t u2any __attribute__((ext_vector_type(2), aligned(2)));
    const u2any q = *reinterpret_cast<const u2any*>(p);
    return f4{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xFFFF0000u),
              __uint_as_float(q[1] << 16), __uint_as_float(q[1] & 0xFFFF0000u)};
}

// A row-major view [tokens][cols] of the chunk's tokens lo .. rows - 1: zeros outside.  What lies
// outside is read from the last row and column instead (of no rows, the first) and replaced, so no
// load is under a branch and waits for another.  W: cols is a multiple of 16, so four consecutive
// columns are inside or outside.
template <class S, bool W>
struct View {
    const typename S::T* p;
    int64_t row;
    int rows, cols, lo = 0;
    __device__ __forceinline__ bool has(int r) const { return static_cast<unsigned>(r - lo) < static_cast<unsigned>(rows - lo); }
    __device__ __forceinline__ int row_at(int r) const { return r < rows ? r : rows > 0 ? rows - 1 : 0; }
    __device__ __forceinline__ float at(int r, int c) const {
        const float v = S::load(p, row_at(r) * row + (c < cols ? c : cols - 1));
        return has(r) && c < cols ? v : 0.0f;
    }
    // operand with the contraction along the row: row r, columns k .. k + 3
    __device__ __forceinline__ f4 along(int r, int k) const {
        if constexpr (W) {
            const f4 v = load4(p + row_at(r) * row + k);  // k < cols: called for 16 at a time
            return has(r) ? v : f4{0, 0, 0, 0};
        } else {
            return f4{at(r, k), at(r, k + 1), at(r, k + 2), at(r, k + 3)};
        }
    }
    // operand with the contraction over the rows: rows k .. k + 3 of column c
    __device__ __forceinline__ f4 down(int k, int c) const {
        return f4{at(k, c), at(k + 1, c), at(k + 2, c), at(k + 3, c)};
    }
};

// ---------------------------------------------------------------------------------------
// each chunk's share of the next S (blockIdx.y = 0) and of the previous G (blockIdx.y = 1)
// ---------------------------------------------------------------------------------------
template <class S, bool W>
__global__ void __launch_bounds__(256) sb_local_kernel(ScanBwdArgs a) {
    __shared__ ChunkDecay cd;
    const Where w = where(a, blockIdx.x);
    const bool rev = blockIdx.y != 0;
    chunk_decay(cd, a.dt + (w.b * a.L + w.t0) * a.H + w.h, a.H, a.A[w.h],
                a.seq ? a.seq + w.b * a.L : nullptr, w.t0, w.nv);
    using T = typename S::T;
    const int64_t tok = w.b * a.L + w.t0;
    const int P = static_cast<int>(a.P), N = static_cast<int>(a.N);
    // Tokens across a start hand nothing on (forward those before the chunk's last start, in reverse
    // those from its first on).  Their factor is 0, and so are both operands: a NaN or infinity of a
    // sequence that ends in this chunk, times 0, would reach the chunks behind it.
    const int lo = rev ? 0 : cd.tail, hi = rev && cd.head < w.nv ? cd.head : w.nv;
    const View<S, W> xv{static_cast<const T*>(rev ? a.dy : a.x) + tok * (rev ? a.dy_row : a.x_row) + w.h * P,
                     rev ? a.dy_row : a.x_row, hi, P, lo};
    const View<S, W> bv{static_cast<const T*>(rev ? a.C : a.Bm) + tok * (rev ? a.c_row : a.b_row) + w.g * N,
                     rev ? a.c_row : a.b_row, hi, N, lo};
    float* out = (rev ? a.grads : a.states) + ((w.b * a.H + w.h) * a.chunks + w.c) * a.P * a.N;
    const int lane = threadIdx.x & 63, li = lane & 15, g4 = lane >> 4;
    if (!rev && threadIdx.x == 0) a.through[(w.b * a.H + w.h) * a.chunks + w.c] = cd.through;
    // A wavefront takes kLP x kLN tiles at a time: an operand serves all tiles of its row or column
    // (4 x 8192 x 64 heads x 64 x 128, fp32: 1337 us, one tile at a time 2570; narrow heads have
    // too few tiles, 2048 x 16 x 24 x 16: 13 and 8 us).
    constexpr int kLP = W ? 2 : 1, kLN = W ? 4 : 1;
    const int np = (P + 16 * kLP - 1) / (16 * kLP), nn = (N + 16 * kLN - 1) / (16 * kLN);
    for (int tile = threadIdx.x >> 6; tile < np * nn; tile += 4) {
        const int p0 = tile / nn * 16 * kLP, n0 = tile % nn * 16 * kLN;
        f4 acc[kLP][kLN] = {};
        for (int k = 0; k < kQ; k += 16) {
            f4 x[kLP], y[kLN], scale;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = k + 4 * g4 + j;
                scale[j] = rev ? cd.f[t] : cd.dt[t] * cd.e[t];
            }
#pragma unroll
            for (int i = 0; i < kLP; ++i) x[i] = xv.down(k + 4 * g4, p0 + 16 * i + li) * scale;
#pragma unroll
            for (int i = 0; i < kLN; ++i) y[i] = bv.down(k + 4 * g4, n0 + 16 * i + li);
#pragma unroll
            for (int i = 0; i < kLP; ++i)
#pragma unroll
                for (int h = 0; h < kLN; ++h) acc[i][h] = mfma4(x[i], y[h], acc[i][h]);
        }
#pragma unroll
        for (int i = 0; i < kLP; ++i)
#pragma unroll
            for (int h = 0; h < kLN; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int p = p0 + 16 * i + 4 * g4 + e, n = n0 + 16 * h + li;
                    if (p < P && n < N) out[p * N + n] = acc[i][h][e];
                }
    }
}

// Sums along the row, in place: the share of chunk c becomes the state before it (blockIdx.y =
// 0), or the gradient of the state after it (1, which also gives the initial state's).  A
// chunk that holds a start takes nothing over, whatever the state was.
__global__ void __launch_bounds__(256) sb_pass_kernel(ScanBwdArgs a) {
    const int64_t PN = a.P * a.N, per = (PN + 255) / 256;
    const int64_t bh = blockIdx.x / per, i = blockIdx.x % per * 256 + threadIdx.x;
    if (i >= PN) return;
    const bool rev = blockIdx.y != 0;
    float* s = (rev ? a.grads : a.states) + bh * a.chunks * PN + i;
    const float* f = a.through + bh * a.chunks;
    const float* from = rev ? a.dhT : a.h0;
    float v = from ? from[bh * PN + i] : 0.0f;
    for (int64_t j = 0; j < a.chunks; ++j) {
        const int64_t c = rev ? a.chunks - 1 - j : j;
        const float own = s[c * PN], th = f[c];
        s[c * PN] = v;
        v = th == 0.0f ? own : th * v + own;
    }
    if (rev && a.dh0) a.dh0[bh * PN + i] = v;
}

// sums along aligned spans of LEN lanes: from the lane to the span's end, and before the lane
template <int LEN>
__device__ __forceinline__ double from_lane(double v, int lane) {
#pragma unroll
    for (int o = 1; o < LEN; o <<= 1) {
        const double u = __shfl_down(v, o);
        if ((lane & (LEN - 1)) + o < LEN) v += u;
    }
    return v;
}
template <int LEN>
__device__ __forceinline__ double before_lane(double v, int lane) {
    const double own = v;
#pragma unroll
    for (int o = 1; o < LEN; o <<= 1) {
        const double u = __shfl_up(v, o);
        if ((lane & (LEN - 1)) >= o) v += u;
    }
    return v - own;
}

// ---------------------------------------------------------------------------------------
// gradients of one chunk and head
// ---------------------------------------------------------------------------------------
template <class S, bool W>
__global__ void __launch_bounds__(512) sb_grad_kernel(ScanBwdArgs a) {
    __shared__ ChunkDecay cd;
    __shared__ float pair[kQ][kQ + 1];  // [t][s] L_ts (C_t.B_s)
    __shared__ float lw[kQ][kQ + 1];    // [t][s] L_ts (dy_t.x_s) dt_s
    // in double, formed from the fp32 dot products without another rounding: the part of q_t within
    // its tile is a difference of these, and dA, a sum over all tokens, may cancel further
    __shared__ double rowp[4][kQ];      // sums over the s of one 16-column tile, s < t, of W
    __shared__ double colp[4][kQ];      // sums over the t of one 16-row tile, t > s, of W / dt_s
    __shared__ float diag[kQ];          // W_ss / dt_s
    __shared__ double uu[2][kQ], vv[2][kQ];  // u_t, v_s / dt_s, by the columns' share
    __shared__ double gs[8];
    const Where w = where(a, blockIdx.x);
    chunk_decay(cd, a.dt + (w.b * a.L + w.t0) * a.H + w.h, a.H, a.A[w.h],
                a.seq ? a.seq + w.b * a.L : nullptr, w.t0, w.nv);
    using T = typename S::T;
    const int64_t tok = w.b * a.L + w.t0;
    const int P = static_cast<int>(a.P), N = static_cast<int>(a.N);
    const View<S, W> xv{static_cast<const T*>(a.x) + tok * a.x_row + w.h * P, a.x_row, w.nv, P};
    const View<S, W> dyv{static_cast<const T*>(a.dy) + tok * a.dy_row + w.h * P, a.dy_row, w.nv, P};
    const View<S, W> bv{static_cast<const T*>(a.Bm) + tok * a.b_row + w.g * N, a.b_row, w.nv, N};
    const View<S, W> cv{static_cast<const T*>(a.C) + tok * a.c_row + w.g * N, a.c_row, w.nv, N};
    const int64_t at = ((w.b * a.H + w.h) * a.chunks + w.c) * a.P * a.N;
    const View<F32, W> sv{a.states + at, N, P, N}, gv{a.grads + at, N, P, N};
    const int lane = threadIdx.x & 63, li = lane & 15, g4 = lane >> 4, wave = threadIdx.x >> 6;

    // pairs s <= t: the ten 16 x 16 tiles on and below the diagonal
    for (int tile = wave; tile < 10; tile += 8) {
        const int ti = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3;
        const int si = tile - ti * (ti + 1) / 2;
        f4 cb{0, 0, 0, 0}, yx{0, 0, 0, 0};
        for (int k = 0; k < N; k += 16)
            cb = mfma4(cv.along(16 * ti + li, k + 4 * g4), bv.along(16 * si + li, k + 4 * g4), cb);
        for (int k = 0; k < P; k += 16)
            yx = mfma4(dyv.along(16 * ti + li, k + 4 * g4), xv.along(16 * si + li, k + 4 * g4), yx);
        const int s = 16 * si + li;
        const double css = cd.cs[s];
        const int rs = cd.starts[s];
        const float dts = cd.dt[s];
        double below = 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 16 * ti + 4 * g4 + e;
            const bool in = t >= s && cd.starts[t] == rs;
            const double ld = in ? exp2(cd.cs[t] - css) : 0.0;
            const float l = static_cast<float>(ld);
            const float pv = in ? l * cb[e] : 0.0f, yv = in ? l * yx[e] * dts : 0.0f;
            pair[t][s] = pv;
            lw[t][s] = yv;
            const double w0 = in ? ld * (static_cast<double>(cb[e]) * yx[e]) : 0.0;
            if (t == s) diag[s] = static_cast<float>(w0);
            else below += w0;
            double row = t > s ? w0 * dts : 0.0;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) row += __shfl_xor(row, o);
            if (li == 0) rowp[si][t] = row;
        }
        below += __shfl_xor(below, 16);
        below += __shfl_xor(below, 32);
        if (g4 == 0) colp[ti][s] = below;
    }
    // <G, S>
    {
        double d = 0.0;
        for (int i = threadIdx.x; i < P * N; i += 512) d += static_cast<double>(sv.p[i]) * gv.p[i];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) d += __shfl_xor(d, o);
        if (lane == 0) gs[wave] = d;
    }
    __syncthreads();

    // this wavefront's 16 tokens r0 .. r0 + 15 of every output, every other 16 columns of them
    const int r0 = 16 * (wave & 3), part = wave >> 2;
    T* dxo = static_cast<T*>(a.dx) + tok * a.dx_row + w.h * P;
    double v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};  // without e and f
    for (int p0 = 16 * part; p0 < P; p0 += 32) {
        f4 in{0, 0, 0, 0}, out{0, 0, 0, 0};
        for (int k = r0; k < kQ; k += 16) {
            const int t = k + 4 * g4;
            in = mfma4(f4{pair[t][r0 + li], pair[t + 1][r0 + li], pair[t + 2][r0 + li], pair[t + 3][r0 + li]},
                       dyv.down(t, p0 + li), in);
        }
        for (int k = 0; k < N; k += 16)
            out = mfma4(bv.along(r0 + li, k + 4 * g4), gv.along(p0 + li, k + 4 * g4), out);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int s = r0 + 4 * g4 + e, p = p0 + li;
            const float o = cd.e[s] == 0.0f ? 0.0f : cd.e[s] * out[e];
            if (o != 0.0f) v[e] += static_cast<double>(xv.at(s, p)) * out[e];
            if (s < w.nv && p < P) S::store(dxo, s * a.dx_row + p, cd.dt[s] * (in[e] + o));
        }
    }
    const int64_t ho = (tok * a.H + w.h) * N;  // [row][token][head][N]
    for (int n0 = 16 * part; n0 < N; n0 += 32) {
        f4 in{0, 0, 0, 0}, out{0, 0, 0, 0}, bin{0, 0, 0, 0}, bout{0, 0, 0, 0};
        for (int k = 0; k < r0 + 16; k += 16) {
            const int s = k + 4 * g4;
            in = mfma4(f4{lw[r0 + li][s], lw[r0 + li][s + 1], lw[r0 + li][s + 2], lw[r0 + li][s + 3]},
                       bv.down(s, n0 + li), in);
        }
        for (int k = r0; k < kQ; k += 16) {
            const int t = k + 4 * g4;
            bin = mfma4(f4{lw[t][r0 + li], lw[t + 1][r0 + li], lw[t + 2][r0 + li], lw[t + 3][r0 + li]},
                        cv.down(t, n0 + li), bin);
        }
        for (int k = 0; k < P; k += 16) {
            out = mfma4(dyv.along(r0 + li, k + 4 * g4), sv.down(k + 4 * g4, n0 + li), out);
            bout = mfma4(xv.along(r0 + li, k + 4 * g4), gv.down(k + 4 * g4, n0 + li), bout);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = r0 + 4 * g4 + e, n = n0 + li;
            const float o = cd.f[t] == 0.0f ? 0.0f : cd.f[t] * out[e];
            const float bo = cd.e[t] == 0.0f ? 0.0f : cd.e[t] * cd.dt[t] * bout[e];
            if (o != 0.0f) u[e] += static_cast<double>(cv.at(t, n)) * out[e];
            if (t < w.nv && n < N) {
                a.dC_head[ho + t * a.H * N + n] = in[e] + o;
                a.dB_head[ho + t * a.H * N + n] = bin[e] + bo;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            u[e] += __shfl_xor(u[e], o);
            v[e] += __shfl_xor(v[e], o);
        }
        if (li == 0) {
            const int t = r0 + 4 * g4 + e;
            uu[part][t] = cd.f[t] == 0.0f ? 0.0 : u[e] * exp2(cd.cs[t]);
            vv[part][t] = cd.e[t] == 0.0f ? 0.0 : v[e] * exp2(cd.cs[kQ - 1] - cd.cs[t]);
        }
    }
    __syncthreads();

    // the sums that ddt and dA are formed from (lane = token)
    if (wave != 0) return;
    const int t = lane, j = t / 16;
    float* out = a.sums + ((w.b * a.H + w.h) * a.chunks + w.c) * (kSums * kQ + kSumTail);
    double row = 0.0, below = 0.0;
    for (int i = 0; i < j; ++i) row += rowp[i][t];
    for (int i = j + 1; i < 4; ++i) below += colp[i][t];
    // the W that span t: rows from t to its tile's end over earlier tiles, columns of its tile
    // before t under later tiles, the pairs within its tile, and the tile pairs around it
    const double dts = cd.dt[t];
    double q = from_lane<16>(row, t) + before_lane<16>(below * dts, t);
    q += from_lane<16>(rowp[j][t] - colp[j][t] * dts, t);
    for (int tj = j + 1; tj < 4; ++tj)
        for (int i = 0; i < 16 * j; ++i) q += rowp[i >> 4][16 * tj + (i & 15)];
    // each as the sum of two floats
    auto both = [](float* hi, float* lo, double v) {
        *hi = static_cast<float>(v);
        *lo = static_cast<float>(v - *hi);
    };
    both(out + kSumU * kQ + t, out + kSumULow * kQ + t, uu[0][t] + uu[1][t]);
    both(out + kSumV * kQ + t, out + kSums * kQ + t, vv[0][t] + vv[1][t]);
    both(out + kSumSpan * kQ + t, out + kSumSpanLow * kQ + t, q);
    out[kSumColOff * kQ + t] = static_cast<float>(below + colp[j][t]);
    out[kSumDiag * kQ + t] = diag[t];
    if (t == 0)
        both(out + kSums * kQ + 64, out + kSums * kQ + 65,
             cd.through == 0.0f ? 0.0 : exp2(cd.cs[kQ - 1]) * (((gs[0] + gs[1]) + (gs[2] + gs[3])) + ((gs[4] + gs[5]) + (gs[6] + gs[7]))));
}

// q, ddt and a chunk's share of dA: one wavefront a head and chunk, Q / 64 tokens a lane; a block
// takes kAnchor chunks of two heads (the chunks that share an f <G, S>).  Blocks of one row and
// chunk range follow each other at the distance of all ranges: on one XCD where that is a
// multiple of 8, so that their stores of ddt meet in its L2.
template <int Q>
__global__ void __launch_bounds__(128 * kAnchor) sb_ddt_kernel(ScanBwdArgs a) {
    constexpr int K = Q / 64;
    __shared__ double usum[2][kAnchor], vsum[2][kAnchor], most[2][kAnchor];
    __shared__ float thr[2][kAnchor];
    const int64_t ranges = (a.chunks + kAnchor - 1) / kAnchor, br = a.B * ranges;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, hw = wave / kAnchor, ci = wave % kAnchor;
    const int64_t h = blockIdx.x / br * 2 + hw, b = blockIdx.x % br / ranges, range = blockIdx.x % ranges;
    const int64_t c = range * kAnchor + ci, t0 = c * Q;
    const int64_t last = (range + 1) * kAnchor < a.chunks ? (range + 1) * kAnchor - 1 : a.chunks - 1;
    const bool on = h < a.H && c < a.chunks;
    const int64_t at = on ? (b * a.H + h) * a.chunks + c : 0;
    const float* in = a.sums + at * (kSums * Q + kSumTail);
    double q[K], after = 0.0, before = 0.0;
    float direct[K], dts[K];
    if (on) {
        double u[K], v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = lane + 64 * k;
            dts[k] = t0 + t < a.L ? (Q == 128 ? a.decay[(at * 5 + 4) * Q + t] : a.dt[(b * a.L + t0 + t) * a.H + h]) : 0.0f;
            const float coff = in[kSumColOff * Q + t], vt = in[kSumV * Q + t];
            u[k] = in[kSumU * Q + t];
            v[k] = static_cast<double>(vt) * dts[k];
            if constexpr (Q == kQ) {  // the span's W are summed already; two floats each
                direct[k] = (coff + in[kSumDiag * Q + t]) + vt;
                u[k] += in[kSumULow * Q + t];
                v[k] += static_cast<double>(in[kSums * Q + t]) * dts[k];
                q[k] = static_cast<double>(in[kSumSpan * Q + t]) + in[kSumSpanLow * Q + t];
                continue;
            }
            const float cdiag = in[kSumColDiag * Q + t];
            direct[k] = ((coff + cdiag) + in[kSumDiag * Q + t]) + vt;
            q[k] = from_lane<16>(in[kSumRowOff * Q + t], lane) + before_lane<16>(static_cast<double>(coff) * dts[k], lane);
            q[k] += in[kSumRowDiag * Q + t];
        }
        if constexpr (Q != kQ) {  // the tile pairs around the token's tile
#pragma unroll
            for (int j2 = 2; j2 < Q / 16; ++j2)
#pragma unroll
                for (int i = 0; i < j2 - 1; ++i) {
                    const double w = in[kSums * Q + 8 * j2 + i];
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const int j = (lane >> 4) + 4 * k;
                        q[k] += i < j && j < j2 ? w : 0.0;
                    }
                }
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            const double s = from_lane<64>(u[k], lane);
            q[k] += s + after;
            after += __shfl(s, 0);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const double s = before_lane<64>(v[k], lane);
            q[k] += s + before;
            before += __shfl(s + v[k], 63);
        }
        // |f_last <G, S>| of this chunk is at most f_last |G| |S|
        const float th = a.through[at];
        double norms = 0.0;
        if constexpr (Q != kQ) {
            const int i = lane & 7;
            float ns = i < a.N / 16 ? in[kSums * Q + 64 + i] : 0.0f, ng = i < a.N / 16 ? in[kSums * Q + 72 + i] : 0.0f;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                ns += __shfl_xor(ns, o);
                ng += __shfl_xor(ng, o);
            }
            norms = sqrt(static_cast<double>(ns)) * sqrt(static_cast<double>(ng)) / static_cast<double>(uint64_t{1} << (2 * kNormExp - 1)) / 2;
        }
        if (lane == 0) {
            usum[hw][ci] = after;
            vsum[hw][ci] = before;
            thr[hw][ci] = th;
            most[hw][ci] = 1.00001 * th * norms;
        }
    }
    __syncthreads();
    if (!on) return;
    // f_last <G, S> of this chunk: from the range's last chunk back (nothing across a start or a
    // decay to 0)
    double pass = 0.0;
    if constexpr (Q == kQ) {
        if (thr[hw][ci] != 0.0f) pass = static_cast<double>(in[kSums * Q + 64]) + in[kSums * Q + 65];
    } else {
        const int end = static_cast<int>(last - range * kAnchor);
        if (thr[hw][end] != 0.0f) pass = a.anchor[(b * a.H + h) * ranges + range];
        for (int k = end - 1; k >= ci; --k) {
            const double m = most[hw][k];
            pass += usum[hw][k + 1] - vsum[hw][k];
            if (pass > m) pass = m;
            if (pass < -m) pass = -m;
            if (thr[hw][k] == 0.0f) pass = 0.0;
        }
    }
    const double A = a.A[h];
    double da = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t t = t0 + lane + 64 * k;
        if (t >= a.L) continue;
        q[k] += pass;
        if (a.seq && t > 0 && a.seq[b * a.L + t] != a.seq[b * a.L + t - 1]) q[k] = 0.0;  // a start takes nothing over
        a.ddt[(b * a.L + t) * a.H + h] = static_cast<float>(q[k] * A + direct[k]);
        da += q[k] * dts[k];
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) da += __shfl_xor(da, o);
    if (lane == 0) a.dA_part[(b * a.chunks + c) * a.H + h] = da;
}

// dB, dC: the heads of a group added in order, rounded once
template <class S>
__global__ void __launch_bounds__(256) sb_heads_kernel(ScanBwdArgs a) {
    using T = typename S::T;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t GN = a.G * a.N;
    if (i >= a.B * a.L * GN) return;
    const int64_t k = a.H / a.G, tok = i / GN, g = i % GN / a.N, n = i % a.N;
    const float* p = (blockIdx.y ? a.dC_head : a.dB_head) + (tok * a.H + g * k) * a.N + n;
    float s = 0.0f;
    for (int64_t j = 0; j < k; ++j) s += p[j * a.N];
    if (blockIdx.y) S::store(static_cast<T*>(a.dC) + tok * a.dc_row, g * a.N + n, s);
    else S::store(static_cast<T*>(a.dB) + tok * a.db_row, g * a.N + n, s);
}

// dA: the chunks' shares in a fixed order, in double; one block a head
__global__ void __launch_bounds__(256) sb_dA_kernel(ScanBwdArgs a) {
    __shared__ double sum[4];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < a.B * a.chunks; i += 256) s += a.dA_part[i * a.H + blockIdx.x];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.dA[blockIdx.x] = static_cast<float>((sum[0] + sum[1]) + (sum[2] + sum[3]));
}

template <class S>
hipError_t launch_general(const ScanBwdArgs& a, hipStream_t s) {
    const uint32_t bhc = static_cast<uint32_t>(a.B * a.H * a.chunks);
    const bool whole = a.P % 16 == 0 && a.N % 16 == 0;
    if (whole) sb_local_kernel<S, true><<<dim3(bhc, 2), 256, 0, s>>>(a);
    else sb_local_kernel<S, false><<<dim3(bhc, 2), 256, 0, s>>>(a);
    sb_pass_kernel<<<dim3(static_cast<uint32_t>(a.B * a.H * ((a.P * a.N + 255) / 256)), 2), 256, 0, s>>>(a);
    if (whole) sb_grad_kernel<S, true><<<bhc, 512, 0, s>>>(a);
    else sb_grad_kernel<S, false><<<bhc, 512, 0, s>>>(a);
    sb_heads_kernel<S><<<dim3(static_cast<uint32_t>((a.B * a.L * a.G * a.N + 255) / 256), 2), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_scan_bwd_ddt(a, kQ, s) : e;
}

size_t r256(size_t n) { return (n + 255) / 256 * 256; }

// places the workspace's parts; returns its size
size_t lay_out(ScanBwdArgs& a, uint8_t* base) {
    size_t at = 0;
    auto part = [&](auto*& p, size_t n) {
        p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at);
        at += r256(n * sizeof(*p));
    };
    const size_t bh = static_cast<size_t>(a.B * a.H), bhc = bh * a.chunks;
    part(a.dA_part, bhc);
    part(a.through, bhc);
    part(a.sums, bhc * (kSums * kQ + kSumTail));
    part(a.states, bhc * a.P * a.N);
    part(a.grads, bhc * a.P * a.N);
    part(a.dB_head, bh * a.L * a.N);
    part(a.dC_head, bh * a.L * a.N);
    return at;
}

}  // namespace

hipError_t launch_scan_bwd_ddt(const ScanBwdArgs& a, int tokens, hipStream_t s) {
    const uint32_t grid = static_cast<uint32_t>(a.B * ((a.chunks + kAnchor - 1) / kAnchor) * ((a.H + 1) / 2));
    if (tokens == 128) sb_ddt_kernel<128><<<grid, 1024, 0, s>>>(a);
    else sb_ddt_kernel<64><<<grid, 1024, 0, s>>>(a);
    sb_dA_kernel<<<static_cast<uint32_t>(a.H), 256, 0, s>>>(a);
    return hipGetLastError();
}

size_t scan_bwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N,
                                ssm_dtype_t dtype) {
    if (scan_bwd_mfma_supported(H, P, G, N, dtype)) return scan_bwd_mfma_workspace_bytes(B, L, H, P, G, N);
    ScanBwdArgs a{};
    a.B = B; a.L = L; a.H = H; a.P = P; a.G = G; a.N = N;
    a.chunks = (L + kQ - 1) / kQ;
    return lay_out(a, nullptr);
}

// blocks of the largest launch, against the grid's limit
int64_t scan_bwd_blocks(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N) {
    const int64_t a = B * H * ((L + kQ - 1) / kQ), b = B * H * ((P * N + 255) / 256);
    const int64_t c = (B * L * G * N + 255) / 256;
    return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

hipError_t launch_scan_bwd(ScanBwdArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t s) {
    if (scan_bwd_mfma_supported(a.H, a.P, a.G, a.N, dtype)) return launch_scan_bwd_mfma(a, workspace, s);
    a.chunks = (a.L + kQ - 1) / kQ;
    lay_out(a, static_cast<uint8_t*>(workspace));
    return dtype == SSM_BF16 ? launch_general<BF16>(a, s) : launch_general<F32>(a, s);
}

// no tokens: the initial state's gradient is the final state's, dA = 0
__global__ void sb_empty_kernel(const float* dhT, float* dh0, float* dA, int64_t n, int64_t H) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < H) dA[i] = 0.0f;
    if (dh0 && i < n) dh0[i] = dhT ? dhT[i] : 0.0f;
}
hipError_t launch_scan_bwd_empty(const float* dhT, float* dh0, float* dA, int64_t n, int64_t H,
                                 hipStream_t s) {
    const int64_t m = n > H ? n : H;
    sb_empty_kernel<<<static_cast<uint32_t>((m + 255) / 256), 256, 0, s>>>(dhT, dh0, dA, n, H);
    return hipGetLastError();
}

}  // namespace ssm
