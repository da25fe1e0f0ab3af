// delta.h -- what the kernels of the gated delta rule share: the arguments, the two arithmetics
// (bf16 matrix instructions on split operands, fp32 matrix instructions) and the workspace.
//
// Per head, with state h [P, N], a_t = e^gate_t and b_t = beta_t:
//     e_t = v_t - a_t h_{t-1} k_t,   h_t = a_t h_{t-1} + b_t e_t k_t^T,   y_t = scale h_t q_t
// Over a chunk of Q tokens that starts from h_0, with G_t the sum of the gates from the chunk's
// start on (from a packed sequence's where that starts later) and r_ts = e^(G_t - G_s) (0 where a
// packed sequence starts in (s, t]):
//     D_ts = r_ts (k_t . k_s) b_s (s < t),   T = (I + D)^-1,   M_ts = scale r_ts q_t . k_s (s <= t)
//     Z = V - e^G K h_0^T,   E = T Z,   U = b E
//     Y = scale e^G Q h_0^T + M U,   h_Q = e^{G_Q} h_0 + U^T e^{G_Q - G} K
// (E and b U keep apart so that b = 0 needs no division.)  T and M need no state: delta_prep forms
// them for all chunks at once, and only the products with the state walk along the row.
//
// Layout of a walk: a wavefront owns 16 channels of one head for the whole row, with their state in
// accumulators (rows: state dimension, columns: channels).  Every product's result has the tokens or
// the state dimensions as rows and the wavefront's channels as columns, which is the next product's
// right operand as it stands (mfma_tiles.h: "token order"), so no value passes between
// wavefronts; K, Q, T and M are the left operands, shared in LDS.
#pragma once

#include "internal.h"
#include "mfma_tiles.h"

namespace ssm {

struct DeltaArgs {
    const void* q;  // [B, L, G, N], token rows q_row elements apart
    const void* k;
    const void* v;  // [B, L, H, P]
    const void* dy;
    const float* beta;  // [B, L, H]
    const float* gate;  // [B, L, H] or NULL (= 0)
    const float* h0;    // [B, H, P, N] or NULL
    const float* dhT;   // [B, H, P, N] or NULL
    const int32_t* seq;
    void* y;
    void* dq;
    void* dk;
    void* dv;
    float* dbeta;
    float* dgate;        // or NULL
    float* dh0;          // or NULL
    float* final_state;  // [B, H, P, N] or NULL
    int64_t q_row, k_row, v_row, y_row, dy_row, dq_row, dk_row, dv_row;
    int64_t B, L, H, P, G, N;
    float scale;
    // set by the launchers: whether tokens go straight into LDS (16-byte aligned rows that do not overlap, dstate
    // and headdim whole pieces, a chunk's rows of every token tensor within 30 bits of bytes); the chunks' part
    // of the workspace
    bool direct;
    int64_t chunks;
    uint8_t* T;      // [B, H, chunks] images
    uint8_t* M;
    uint8_t* Tt;     // transposed, backward only (M is transposed there)
    // rows cut into `segs` segments of seg_chunks chunks where there are few (plan_segments)
    int64_t segs, seg_chunks;
    float* phi;      // [B, H, segs, N, N]: what a segment makes of the state before it, from the right; row m
    int32_t* power;  // [B, H, segs, N]: times 2^power[m]
    float* gain;     // [B, H, segs, P, N]: what its own tokens bring
    float* entry;    // [B, H, segs, P, N]: the state before it (backward: the gradient of the state after it)
    double* gates;   // [B, H, chunks, Q]: sums of gates (TokenSums), backward only
    float* factors;  // [B, H, chunks, kFactors, Q]: e^G from the chunk's start, e^{G_Q - G}, beta, sequences begun
};

namespace delta {

constexpr int kFactors = 4;
// added to the sequences begun of a chunk's tokens where its keys or queries are not all finite
constexpr float kNotFinite = 1024.0f;
constexpr double kLog2e = 1.4426950408889634;

// Sums of gates below this are as good as minus infinity (e^-1e4 = 0 in fp32), and finite: their
// differences are no NaN.  A NaN stays one.
constexpr float kLeastGate = -1e4f;
__device__ __forceinline__ double gate_of(float g) { return g < kLeastGate ? kLeastGate : g; }

// e^x of a sum kept in double
__device__ __forceinline__ float exp_of(double x) { return exp2_of(x * kLog2e); }

// ---------------------------------------------------------------------------------------
// bf16: exact operands as they are, fp32 operands in bf16 parts (three hold all 24 bits)
// ---------------------------------------------------------------------------------------
struct ByBf16 {
    using S = uint16_t;
    static constexpr int Q = 64;   // tokens a chunk
    static constexpr int KB = 32;  // contraction of one operand pair
    static constexpr int R = 8;    // of it, values a lane
    static constexpr int TP = 3;   // parts of T, M and every other fp32 operand that is kept
    template <int PARTS>
    struct Frag {
        bf8 p[PARTS];
    };
    template <int PARTS>
    __device__ __forceinline__ static Frag<PARTS> parts(const float (&v)[8]) {
        Frag<PARTS> f;
        split<PARTS>(v, f.p);
        return f;
    }
    // rows of the right operand's contraction block kk, from result tiles
    template <int PARTS>
    __device__ __forceinline__ static Frag<PARTS> of_tiles(const f4* tile, int kk) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = tile[2 * kk + (j >> 2)][j & 3];
        return parts<PARTS>(v);
    }
    // products of parts whose orders sum below the more exact side's
    template <int PA, int PB>
    __device__ __forceinline__ static void mac(f4& c, const Frag<PA>& a, const Frag<PB>& b) {
#pragma unroll
        for (int i = PA - 1; i >= 0; --i)
#pragma unroll
            for (int j = PB - 1; j >= 0; --j)
                if (i + j < (PA > PB ? PA : PB)) c = mfma(a.p[i], b.p[j], c);
    }
    __device__ __forceinline__ static float value(const S* p, int64_t i) { return bf16_to_f32(p[i]); }
    __device__ __forceinline__ static void store(S* p, int64_t i, float v) { p[i] = f32_to_bf16(v); }

    // LDS tiles of W columns: rows of 2 W bytes (128 or more) in swizzled 16-byte pieces
    template <int W>
    static constexpr int tile_bytes(int rows) { return rows * 2 * W; }
    template <int W>
    __device__ __forceinline__ static int piece_at(int row, int q) { return piece<2 * W>(row, q); }
    // left operand, rows r0 + li, contraction block kk in token order
    template <int W>
    __device__ __forceinline__ static Frag<1> rows(const uint8_t* t, int r0, int kk, int li, int g4) {
        const int at = (((g4 >> 1) ^ sw<2 * W>(li)) << 4 | (g4 & 1) << 3) ^ (kk << 6);
        const uint8_t* p = t + (r0 + li) * (2 * W);
        Frag<1> f;
        f.p[0] = join(lds<s4>(p + at), lds<s4>(p + (at ^ 32)));
        return f;
    }
    // the same in natural order
    template <int W>
    __device__ __forceinline__ static Frag<1> along(const uint8_t* t, int r0, int kk, int li, int g4) {
        Frag<1> f;
        f.p[0] = ssm::along<2 * W>(t, along_off<2 * W>(li, g4), r0, kk);
        return f;
    }
    // first column of the 16 bytes that lie at slot `s` of a row
    template <int W>
    __device__ __forceinline__ static int column_of(int row, int s) { return 8 * (s ^ sw<2 * W>(row)); }
    // Tiles that a state is multiplied with: the same pieces under a swizzle of their own (rows 0 - 7
    // and 8 - 15 apart but for its bit 1), for the operand along rows in natural order and a
    // transposing read whose four columns a lane are half b ^ (j & 1) of piece j: 32 lanes at 64 banks.
    // A state's tile i holds, in lane group g4, the dimensions state_row(i, g4) .. + 3.
    template <int W>
    __device__ __forceinline__ static int state_sw(int row) {
        const int b0 = row & 1, b1 = (row >> 1) & 1, b2 = (row >> 2) & 1, b3 = (row >> 3) & 1;
        return W == 64 ? b1 << 2 | b3 << 1 | b2 : b0 << 3 | b1 << 2 | b3 << 1 | b2;
    }
    template <int W>
    __device__ __forceinline__ static int state_piece(int row, int q) { return row * (2 * W) + ((q ^ state_sw<W>(row)) << 4); }
    template <int W>
    __device__ __forceinline__ static int state_column(int row, int slot) { return 8 * (slot ^ state_sw<W>(row)); }
    __device__ __forceinline__ static int state_row(int i, int g4) { return 32 * (i >> 1) + 8 * g4 + 4 * ((i & 1) ^ (g4 & 1)); }
    template <int W>
    __device__ __forceinline__ static Frag<1> state_rows(const uint8_t* t, int r0, int kk, int li, int g4) {
        Frag<1> f;
        f.p[0] = lds<bf8>(t + r0 * (2 * W) + (state_piece<W>(li, g4) ^ (kk << 6)));
        return f;
    }
    template <int W>
    __device__ __forceinline__ static Frag<1> state_columns(const uint8_t* t, int r0, int i, int li, int g4) {
        const int j = li & 3, row = 4 * g4 + (li >> 2);
        const uint8_t* p = t + r0 * (2 * W) + ((state_piece<W>(row, j) + 8 * (j & 1)) ^ ((i >> 1) << 6) ^ ((i & 1) << 3));
        Frag<1> f;
        f.p[0] = join(tr_read(p), tr_read(p + 16 * 2 * W));
        return f;
    }
    template <int PARTS>
    __device__ __forceinline__ static Frag<PARTS> of_state(const f4* tile, int kk, int g4) {
        const f4 lo = tile[2 * kk], hi = tile[2 * kk + 1];
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = g4 & 1 ? hi[e] : lo[e];
            v[4 + e] = g4 & 1 ? lo[e] : hi[e];
        }
        return parts<PARTS>(v);
    }
    // left operand, columns 16 c + li as rows, contraction over the tile's rows r0 .. r0 + KB in token order
    template <int W>
    __device__ __forceinline__ static Frag<1> columns(const uint8_t* t, int r0, int c, int li, int g4) {
        Frag<1> f;
        f.p[0] = down<2 * W>(t, down_off<2 * W>(4 * g4, li), r0, c);
        return f;
    }
    template <int W>
    __device__ __forceinline__ static float at(const uint8_t* t, int row, int col) {
        return bf16_to_f32(lds<uint16_t>(t + piece<2 * W>(row, col >> 3) + 2 * (col & 7)));
    }
    // rows r0 + 4 g4 .. + 3 of column 16 c + li
    template <int W>
    __device__ __forceinline__ static f4 four_rows(const uint8_t* t, int r0, int c, int li, int g4) {
        const u2 v = __builtin_bit_cast(u2, tr_read(t + r0 * (2 * W) + (down_off<2 * W>(4 * g4, li) ^ (c << 5))));
        return f4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                  __uint_as_float(v[1] & 0xFFFF0000u)};
    }
    template <int W>
    __device__ __forceinline__ static void put(uint8_t* t, int row, int col, float v) {
        *reinterpret_cast<uint16_t*>(t + piece<2 * W>(row, col >> 3) + 2 * (col & 7)) = f32_to_bf16(v);
    }
    // values n .. n + R of a row of N (a multiple of 4), zeros past its end
    __device__ __forceinline__ static u4 load_run(const S* p, int n, int N) {
        u4 v{0, 0, 0, 0};
        if (n + 8 <= N) {
            v = *reinterpret_cast<const u4any*>(p + n);
        } else if (n < N) {
            const u2 h = *reinterpret_cast<const u2any*>(p + n);
            v[0] = h[0];
            v[1] = h[1];
        }
        return v;
    }
    __device__ __forceinline__ static Frag<1> exact(u4 v) {
        Frag<1> f;
        f.p[0] = __builtin_bit_cast(bf8, v);
        return f;
    }
    __device__ __forceinline__ static bool not_finite(const Frag<1>& f) {
        const u4 v = __builtin_bit_cast(u4, f.p[0]);
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) bad = bad || (v[i] & 0x7F800000u) == 0x7F800000u || (v[i] & 0x7F80u) == 0x7F80u;
        return bad;
    }
};

// ---------------------------------------------------------------------------------------
// fp32: the same operands, whole (the number of parts says nothing here)
// ---------------------------------------------------------------------------------------
typedef uint32_t u4any4 __attribute__((ext_vector_type(4), aligned(4)));  // any fp32 address
struct ByF32 {
    using S = float;
    static constexpr int Q = 32;
    static constexpr int KB = 16;
    static constexpr int R = 4;
    static constexpr int TP = 1;
    template <int PARTS>
    struct Frag {
        f4 v;
    };
    template <int PARTS>
    __device__ __forceinline__ static Frag<PARTS> parts(const float (&v)[4]) {
        return {f4{v[0], v[1], v[2], v[3]}};
    }
    template <int PARTS>
    __device__ __forceinline__ static Frag<PARTS> of_tiles(const f4* tile, int kk) {
        return {tile[kk]};
    }
    // one 16 x 16 x 4 instruction a value: lane groups g4 hold k = 4 g4 + e
    template <int PA, int PB>
    __device__ __forceinline__ static void mac(f4& c, const Frag<PA>& a, const Frag<PB>& b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    }
    __device__ __forceinline__ static float value(const S* p, int64_t i) { return p[i]; }
    __device__ __forceinline__ static void store(S* p, int64_t i, float v) { p[i] = v; }

    // LDS tiles of W columns: rows of W + 4 floats, so that 16 rows, and every fourth row, start at
    // banks of their own
    template <int W>
    static constexpr int tile_bytes(int rows) { return rows * (W + 4) * 4; }
    template <int W>
    __device__ __forceinline__ static int piece_at(int row, int q) { return (row * (W + 4) + 4 * q) * 4; }
    template <int W>
    __device__ __forceinline__ static Frag<1> rows(const uint8_t* t, int r0, int kk, int li, int g4) {
        return {lds<f4>(t + piece_at<W>(r0 + li, 4 * kk + g4))};
    }
    template <int W>
    __device__ __forceinline__ static Frag<1> along(const uint8_t* t, int r0, int kk, int li, int g4) {
        return rows<W>(t, r0, kk, li, g4);
    }
    template <int W>
    __device__ __forceinline__ static Frag<1> columns(const uint8_t* t, int r0, int c, int li, int g4) {
        Frag<1> f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[e] = lds<float>(t + ((r0 + 4 * g4 + e) * (W + 4) + 16 * c + li) * 4);
        return f;
    }
    template <int W>
    __device__ __forceinline__ static float at(const uint8_t* t, int row, int col) {
        return lds<float>(t + (row * (W + 4) + col) * 4);
    }
    template <int W>
    __device__ __forceinline__ static f4 four_rows(const uint8_t* t, int r0, int c, int li, int g4) {
        return columns<W>(t, r0, c, li, g4).v;
    }
    template <int W>
    __device__ __forceinline__ static void put(uint8_t* t, int row, int col, float v) {
        *reinterpret_cast<float*>(t + (row * (W + 4) + col) * 4) = v;
    }
    template <int W>
    __device__ __forceinline__ static int column_of(int, int s) { return 4 * s; }
    template <int W>
    __device__ __forceinline__ static int state_piece(int row, int q) { return piece_at<W>(row, q); }
    template <int W>
    __device__ __forceinline__ static int state_column(int, int slot) { return 4 * slot; }
    __device__ __forceinline__ static int state_row(int i, int g4) { return 16 * i + 4 * g4; }
    template <int W>
    __device__ __forceinline__ static Frag<1> state_rows(const uint8_t* t, int r0, int kk, int li, int g4) {
        return rows<W>(t, r0, kk, li, g4);
    }
    template <int W>
    __device__ __forceinline__ static Frag<1> state_columns(const uint8_t* t, int r0, int i, int li, int g4) {
        return columns<W>(t, r0, i, li, g4);
    }
    template <int PARTS>
    __device__ __forceinline__ static Frag<PARTS> of_state(const f4* tile, int kk, int) {
        return {tile[kk]};
    }
    __device__ __forceinline__ static u4 load_run(const S* p, int n, int N) {
        u4 v{0, 0, 0, 0};
        if (n < N) v = *reinterpret_cast<const u4any4*>(p + n);
        return v;
    }
    __device__ __forceinline__ static Frag<1> exact(u4 v) { return {__builtin_bit_cast(f4, v)}; }
    __device__ __forceinline__ static bool not_finite(const Frag<1>& f) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) bad = bad || !__builtin_isfinite(f.v[i]);
        return bad;
    }
};

// T and M in the workspace and in LDS: left operands as the instruction takes them, 64 lanes x 16 bytes
// a part, of the 16-row tiles rt and contraction blocks kk that are not all 0, rt slowest.  As they
// are: rows t, contraction over s <= t.  Transposed: rows s, contraction over t >= s.
template <class MM>
constexpr int first_frag(int rt, bool transposed) {
    int n = 0;
    for (int r = 0; r < rt; ++r)
        n += transposed ? MM::Q / MM::KB - 16 * r / MM::KB : 16 * r / MM::KB + 1;
    return n;
}
template <class MM>
constexpr int frag_count() { return first_frag<MM>(MM::Q / 16, false); }
template <class MM>
constexpr int frag_at(int rt, int kk, bool transposed) {
    return first_frag<MM>(rt, transposed) + kk - (transposed ? 16 * rt / MM::KB : 0);
}
template <class MM>
constexpr int image_bytes(int parts) { return parts * frag_count<MM>() * 1024; }

// one part of an operand kept as PARTS tiles behind each other
template <class MM, int PARTS, class F>
__device__ __forceinline__ typename MM::template Frag<PARTS> of_parts(F load) {
    typename MM::template Frag<PARTS> f;
    if constexpr (MM::TP == 1) {
        f.v = load(0).v;
    } else {
#pragma unroll
        for (int i = 0; i < PARTS; ++i) f.p[i] = load(i).p[0];
    }
    return f;
}
template <class MM, int PARTS>
__device__ __forceinline__ typename MM::template Frag<PARTS> frag(const uint8_t* image, int at, int lane) {
    return of_parts<MM, PARTS>([&](int q) { return MM::exact(lds<u4>(image + (at * PARTS + q) * 1024 + lane * 16)); });
}

// Raw buffers: loads past the end give 0, stores past it are dropped.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr int kOutside = 0x7FFFFFF0;
__device__ __forceinline__ Buffer buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}
// token rows from t0 on that a chunk has, of `width` elements; rows times stride within 31 bits (DeltaArgs::direct)
template <class S>
__device__ __forceinline__ Buffer token_buffer(const void* p, int64_t t0, int64_t row, int64_t col, int valid, int64_t width) {
    return buffer(static_cast<const S*>(p) + t0 * row + col, ((valid - 1) * row + width) * sizeof(S));
}
// 64 x 16 bytes straight into 1 KB of LDS, lane l at byte 16 l
__device__ __forceinline__ void to_lds(Buffer r, uint32_t at, uint8_t* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, at, 0, 0, 0);
}
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)
// LDS reads are done before anything behind this (direct loads into LDS do not wait for them)
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// an element as it lies in memory; value_of where it is used, which is where the load is waited for
template <class S>
__device__ __forceinline__ S load_at(Buffer r, uint32_t at) {
    if constexpr (sizeof(S) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
    else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
}
__device__ __forceinline__ float value_of(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float value_of(float v) { return v; }
template <class S>
__device__ __forceinline__ void store_at(Buffer r, uint32_t at, float v) {
    if constexpr (sizeof(S) == 2) __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v), r, at, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at, 0, 0);
}

// LDS of a tile of W columns that one wavefront stages: whole kilobytes
template <class MM, int W>
constexpr int staged_bytes() { return (MM::template tile_bytes<W>(MM::Q) + 1023) / 1024 * 1024; }
// a tile's rows straight into LDS by WAVES wavefronts (w of them): N columns, zeros past them and past the rows
template <class MM, int W, bool STATE, int WAVES = 1>
__device__ __forceinline__ void direct_rows(uint8_t* tile, Buffer r, int row, int N, int lane, int w = 0) {
    constexpr int ES = sizeof(typename MM::S), SLOTS = MM::template tile_bytes<W>(MM::Q) / MM::Q / 16;
#pragma unroll
    for (int at = 0; at < staged_bytes<MM, W>() / 1024; at += WAVES) {
        const int i = at + w;
        if (WAVES > 1 && i >= staged_bytes<MM, W>() / 1024) continue;
        const int slot = 64 * i + lane, t = slot / SLOTS;
        const int n = STATE ? MM::template state_column<W>(t, slot % SLOTS) : MM::template column_of<W>(t, slot % SLOTS);
        to_lds(r, t < MM::Q && n < N ? (t * row + n) * ES : kOutside, tile + 1024 * i);
    }
}
// an image's kilobytes by one wavefront
template <int BYTES>
__device__ __forceinline__ void direct_image(uint8_t* to, const uint8_t* from, int lane) {
    const Buffer r = buffer(from, BYTES);
#pragma unroll
    for (int i = 0; i < (BYTES + 1023) / 1024; ++i) to_lds(r, i * 1024 + lane * 16, to + i * 1024);
}

// Q rows of W columns from global memory (rows `row` elements apart, `valid` of them, N columns;
// zeros elsewhere) into a tile, or one that a state is multiplied with
template <class MM, int W, int THREADS, bool STATE>
__device__ __forceinline__ void stage_rows(uint8_t* tile, const typename MM::S* src, int64_t row, int valid, int N) {
    constexpr int E = 16 / sizeof(typename MM::S), PIECES = W / E;
    for (int i = threadIdx.x % THREADS; i < MM::Q * PIECES; i += THREADS) {
        const int r = i / PIECES, q = i % PIECES;
        u4 v{0, 0, 0, 0};
        if (r < valid) v = MM::load_run(src + r * row, q * E, N);
        *reinterpret_cast<u4*>(tile + (STATE ? MM::template state_piece<W>(r, q) : MM::template piece_at<W>(r, q))) = v;
    }
}
// Q rows of 64 columns, `have` of them, element by element (rows that are not whole pieces)
template <class MM, int THREADS>
__device__ __forceinline__ void stage_elements(uint8_t* tile, const typename MM::S* src, int64_t row, int valid, int have) {
    for (int i = threadIdx.x % THREADS; i < MM::Q * 64; i += THREADS)
        MM::template put<64>(tile, i / 64, i % 64, i / 64 < valid && i % 64 < have ? MM::value(src + (i / 64) * row, i % 64) : 0.0f);
}

// A NaN or infinity of one packed sequence times the 0 that keeps the sequences apart would reach the
// others, and with the state the chunks that those go on in.  So where a chunk holds several sequences
// and an operand of a product over its tokens is not finite, such values are 0 in the product and the
// rows of their sequences NaN in its result, and rows of K and Q whose factor is 0 are cleared before
// they enter the state.
template <int RT>
__device__ __forceinline__ bool all_finite(const f4 (&v)[RT]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s += v[i][e] * 0.0f;
    return __all(s == 0.0f);
}
// MM::of_tiles of finite values, 0 for the others
template <class MM, int PARTS, bool FINITE, int RT>
__device__ __forceinline__ typename MM::template Frag<PARTS> finite_tiles(const f4 (&v)[RT], int kk) {
    if constexpr (!FINITE) {
        return MM::template of_tiles<PARTS>(v, kk);
    } else {
        constexpr int N = MM::KB / 16;
        f4 t[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[i][e] = __builtin_isfinite(v[N * kk + i][e]) ? v[N * kk + i][e] : 0.0f;
        return MM::template of_tiles<PARTS>(t, 0);
    }
}
// all rows of the sequences that have one of `rows` (starts: a bit for each sequence's first row but the chunk's)
__device__ __forceinline__ uint64_t whole_sequences(uint64_t rows, uint64_t starts) {
    uint64_t all = 0;
    for (int from = 0; from < 64;) {  // as many rounds as sequences
        const int to = starts ? __builtin_ctzll(starts) : 64;
        starts &= starts - 1;
        const uint64_t own = (~0ull >> (64 - (to - from))) << from;
        all |= rows & own ? own : 0;
        from = to;
    }
    return all;
}
// After out += product of in's finite values: the rows of the sequences (begun: of the chunk's Q tokens) that have
// others in the lane's column
template <bool STARTS, int Q, int RT>
__device__ __forceinline__ void mark_sequences(f4 (&out)[RT], const f4 (&in)[RT], const float* begun, int lane) {
    if (!STARTS || all_finite(in)) return;
    const int g4 = lane >> 4;
    unsigned long long rows = 0;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) rows |= static_cast<unsigned long long>(!__builtin_isfinite(in[i][e])) << (16 * i + e);
    rows <<= 4 * g4;
    rows |= __shfl_xor(rows, 16);
    rows |= __shfl_xor(rows, 32);
    const uint64_t starts = __ballot(lane > 0 && lane < Q && begun[lane < Q ? lane : 0] != begun[lane > 0 && lane < Q ? lane - 1 : 0]);
    rows = whole_sequences(rows, starts) >> (4 * g4);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][e] = rows >> (16 * i + e) & 1 ? __builtin_nanf("") : out[i][e];
}
// Products with the factors of a chunk's tokens.  Only where a sequence starts within the chunk (STARTS) is
// a factor 0 by more than underflow: there it leaves nothing of what is not finite either.
template <bool STARTS, int RT>
__device__ __forceinline__ void scale_rows(f4 (&v)[RT], const float* factor, float more, int g4) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const f4 f = lds<f4>(reinterpret_cast<const uint8_t*>(factor + 16 * i + 4 * g4));
        v[i] *= f * more;
        if (STARTS) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = f[e] != 0.0f ? v[i][e] : 0.0f;
        }
    }
}
// (with a start the state before the chunk does not reach its end)
template <bool STARTS, int NT>
__device__ __forceinline__ void scale_state(f4 (&v)[NT], float through) {
#pragma unroll
    for (int i = 0; i < NT; ++i) v[i] = STARTS && through == 0.0f ? f4{0, 0, 0, 0} : v[i] * through;
}

// A unit row's walk through a segment of gates above 0 may pass fp32's range where the state that it is multiplied
// with is 0 or small.  So the row keeps a power of 2, from 0 on, that holds its largest value below 2.
template <int NT>
__device__ __forceinline__ void keep_in_range(f4 (&row)[NT], int& power) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(row[i][e]));
    if (!__any(most >= 2.0f || power > 0)) return;
    most = fmaxf(most, __shfl_xor(most, 16));
    most = fmaxf(most, __shfl_xor(most, 32));
    // (a row that is 0 or not finite stays as it is)
    const int want = most > 0.0f && most < __builtin_inff() ? max(power + __builtin_amdgcn_frexp_expf(most) - 1, 0) : power;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) row[i][e] = __builtin_ldexpf(row[i][e], power - want);
    power = want;
}

// rows of a tile whose factor is 0, by the four wavefronts that walk
template <class MM, int W>
__device__ __forceinline__ void clear_rows(uint8_t* tile, const float* factor) {
    constexpr int PIECES = W * sizeof(typename MM::S) / 16;
    for (int i = threadIdx.x; i < MM::Q * PIECES; i += 256)
        if (factor[i / PIECES] == 0.0f) *reinterpret_cast<u4*>(tile + MM::template state_piece<W>(i / PIECES, i % PIECES)) = u4{0, 0, 0, 0};
}

// Blocks are dealt round-robin over the 8 XCDs: neighbours in the result run on one XCD and share
// its L2.
__device__ __forceinline__ int xcd_order(int block, int blocks) {
    const int x = block & 7, per = blocks >> 3, more = blocks & 7;
    return x * per + (x < more ? x : more) + (block >> 3);
}

// Of the chunk's token `lane`: the sum of the gates from the chunk's start on, or from its sequence's where that
// starts within the chunk (a first token's gate counts for nothing), the packed sequences begun since the chunk's
// start, and beta (tokens behind the row: gate 0, beta 0).  Sums of two tokens are compared within a sequence only,
// and what one sequence's gates hold is not in the next one's.  All 64 lanes call it.
struct TokenSums {
    double gates;
    int starts;
    float beta;
};
template <int Q>
__device__ __forceinline__ TokenSums token_sums(const DeltaArgs& a, int64_t b, int64_t h, int64_t t0, int valid, int lane) {
    TokenSums s{0.0, 0, 0.0f};
    if (lane < valid) {
        const int64_t t = b * a.L + t0 + lane;
        s.beta = a.beta[t * a.H + h];
        if (a.seq && t0 + lane > 0) s.starts = a.seq[t] != a.seq[t - 1];
        if (a.gate && s.starts == 0) s.gates = gate_of(a.gate[t * a.H + h]);
    }
#pragma unroll
    for (int d = 1; d < Q; d <<= 1) {
        const double o = __shfl_up(s.gates, d);
        const int r = __shfl_up(s.starts, d);
        if (lane >= d) {
            s.gates += s.starts == 0 ? o : 0.0;  // (starts among the d tokens up to this one)
            s.starts += r;
        }
    }
    return s;
}

// (rows that overlap, a token that stands for all of them say, do not end where a buffer of them ends)
inline bool direct_rows_fit(const void* p, int64_t row, int64_t width, size_t es) {
    return row >= width && row < (int64_t{1} << 30) / 64 / static_cast<int64_t>(es) &&
           reinterpret_cast<uintptr_t>(p) % 16 == 0 && row * es % 16 == 0;
}

// Rows are cut into segments where their walks do not fill the 256 CUs: all segments from zero, with the
// N unit rows as further channels that give what a segment makes of the state before it; the states
// before the segments from those; then the walk proper, all segments side by side.  The cut is the
// one with the smallest sum of its walks' rounds, in units fitted to calls in bf16 of 512 to 32845 tokens, dstate 64
// and 128 (a choice between cuts, not microseconds; fp32 and other widths take it as it is): a chunk
// 2.5 uncut, 2.0 (from zero) and 2.9 forward; 5.7 uncut, 2.0 (from zero) and 8.7 (three walks) backward; 2 a
// segment and walk for the states between, 10 a direction for the launches.  (bf16, 1024 tokens of 8 heads x
// 64 x 128 backward: 131 us cut, 166 uncut; of 8 rows of 4 heads forward: 70 us cut, 65 uncut.)
inline void plan_segments(DeltaArgs& a, bool bwd) {
    const int64_t units = a.B * a.H, own = (a.P + 63) / 64, all = own + (a.N + 63) / 64;
    const auto rounds = [](int64_t blocks) { return static_cast<double>((blocks + 255) / 256); };
    a.segs = 1;
    a.seg_chunks = a.chunks;
    double best = rounds(units * own) * a.chunks * (bwd ? 5.7 : 2.5);
    for (int64_t n = 2; n <= 64 && n * 4 <= a.chunks; ++n) {
        const int64_t each = (a.chunks + n - 1) / n;
        if ((a.chunks + each - 1) / each != n) continue;
        const double t = rounds(units * all * n) * each * 2.0 + rounds(units * own * n) * each * (bwd ? 8.7 : 2.9) +
                         n * (bwd ? 4.0 : 2.0) + (bwd ? 20.0 : 10.0);
        if (t < best) {
            best = t;
            a.segs = n;
            a.seg_chunks = each;
        }
    }
}

// the chunks' part of the workspace; returns its bytes
template <class MM>
size_t place_chunks(DeltaArgs& a, uint8_t* ws, bool bwd) {
    a.chunks = (a.L + MM::Q - 1) / MM::Q;
    const size_t n = static_cast<size_t>(a.B * a.H * a.chunks);
    size_t at = 0;
    a.T = ws;
    at += n * image_bytes<MM>(MM::TP);
    a.M = ws + at;
    at += n * image_bytes<MM>(MM::TP);
    a.Tt = ws + at;
    if (bwd) at += n * image_bytes<MM>(MM::TP);
    a.factors = reinterpret_cast<float*>(ws + at);
    at += n * kFactors * MM::Q * 4;
    a.gates = reinterpret_cast<double*>(ws + at);
    at += bwd ? n * MM::Q * 8 : 0;
    plan_segments(a, bwd);
    const size_t states = a.segs > 1 ? static_cast<size_t>(a.B * a.H * a.segs) : 0;
    a.phi = reinterpret_cast<float*>(ws + at);
    at += states * a.N * a.N * 4;
    a.power = reinterpret_cast<int32_t*>(ws + at);
    at += states * a.N * 4;
    a.gain = reinterpret_cast<float*>(ws + at);
    at += states * a.P * a.N * 4;
    a.entry = reinterpret_cast<float*>(ws + at);
    at += states * a.P * a.N * 4;
    return (at + 255) / 256 * 256;
}

}  // namespace delta

// what the backward keeps of a walk: the state before every chunk, and E (and T and M transposed)
struct DeltaSaved {
    float* states;  // [B, H, chunks, P, N]
    float* e;       // [B, L, H, P]
};
hipError_t launch_delta_walk_saved(const DeltaArgs& a, const DeltaSaved& s, ssm_dtype_t dtype, hipStream_t stream);
// the gradients of the states after the segments
hipError_t launch_delta_join_back(const DeltaArgs& a, ssm_dtype_t dtype, hipStream_t stream);
// of sizes whose products stay within 63 bits
bool delta_launches_fit(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype, bool bwd);
size_t delta_fwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype);
size_t delta_bwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype);
hipError_t launch_delta_fwd(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream);
hipError_t launch_delta_bwd(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream);
// token by token on state slots (row b's state at state + slot * H * P * N)
struct DeltaStep {
    DeltaArgs a;
    float* state;
    const int32_t* slots;  // [B] or NULL (slot b)
    int64_t n_slots;
};
hipError_t launch_delta_step(const DeltaStep& s, ssm_dtype_t dtype, hipStream_t stream);

}  // namespace ssm
