// gscan.hip -- the per-channel gated recurrence (ssm_gated_scan_fwd, ssm_gated_scan_bwd,
// ssm_gated_scan_step): length-generalization reading notes, Sec. 2.1 Eq. (1) with a state of
// one value per channel, per channel c of row b
//     h_t = a_t h_{t-1} + i_t x_t,    y_t = h_t
// with a = e^g, i = 1 (log form) or a = sigmoid(g), i = 1 - a = sigmoid(-g) (sigmoid form),
// from h_{-1} = the initial state; a_t counts as 0 where a packed sequence starts.  Backward,
// with E_t the gradient that token t hands to h_{t-1}:
//     D_t = dy_t + E_{t+1},  E_t = a_t D_t (0 at a start),  E_L = d(final state),
//     dx_t = i_t D_t,  dlog a_t = D_t a_t h_{t-1},  d(initial state) = E_0,
//     dg_t = dlog a_t  or  i_t dlog a_t - D_t x_t i_t a_t.
//
// Bound by memory, so the recurrence is cut along the row to keep the GPU full, and joined
// again on chip: h over a span of tokens is A h_in + H (Sec. 2.5 Eq. (4): A the product of its
// decays, H its own tokens' share).  A block takes 64 channels (one a lane) of one row and
// walks over tiles of 128 tokens, 8 wavefronts of 16 tokens each: every wavefront forms its
// (A, H), and (A, E) backward, from registers, the 8 spans are joined through LDS, and a
// second walk over the registers applies the state that comes in.  So a tile is read once.
// The next tile's loads are issued before the current one is worked on.  4 x 8192 tokens x 4096
// channels, bf16, sigmoid form, packed: 200 us (0.80 GB, 4.0 TB/s), 158 us with all loads from
// one tile: the instructions (nine a token and lane for the gates alone, two of them at a
// quarter of the rate) bound it as much as the traffic.  16 wavefronts of 8 tokens join twice
// the spans for the same tokens: 221 us.
//
// Rows and channels too few to fill the GPU (under kFill blocks) are cut into segments of
// tiles: a first kernel joins each segment to one (A, H), which reads the inputs once more,
// and each block of the second folds the segments before (and behind) its own.  One row of
// 65573 tokens x 333 channels, fp32, log form: 37 + 69 us.
// The backward needs h before each tile: its first kernel walks forward and stores (A, H) from
// the segment's start to each tile's (8 bytes a channel and 128 tokens).  At the size above
// 161 + 326 us (0.56 + 1.36 GB).
//
// A span that holds a sequence start passes nothing on; it is marked by A = -1 (a product of
// decays is never negative) and folded by a select, so a NaN or infinity of one sequence does
// not reach the next.  Everything is fp32; outputs are rounded once.
#include <type_traits>

#include "internal.h"

namespace ssm {
namespace {

constexpr int kGW = 8;              // wavefronts a block
constexpr int kGT = 16;             // tokens a wavefront and tile
constexpr int kGTile = kGW * kGT;   // 128
constexpr int kGThreads = 64 * kGW;

struct GArgs {
    const void *x, *gate, *dy;
    void *y, *dx, *dgate;
    int64_t x_row, gate_row, dy_row, y_row, dx_row, dgate_row;  // token strides (elements)
    const float *h0, *dhT;
    float *final_state, *dh0;
    const int32_t* seq;
    int64_t B, L, C;
    int64_t tiles, nseg, seg_tiles;
    float* seg;   // [B][nseg][3][C]: A, H, E of each segment (forward: the initial state in segment 0's E)
    float* ckpt;  // [B][tiles][2][C]: A, H from the segment's start to the tile's
};

// decay a and input factor i of a gate: e = exp(-g), a = 1 / (1 + e) and i = e a keep both to full
// relative accuracy; e is held below 2^126, where 1 / (1 + e) is still a normal number
template <bool SIG>
__device__ __forceinline__ void gates(float g, float& a, float& i) {
    if constexpr (SIG) {
        const float z = g * -1.44269504f;
        const float e = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(z, 126.0f));  // NaN stays NaN
        a = __builtin_amdgcn_rcpf(1.0f + e);
        i = e * a;
    } else {
        a = __expf(g);
        i = 1.0f;
    }
}

// h after a span (A, H); MARKS: A may be the mark of a span that passes nothing on
template <bool MARKS>
__device__ __forceinline__ float fold(float A, float H, float h) {
    return MARKS && A < 0.0f ? H : A * h + H;
}
template <bool MARKS>
__device__ __forceinline__ float fold_mark(float A, float P) {
    return MARKS && (P < 0.0f || A < 0.0f) ? -1.0f : P * A;
}

// a wavefront's tokens of one tile, as loaded; token i is row tok0 + i of the row b.  SEQ: the rows
// are packed
template <class S, bool DY, bool SEQ>
struct GRaw {
    static constexpr bool kSeq = SEQ;
    typename S::T x[kGT], g[kGT], d[DY ? kGT : 1];
    int32_t id;  // lane j: sequence id of token tok0 - 1 + j
};

struct GPos {
    int64_t b, c;
    int lane, wave;
    bool live;  // the lane's channel exists
};

// A 32-bit lane offset that stays one: added to a uniform base it is part of the access (left to
// itself the compiler widens it once and adds 64 bits for every token)
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}
template <class T>
__device__ __forceinline__ T g_at(const char* token, uint32_t lane_bytes) {
    return *reinterpret_cast<const T*>(token + lane_bytes);
}
template <class S, bool DY, bool SEQ>
__device__ __forceinline__ void g_load(const GArgs& a, const GPos& p, int64_t tile, GRaw<S, DY, SEQ>& r) {
    using T = typename S::T;
    const int64_t t0 = tile * kGTile + p.wave * kGT, row0 = p.b * a.L;
    const uint32_t lb = here(static_cast<uint32_t>(p.c) * static_cast<uint32_t>(sizeof(T)));
    // tokens past the row's end: its last one, read and not used
    const int64_t from = row0 + (t0 < a.L ? t0 : a.L - 1);
    // tokens of this wavefront behind its first
    const int left = a.L - 1 - t0 < kGT ? (a.L - 1 > t0 ? static_cast<int>(a.L - 1 - t0) : 0) : kGT;
    const char* x = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + from * a.x_row);
    const char* g = reinterpret_cast<const char*>(static_cast<const T*>(a.gate) + from * a.gate_row);
    const char* d = DY ? reinterpret_cast<const char*>(static_cast<const T*>(a.dy) + from * a.dy_row) : nullptr;
    // in the order of their use: a wait for one load is a wait for those before it
    if constexpr (SEQ) {
        int64_t t = t0 - 1 + p.lane;
        t = t < 0 ? 0 : t < a.L ? t : a.L - 1;
        r.id = a.seq[row0 + t];
    }
    auto rows = [&](const char* p, int64_t step, typename S::T (&v)[kGT]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kGT; ++i) {
            v[i] = g_at<T>(p, lb);
            p += step & -static_cast<int64_t>(i < left);
        }
    };
    rows(g, sizeof(T) * a.gate_row, r.g);
    rows(x, sizeof(T) * a.x_row, r.x);
    if constexpr (DY) rows(d, sizeof(T) * a.dy_row, r.d);
}

// bit i: token i starts a sequence (token 0 of the row never does)
template <class R>
__device__ __forceinline__ uint32_t g_starts(const GArgs& a, const GPos& p, int64_t tile, const R& r) {
    if constexpr (!R::kSeq) return 0;
    const int64_t t = tile * kGTile + p.wave * kGT - 1 + p.lane;
    const int32_t before = __shfl_up(r.id, 1);
    const uint64_t m = __ballot(p.lane >= 1 && p.lane <= kGT && t > 0 && t < a.L && r.id != before);
    return static_cast<uint32_t>(m >> 1);
}

__device__ __forceinline__ int g_valid(const GArgs& a, const GPos& p, int64_t tile) {
    const int64_t n = a.L - (tile * kGTile + p.wave * kGT);
    return n < 0 ? 0 : n < kGT ? static_cast<int>(n) : kGT;
}

__device__ __forceinline__ GPos g_pos(const GArgs& a, int64_t row_group) {
    GPos p;
    p.lane = threadIdx.x & 63;
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t groups = (a.C + 63) / 64;
    p.b = row_group / groups;
    const int64_t c = (row_group % groups) * 64 + p.lane;
    p.live = c < a.C;
    p.c = p.live ? c : a.C - 1;
    return p;
}

__device__ __forceinline__ float seg_at(const GArgs& a, const GPos& p, int64_t s, int k) {
    return a.seg[((p.b * a.nseg + s) * 3 + k) * a.C + p.c];
}

// Folds the pairs (A, value k) of the segments s0, s0 + ds, .. (n of them) onto v: every wavefront
// takes a share of them, eight loads in flight, and the shares are joined in `buf`.
__device__ __forceinline__ float fold_segments(const GArgs& a, const GPos& p, float2 (&buf)[kGW][64],
                                               int64_t s0, int64_t ds, int64_t n, int k, float v) {
    if (n == 0) return v;
    const int64_t share = (n + kGW - 1) / kGW;
    const int64_t to = (p.wave + 1) * share < n ? (p.wave + 1) * share : n;
    float P = 1.0f, X = 0.0f;
    for (int64_t s = p.wave * share; s < to; s += 8) {
        float A[8], V[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = s0 + ds * (s + j < to ? s + j : to - 1);
            A[j] = seg_at(a, p, at, 0);
            V[j] = seg_at(a, p, at, k);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float Aj = s + j < to ? A[j] : 1.0f, Vj = s + j < to ? V[j] : 0.0f;
            X = fold<true>(Aj, Vj, X);
            P = fold_mark<true>(Aj, P);
        }
    }
    buf[p.wave][p.lane] = make_float2(P, X);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kGW; ++w) v = fold<true>(buf[w][p.lane].x, buf[w][p.lane].y, v);
    return v;
}

// decays and input factors of the tile's tokens in this wavefront: past the row's end a = 1, i = 0
template <class S, bool SIG, class R>
__device__ __forceinline__ void g_gates(const R& r, int nv, float (&av)[kGT], float (&in)[kGT]) {
#pragma unroll
    for (int i = 0; i < kGT; ++i) gates<SIG>(S::load(r.g, i), av[i], in[i]);
    if (nv < kGT) {
#pragma unroll
        for (int i = 0; i < kGT; ++i)
            if (i >= nv) {
                av[i] = 1.0f;
                in[i] = 0.0f;
            }
    }
}
// inputs i x (x is finite or not: past the end 0)
template <class S, class R>
__device__ __forceinline__ void g_inputs(const R& r, int nv, const float (&in)[kGT], float (&uv)[kGT]) {
#pragma unroll
    for (int i = 0; i < kGT; ++i) uv[i] = in[i] * S::load(r.x, i);
    if (nv < kGT) {
#pragma unroll
        for (int i = 0; i < kGT; ++i)
            if (i >= nv) uv[i] = 0.0f;
    }
}

// (A, H) of the wavefront's tokens
__device__ __forceinline__ float2 g_span(const float (&av)[kGT], const float (&uv)[kGT], uint32_t st) {
    float A = av[0], H = uv[0];
    if (st == 0) {
#pragma unroll
        for (int i = 1; i < kGT; ++i) {
            H = av[i] * H + uv[i];
            A *= av[i];
        }
    } else {
#pragma unroll
        for (int i = 1; i < kGT; ++i) H = (st >> i) & 1 ? uv[i] : av[i] * H + uv[i];
        A = -1.0f;
    }
    return make_float2(A, H);
}

// E that the wavefront's tokens hand to the token before them, with E = 0 behind them
template <class S, class R>
__device__ __forceinline__ float g_back(const R& r, int nv, const float (&av)[kGT], uint32_t st) {
    float e = 0.0f;
    if (st == 0 && nv == kGT) {
#pragma unroll
        for (int i = kGT - 1; i >= 0; --i) e = av[i] * (S::load(r.d, i) + e);
    } else {
#pragma unroll
        for (int i = kGT - 1; i >= 0; --i) {
            const float d = (i < nv ? S::load(r.d, i) : 0.0f) + e;
            e = (st >> i) & 1 ? 0.0f : av[i] * d;
        }
    }
    return e;
}

// whether any span of the tile is marked (uniform); A as stored by the 16 wavefronts
template <bool SEQ>
__device__ __forceinline__ bool g_marked(const float2 (&s)[kGW][64], int lane) {
    return SEQ && __ballot(s[lane % kGW][0].x < 0.0f) != 0;
}

// ---------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------
// AGG: only the segment's (A, H), for the join (nseg > 1); else y and the final state.
template <class S, bool SIG, bool SEQ, bool AGG>
__global__ void __launch_bounds__(kGThreads) gscan_fwd_kernel(GArgs a) {
    __shared__ float2 sp[2][kGW][64];
    const int64_t nseg = AGG ? a.nseg - 1 : a.nseg;  // the last segment's (A, H) is not needed
    const int64_t seg = blockIdx.x % nseg;
    const GPos p = g_pos(a, blockIdx.x / nseg);
    const int64_t first = seg * a.seg_tiles;
    const int64_t last = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
    GRaw<S, false, SEQ> cur;
    g_load(a, p, first, cur);
    float carry = 0.0f, P = 1.0f;
    if (AGG) {
        // final_state may be initial_state itself: the second kernel, whose last segment writes
        // it while others may not have begun, takes the initial state from here
        if (seg == 0 && p.wave == 0 && p.live)
            a.seg[(p.b * a.nseg * 3 + 2) * a.C + p.c] = a.h0 ? a.h0[p.b * a.C + p.c] : 0.0f;
    } else {
        if (a.nseg > 1) carry = seg_at(a, p, 0, 2);
        else if (a.h0) carry = a.h0[p.b * a.C + p.c];
        carry = fold_segments(a, p, sp[(first & 1) ^ 1], 0, 1, seg, 1, carry);
        // every wavefront has its initial state in hand before the first barrier, hence before
        // wavefront 0 stores the final state
        asm volatile("" : "+v"(carry));
    }
    auto step = [&](int64_t tile, const GRaw<S, false, SEQ>& cur, GRaw<S, false, SEQ>& nxt) __attribute__((always_inline)) {
        g_load(a, p, tile + 1 < last ? tile + 1 : tile, nxt);
        const int nv = g_valid(a, p, tile);
        const uint32_t st = g_starts(a, p, tile, cur);
        float av[kGT], uv[kGT];
        g_gates<S, SIG>(cur, nv, av, uv);
        g_inputs<S>(cur, nv, uv, uv);
        float2(*s2)[64] = sp[tile & 1];
        s2[p.wave][p.lane] = g_span(av, uv, st);
        __syncthreads();
        float h = carry;
        auto join = [&](auto marks) __attribute__((always_inline)) {
            constexpr bool M = decltype(marks)::value;
#pragma unroll
            for (int w = 0; w < kGW; ++w) {
                if (w == p.wave) h = carry;
                const float2 s = s2[w][p.lane];
                carry = fold<M>(s.x, s.y, carry);
                if (AGG) P = fold_mark<M>(s.x, P);
            }
        };
        if (g_marked<SEQ>(sp[tile & 1], p.lane) || (SEQ && AGG && P < 0.0f)) join(std::true_type{});
        else join(std::false_type{});
        if (!AGG) {
            using T = typename S::T;
            char* y = reinterpret_cast<char*>(static_cast<T*>(a.y) + (p.b * a.L + tile * kGTile + p.wave * kGT) * a.y_row);
            const uint32_t lb = here(static_cast<uint32_t>(p.c) * static_cast<uint32_t>(sizeof(T)));
            auto out = [&](auto plain) __attribute__((always_inline)) {
                constexpr bool PLAIN = decltype(plain)::value;  // all tokens valid, none a start
#pragma unroll
                for (int i = 0; i < kGT; ++i) {
                    h = !PLAIN && (st >> i) & 1 ? uv[i] : av[i] * h + uv[i];
                    if ((PLAIN || i < nv) && p.live) S::store(reinterpret_cast<T*>(y + lb), 0, h);
                    y += a.y_row * sizeof(T);
                }
            };
            if (st == 0 && nv == kGT) out(std::true_type{});
            else out(std::false_type{});
        }
    };
    GRaw<S, false, SEQ> other;
    for (int64_t tile = first; tile < last; tile += 2) {
        step(tile, cur, other);
        if (tile + 1 < last) step(tile + 1, other, cur);
    }
    if (p.wave != 0 || !p.live) return;
    if (AGG) {
        float* o = a.seg + (p.b * a.nseg + seg) * 3 * a.C + p.c;
        o[0] = P;
        o[a.C] = carry;
    } else if (seg == nseg - 1 && a.final_state) {
        a.final_state[p.b * a.C + p.c] = carry;
    }
}

// ---------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------
// Forward walk over a segment: (A, H) from its start to each tile, and with SEG its own
// (A, H, E) for the join.
template <class S, bool SIG, bool SEQ, bool SEG>
__global__ void __launch_bounds__(kGThreads) gscan_bwd_states_kernel(GArgs a) {
    __shared__ float2 sp[2][kGW][64];
    __shared__ float se[2][SEG ? kGW : 1][64];
    const int64_t seg = blockIdx.x % a.nseg;
    const GPos p = g_pos(a, blockIdx.x / a.nseg);
    const int64_t first = seg * a.seg_tiles;
    const int64_t last = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
    GRaw<S, SEG, SEQ> cur;
    g_load(a, p, first, cur);
    float H = 0.0f, P = 1.0f, E = 0.0f;
    auto step = [&](int64_t tile, const GRaw<S, SEG, SEQ>& cur, GRaw<S, SEG, SEQ>& nxt) __attribute__((always_inline)) {
        g_load(a, p, tile + 1 < last ? tile + 1 : tile, nxt);
        if (p.wave == 0 && p.live) {
            float* o = a.ckpt + (p.b * a.tiles + tile) * 2 * a.C + p.c;
            o[0] = P;
            o[a.C] = H;
        }
        const int nv = g_valid(a, p, tile);
        const uint32_t st = g_starts(a, p, tile, cur);
        float av[kGT], uv[kGT];
        g_gates<S, SIG>(cur, nv, av, uv);
        g_inputs<S>(cur, nv, uv, uv);
        float2(*s2)[64] = sp[tile & 1];
        s2[p.wave][p.lane] = g_span(av, uv, st);
        if constexpr (SEG) se[tile & 1][p.wave][p.lane] = g_back<S>(cur, nv, av, st);
        __syncthreads();
        auto join = [&](auto marks) __attribute__((always_inline)) {
            constexpr bool M = decltype(marks)::value;
#pragma unroll
            for (int w = 0; w < kGW; ++w) {
                const float2 s = s2[w][p.lane];
                if constexpr (SEG) E = M && P < 0.0f ? E : P * se[tile & 1][w][p.lane] + E;
                H = fold<M>(s.x, s.y, H);
                P = fold_mark<M>(s.x, P);
            }
        };
        if (g_marked<SEQ>(sp[tile & 1], p.lane) || (SEQ && P < 0.0f)) join(std::true_type{});
        else join(std::false_type{});
    };
    GRaw<S, SEG, SEQ> other;
    for (int64_t tile = first; tile < last; tile += 2) {
        step(tile, cur, other);
        if (tile + 1 < last) step(tile + 1, other, cur);
    }
    if constexpr (SEG) {
        if (p.wave != 0 || !p.live) return;
        float* o = a.seg + (p.b * a.nseg + seg) * 3 * a.C + p.c;
        o[0] = P;
        o[a.C] = H;
        o[2 * a.C] = E;
    }
}

// Backward walk over a segment: gradients of its tokens.
template <class S, bool SIG, bool SEQ>
__global__ void __launch_bounds__(kGThreads) gscan_bwd_kernel(GArgs a) {
    __shared__ float2 sp[2][kGW][64];
    __shared__ float se[2][kGW][64];
    const int64_t seg = blockIdx.x % a.nseg;
    const GPos p = g_pos(a, blockIdx.x / a.nseg);
    const int64_t first = seg * a.seg_tiles;
    const int64_t last = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
    GRaw<S, true, SEQ> cur;
    g_load(a, p, last - 1, cur);
    float hseg = a.h0 ? a.h0[p.b * a.C + p.c] : 0.0f;
    float carry = a.dhT ? a.dhT[p.b * a.C + p.c] : 0.0f;
    if (a.nseg > 1) {
        hseg = fold_segments(a, p, sp[0], 0, 1, seg, 1, hseg);
        carry = fold_segments(a, p, sp[1], a.nseg - 1, -1, a.nseg - 1 - seg, 2, carry);
        __syncthreads();
    }
    using T = typename S::T;
    auto step = [&](int64_t tile, const GRaw<S, true, SEQ>& cur, GRaw<S, true, SEQ>& nxt) __attribute__((always_inline)) {
        const float* ck = a.ckpt + (p.b * a.tiles + tile) * 2 * a.C + p.c;
        const float cA = ck[0], cH = ck[a.C];
        g_load(a, p, tile > first ? tile - 1 : tile, nxt);
        const int nv = g_valid(a, p, tile);
        const uint32_t st = g_starts(a, p, tile, cur);
        float av[kGT], in[kGT], uv[kGT];
        g_gates<S, SIG>(cur, nv, av, in);
        g_inputs<S>(cur, nv, in, uv);
        float2(*s2)[64] = sp[tile & 1];
        float(*s1)[64] = se[tile & 1];
        s2[p.wave][p.lane] = g_span(av, uv, st);
        s1[p.wave][p.lane] = g_back<S>(cur, nv, av, st);
        __syncthreads();
        float h = fold<true>(cA, cH, hseg), E = 0.0f;
        auto join = [&](auto marks) __attribute__((always_inline)) {
            constexpr bool M = decltype(marks)::value;
            // all 16 spans are read at once: a branch around those that do not count would wait
            // for one LDS read after the other
            float A[kGW], t = h;
#pragma unroll
            for (int w = 0; w < kGW; ++w) {
                const float2 s = s2[w][p.lane];
                A[w] = s.x;
                if (w == p.wave) h = t;
                t = fold<M>(s.x, s.y, t);
            }
#pragma unroll
            for (int w = kGW - 1; w >= 0; --w) {
                if (w == p.wave) E = carry;
                carry = fold<M>(A[w], s1[w][p.lane], carry);
            }
        };
        if (g_marked<SEQ>(sp[tile & 1], p.lane)) join(std::true_type{});
        else join(std::false_type{});
        const int64_t t0 = p.b * a.L + tile * kGTile + p.wave * kGT;
        char* dx = reinterpret_cast<char*>(static_cast<T*>(a.dx) + t0 * a.dx_row);
        char* dg = reinterpret_cast<char*>(static_cast<T*>(a.dgate) + t0 * a.dgate_row);
        const uint32_t lb = here(static_cast<uint32_t>(p.c) * static_cast<uint32_t>(sizeof(T)));
        auto out = [&](auto plain) __attribute__((always_inline)) {
            constexpr bool PLAIN = decltype(plain)::value;  // all tokens valid, none a start
            float before[kGT];                              // h_{t-1}, 0 at a start
#pragma unroll
            for (int i = 0; i < kGT; ++i) {
                const bool s = !PLAIN && (st >> i) & 1;
                before[i] = s ? 0.0f : h;
                h = s ? uv[i] : av[i] * h + uv[i];
            }
#pragma unroll
            for (int i = kGT - 1; i >= 0; --i) {
                if (PLAIN || i < nv) {
                    const bool s = !PLAIN && (st >> i) & 1;
                    const float D = S::load(cur.d, i) + E, aD = av[i] * D;
                    float dlog = s ? 0.0f : aD * before[i], dxv = D;
                    if constexpr (SIG) {
                        dxv = D * in[i];
                        dlog = in[i] * dlog - aD * uv[i];
                    }
                    if (p.live) {
                        S::store(reinterpret_cast<T*>(dx + i * a.dx_row * sizeof(T) + lb), 0, dxv);
                        S::store(reinterpret_cast<T*>(dg + i * a.dgate_row * sizeof(T) + lb), 0, dlog);
                    }
                    E = s ? 0.0f : aD;
                }
            }
        };
        if (st == 0 && nv == kGT) out(std::true_type{});
        else out(std::false_type{});
    };
    GRaw<S, true, SEQ> other;
    for (int64_t tile = last - 1; tile >= first; tile -= 2) {
        step(tile, cur, other);
        if (tile > first) step(tile - 1, other, cur);
    }
    if (seg == 0 && p.wave == 0 && p.live && a.dh0) a.dh0[p.b * a.C + p.c] = carry;
}

// ---------------------------------------------------------------------------------------
// decode: the pool row of slot s = slots[b], n_new tokens, V channels a thread
// ---------------------------------------------------------------------------------------
template <class S, bool SIG, int V>
__global__ void __launch_bounds__(256) gscan_step_kernel(GArgs a, float* pool, const int32_t* slots,
                                                         int64_t n_slots) {
    const int64_t per = a.C / V;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= a.B * per) return;
    const int64_t b = e / per, c = (e % per) * V;
    const int64_t slot = slots ? slots[b] : b;
    const bool on = slot >= 0 && slot < n_slots;
    float h[V];
    float* hp = pool + slot * a.C + c;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.0f;
    if (on) {
        if constexpr (V == 4) {
            const float4 q = *reinterpret_cast<const float4*>(hp);
            h[0] = q.x; h[1] = q.y; h[2] = q.z; h[3] = q.w;
        } else {
            h[0] = hp[0];
        }
    }
    using T = typename S::T;
    struct alignas(sizeof(T) * V) Pack { T v[V]; };
    for (int64_t t = 0; t < a.L; ++t) {
        const int64_t r = b * a.L + t;
        const Pack xv = *reinterpret_cast<const Pack*>(static_cast<const T*>(a.x) + r * a.x_row + c);
        const Pack gv = *reinterpret_cast<const Pack*>(static_cast<const T*>(a.gate) + r * a.gate_row + c);
        Pack yv;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float av, in;
            gates<SIG>(S::load(gv.v, v), av, in);
            h[v] = av * h[v] + in * S::load(xv.v, v);
            S::store(yv.v, v, on ? h[v] : 0.0f);
        }
        *reinterpret_cast<Pack*>(static_cast<T*>(a.y) + r * a.y_row + c) = yv;
    }
    if (!on) return;
    if constexpr (V == 4) *reinterpret_cast<float4*>(hp) = make_float4(h[0], h[1], h[2], h[3]);
    else hp[0] = h[0];
}

// Cut along the row: as many segments as bring the grid to kFill blocks, none of fewer than
// kLeast tiles.
constexpr int64_t kFill = 256, kLeast = 4;
void g_cut(GArgs& a) {
    const int64_t blocks = a.B * ((a.C + 63) / 64);
    a.tiles = (a.L + kGTile - 1) / kGTile;
    int64_t want = (kFill + blocks - 1) / blocks;
    const int64_t most = a.tiles / kLeast > 1 ? a.tiles / kLeast : 1;
    if (want > most) want = most;
    a.seg_tiles = (a.tiles + want - 1) / want;
    a.nseg = (a.tiles + a.seg_tiles - 1) / a.seg_tiles;
}

GArgs g_args(const GscanCall& c) {
    GArgs a{};
    a.x = c.x; a.gate = c.gate; a.dy = c.dy; a.y = c.y; a.dx = c.dx; a.dgate = c.dgate;
    a.x_row = c.x_row; a.gate_row = c.gate_row; a.dy_row = c.dy_row; a.y_row = c.y_row;
    a.dx_row = c.dx_row; a.dgate_row = c.dgate_row;
    a.h0 = c.h0; a.dhT = c.dhT; a.final_state = c.final_state; a.dh0 = c.dh0; a.seq = c.seq;
    a.B = c.B; a.L = c.L; a.C = c.C;
    return a;
}

template <class S, bool SIG, bool SEQ>
hipError_t fwd_typed(const GArgs& a, hipStream_t s) {
    const int64_t groups = a.B * ((a.C + 63) / 64);
    if (a.nseg > 1) {
        gscan_fwd_kernel<S, SIG, SEQ, true><<<static_cast<uint32_t>(groups * (a.nseg - 1)), kGThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    gscan_fwd_kernel<S, SIG, SEQ, false><<<static_cast<uint32_t>(groups * a.nseg), kGThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <class S, bool SIG, bool SEQ>
hipError_t bwd_typed(const GArgs& a, hipStream_t s) {
    const uint32_t grid = static_cast<uint32_t>(a.B * ((a.C + 63) / 64) * a.nseg);
    if (a.nseg > 1) gscan_bwd_states_kernel<S, SIG, SEQ, true><<<grid, kGThreads, 0, s>>>(a);
    else gscan_bwd_states_kernel<S, SIG, SEQ, false><<<grid, kGThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    gscan_bwd_kernel<S, SIG, SEQ><<<grid, kGThreads, 0, s>>>(a);
    return hipGetLastError();
}
// one call of f with the kernels' template arguments as values: f(storage, sigmoid form, packed)
template <class F>
hipError_t g_dispatch(const GscanCall& c, F f) {
    auto with = [&](auto storage, auto sig) {
        return c.seq ? f(storage, sig, std::true_type{}) : f(storage, sig, std::false_type{});
    };
    if (c.dtype == SSM_BF16) return c.sigmoid ? with(BF16{}, std::true_type{}) : with(BF16{}, std::false_type{});
    return c.sigmoid ? with(F32{}, std::true_type{}) : with(F32{}, std::false_type{});
}
template <class S, bool SIG>
hipError_t step_typed(const GArgs& a, float* pool, const int32_t* slots, int64_t n_slots, bool vec,
                      hipStream_t s) {
    const uint32_t grid = static_cast<uint32_t>((a.B * (a.C / (vec ? 4 : 1)) + 255) / 256);
    if (vec) gscan_step_kernel<S, SIG, 4><<<grid, 256, 0, s>>>(a, pool, slots, n_slots);
    else gscan_step_kernel<S, SIG, 1><<<grid, 256, 0, s>>>(a, pool, slots, n_slots);
    return hipGetLastError();
}

}  // namespace

int64_t gscan_blocks(int64_t B, int64_t L, int64_t C) {
    GArgs a{};
    a.B = B; a.L = L; a.C = C;
    g_cut(a);
    return B * ((C + 63) / 64) * a.nseg;
}

size_t gscan_workspace_bytes(int64_t B, int64_t L, int64_t C, bool bwd) {
    GArgs a{};
    a.B = B; a.L = L; a.C = C;
    g_cut(a);
    const int64_t seg = a.nseg > 1 ? B * a.nseg * 3 * C : 0;
    return static_cast<size_t>(seg + (bwd ? B * a.tiles * 2 * C : 0)) * 4;
}

hipError_t launch_gscan_fwd(const GscanCall& c, hipStream_t s) {
    GArgs a = g_args(c);
    g_cut(a);
    a.seg = static_cast<float*>(c.workspace);
    return g_dispatch(c, [&](auto S, auto sig, auto seq) {
        return fwd_typed<decltype(S), decltype(sig)::value, decltype(seq)::value>(a, s);
    });
}

hipError_t launch_gscan_bwd(const GscanCall& c, hipStream_t s) {
    GArgs a = g_args(c);
    g_cut(a);
    a.ckpt = static_cast<float*>(c.workspace);
    a.seg = a.ckpt + a.B * a.tiles * 2 * a.C;
    return g_dispatch(c, [&](auto S, auto sig, auto seq) {
        return bwd_typed<decltype(S), decltype(sig)::value, decltype(seq)::value>(a, s);
    });
}

hipError_t launch_gscan_step(const GscanCall& c, float* pool, const int32_t* slots, int64_t n_slots,
                             hipStream_t s) {
    const GArgs a = g_args(c);
    const uintptr_t es = c.dtype == SSM_BF16 ? 2 : 4;
    // four channels a thread where every row starts on four elements' alignment
    auto four = [&](const void* p, int64_t row) {
        return reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && row % 4 == 0;
    };
    const bool vec = a.C % 4 == 0 && reinterpret_cast<uintptr_t>(pool) % 16 == 0 &&
                     four(c.x, c.x_row) && four(c.gate, c.gate_row) && four(c.y, c.y_row);
    if (c.dtype == SSM_BF16)
        return c.sigmoid ? step_typed<BF16, true>(a, pool, slots, n_slots, vec, s)
                         : step_typed<BF16, false>(a, pool, slots, n_slots, vec, s);
    return c.sigmoid ? step_typed<F32, true>(a, pool, slots, n_slots, vec, s)
                     : step_typed<F32, false>(a, pool, slots, n_slots, vec, s);
}

}  // namespace ssm
