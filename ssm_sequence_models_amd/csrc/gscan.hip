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
// decays, H its own tokens' share).  A block takes 64 channels of one row and walks over tiles
// of 128 tokens, 8 wavefronts of 16 tokens each; a lane has two channels of half the tokens, so
// that a load or store moves a pair.  Every wavefront forms its (A, H), and (A, E) backward,
// from registers (the halves against each other with the half-swap of lanes, one channel a
// lane), the 8 spans are joined through LDS, and a second walk over the registers applies the
// state that comes in.  So a tile is read once.
//
// The next tile's loads are issued before the current one is worked on, and its stores are not
// waited for.  That holds as long as the loop has one path: where loads or stores were under a
// branch (a row's last tile, lanes past the last channel), the waits behind it were those of
// the path with the fewest, and 16-bit loads kept the load return path busy for 82 % of the
// time.  So tiles that end within the row have a loop of their own, and lanes past the last
// channel repeat the last pair.  4 x 8192 tokens x 4096 channels, bf16, sigmoid form, packed:
// forward 173 us (0.80 GB, 4.7 TB/s; one channel a lane 200; 16 wavefronts of 8 tokens, which
// join twice the spans, 221), backward 149 + 269 us (0.56 + 1.36 GB; one channel a lane
// 161 + 326).  The instructions bound it as much: nine a token and channel for the gates alone,
// two of them at a quarter of the rate.
//
// Rows and channels too few to fill the GPU (under kFill blocks) are cut into segments of
// tiles: a first kernel joins each segment to one (A, H), which reads the inputs once more,
// and each block of the second folds the segments before (and behind) its own.  One row of
// 65573 tokens x 333 channels, fp32, log form: 37 + 71 us.
// The backward needs h before each tile: its first kernel walks forward and stores (A, H) from
// the segment's start to each tile's (8 bytes a channel and 128 tokens).
//
// A is a product of decays, so it must not leave fp32's range: gates of the log form above 0 are
// served as long as e^(their sum) over consecutive tokens is finite (times a state of 0, infinity
// would be NaN).
//
// A span that holds a sequence start passes nothing on; it is marked by A = -1 (a product of
// decays is never negative) and folded by a select, so a NaN or infinity of one sequence does
// not reach the next.  Everything is fp32; outputs are rounded once.
#include <type_traits>

#include "gscan_groups.h"
#include "internal.h"

namespace ssm {
namespace {

constexpr bool g_splits_sound() {
    for (int64_t C = 1; C <= 300; ++C)
        if (!g_split_sound(C)) return false;
    return true;
}
static_assert(g_splits_sound(), "a channel in two blocks");

constexpr int kGW = 8;              // wavefronts a block
constexpr int kGL = 8;              // tokens a lane and tile
constexpr int kGT = 2 * kGL;        // tokens a wavefront and tile
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
    bool pairs;   // two channels and the lanes' 32-bit offsets serve whole tiles
};

// decay a and input factor i of a gate: e = exp(-g), a = 1 / (1 + e) and i = e a, neither a
// difference, are within (6 + 1.3 |g|) 2^-24 of themselves (the exponent's rounding in e; one step
// each of exp2 and rcp); e is held below 2^126, where 1 / (1 + e) is still a normal number
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

// two consecutive channels of a token, at any element's alignment
template <class S>
struct Two;
template <>
struct Two<BF16> {
    typedef uint32_t R;
    typedef uint32_t M __attribute__((aligned(2)));
    __device__ __forceinline__ static float get(R r, int k) { return __uint_as_float(k ? r & 0xFFFF0000u : r << 16); }
    __device__ __forceinline__ static R of(uint16_t lo, uint16_t hi) { return lo | static_cast<uint32_t>(hi) << 16; }
    __device__ __forceinline__ static R round(float lo, float hi) { return pack_bf16x2(lo, hi); }
};
template <>
struct Two<F32> {
    typedef float R __attribute__((ext_vector_type(2)));
    typedef float M __attribute__((ext_vector_type(2), aligned(4)));
    __device__ __forceinline__ static float get(R r, int k) { return r[k]; }
    __device__ __forceinline__ static R of(float lo, float hi) { return R{lo, hi}; }
    __device__ __forceinline__ static R round(float lo, float hi) { return R{lo, hi}; }
};

// a lane's tokens of one tile, as loaded.  SEQ: the rows are packed
template <class S, bool DY, bool SEQ>
struct GRaw {
    static constexpr bool kSeq = SEQ;
    typename Two<S>::R x[kGL], g[kGL], d[DY ? kGL : 1];
    int32_t id;  // lane j: sequence id of the token before the wavefront's token j
};

// A lane's place: channels c0, c0 + 1 of the tokens 8 half .. 8 half + 7 of a wavefront's 16, and
// one channel, c, of all that is joined over spans.  Past the group's last pair lanes take its last
// two channels once more (of one channel, that one twice): the same values to the same places, by
// the same block (gscan_groups.h).
struct GPos {
    int64_t b, c, c0;
    int lane, wave, half;
    bool live;  // no other lane has channel c
};

// A 32-bit lane offset that stays one: added to a uniform base it is part of the access (left to
// itself the compiler widens it once and adds 64 bits for every token)
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}
// byte offset of a lane's first token and channel from the wavefront's first token
template <class S>
__device__ __forceinline__ uint32_t g_offset(const GPos& p, int64_t row) {
    using T = typename S::T;
    return (static_cast<uint32_t>(p.half * kGL) * static_cast<uint32_t>(row) + static_cast<uint32_t>(p.c0)) * sizeof(T);
}

template <class S>
__device__ __forceinline__ void g_rows(const void* base, int64_t token, int64_t row, uint32_t off, typename Two<S>::R (&v)[kGL]) {
    const char* q = reinterpret_cast<const char*>(static_cast<const typename S::T*>(base) + token * row);
    off = here(off);
#pragma unroll
    for (int i = 0; i < kGL; ++i) {
        v[i] = *reinterpret_cast<const typename Two<S>::M*>(q + off);
        q += row * sizeof(typename S::T);
    }
}
// The same element by element, tokens past the row's end replaced by its last (read and not
// used): the last tile of a row, one channel, or rows too far apart
template <class S>
__device__ __forceinline__ void g_rows_any(const GArgs& a, const GPos& p, const void* base, int64_t t0, int64_t row,
                                           typename Two<S>::R (&v)[kGL]) {
    using T = typename S::T;
    const int64_t second = p.c0 + 1 < a.C ? 1 : 0;
    int64_t t = t0 + here(p.half * kGL);
    if (t >= a.L) t = a.L - 1;
    const T* q = static_cast<const T*>(base) + (p.b * a.L + t) * row + p.c0;
#pragma unroll
    for (int i = 0; i < kGL; ++i) {
        v[i] = Two<S>::of(q[0], q[second]);
        if (t + 1 < a.L) {
            ++t;
            q += row;
        }
    }
}

// FULL: the tile ends within the row, and pairs serve it
template <bool FULL, class S, bool DY, bool SEQ>
__device__ __forceinline__ void g_load(const GArgs& a, const GPos& p, int64_t tile, GRaw<S, DY, SEQ>& r) {
    const int64_t t0 = tile * kGTile + p.wave * kGT, row0 = p.b * a.L;
    // in the order of their use: a wait for one load is a wait for those before it
    if constexpr (SEQ) {
        int64_t t = t0 - 1 + p.lane;
        t = t < 0 ? 0 : t < a.L ? t : a.L - 1;
        r.id = a.seq[row0 + t];
    }
    if constexpr (FULL) {
        g_rows<S>(a.gate, row0 + t0, a.gate_row, g_offset<S>(p, a.gate_row), r.g);
        g_rows<S>(a.x, row0 + t0, a.x_row, g_offset<S>(p, a.x_row), r.x);
        if constexpr (DY) g_rows<S>(a.dy, row0 + t0, a.dy_row, g_offset<S>(p, a.dy_row), r.d);
    } else {
        g_rows_any<S>(a, p, a.gate, t0, a.gate_row, r.g);
        g_rows_any<S>(a, p, a.x, t0, a.x_row, r.x);
        if constexpr (DY) g_rows_any<S>(a, p, a.dy, t0, a.dy_row, r.d);
    }
}

// the first tile that g_load<true> does not serve, from `first` on
__device__ __forceinline__ int64_t g_full(const GArgs& a, int64_t first, int64_t last) {
    const int64_t n = a.pairs ? a.L / kGTile : 0;
    return n < first ? first : n < last ? n : last;
}

// bit i: the wavefront's token i starts a sequence (token 0 of the row never does)
template <class R>
__device__ __forceinline__ uint32_t g_starts(const GArgs& a, const GPos& p, int64_t tile, const R& r) {
    if constexpr (!R::kSeq) return 0;
    const int64_t t = tile * kGTile + p.wave * kGT - 1 + p.lane;
    const int32_t before = __shfl_up(r.id, 1);
    const uint64_t m = __ballot(p.lane >= 1 && p.lane <= kGT && t > 0 && t < a.L && r.id != before);
    return static_cast<uint32_t>(m >> 1);
}

// tokens of the wavefront that the row has
__device__ __forceinline__ int g_valid(const GArgs& a, const GPos& p, int64_t tile) {
    const int64_t n = a.L - (tile * kGTile + p.wave * kGT);
    return n < 0 ? 0 : n < kGT ? static_cast<int>(n) : kGT;
}

__device__ __forceinline__ GPos g_pos(const GArgs& a, int64_t row_group) {
    GPos p;
    p.lane = threadIdx.x & 63;
    p.half = p.lane >> 5;
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t groups = g_groups(a.C);
    p.b = row_group / groups;
    const GChannels g = g_channels(a.C, row_group % groups);
    const int64_t c = g.first + 2 * (p.lane & 31);
    p.live = c + 1 < g.end || (c + 1 == g.end && p.half == 1);
    p.c0 = g_pair(g, p.lane & 31);
    p.c = a.C > 1 ? p.c0 + p.half : 0;
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

// The lane's tokens of a tile: st, nv of its half of the wavefront's 16
template <class S>
struct GTile {
    float av[kGL][2], in[kGL][2], uv[kGL][2];  // decays, input factors, inputs: past the end 1, 0, 0
    uint32_t st;
    int nv;
    bool plain;  // all 16 tokens valid, none a start (uniform)
};
template <bool FULL, class S, bool SIG, class R>
__device__ __forceinline__ void g_terms(const GArgs& a, const GPos& p, int64_t tile, const R& r, GTile<S>& q) {
    const uint32_t st = g_starts(a, p, tile, r);
    const int nv = FULL ? kGT : g_valid(a, p, tile);
    q.plain = st == 0 && nv == kGT;
    q.st = st >> (kGL * p.half) & ((1u << kGL) - 1);
    q.nv = nv - kGL * p.half;
#pragma unroll
    for (int i = 0; i < kGL; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            gates<SIG>(Two<S>::get(r.g[i], k), q.av[i][k], q.in[i][k]);
            q.uv[i][k] = q.in[i][k] * Two<S>::get(r.x[i], k);
        }
    if (!FULL && nv < kGT) {
#pragma unroll
        for (int i = 0; i < kGL; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                q.av[i][k] = i < q.nv ? q.av[i][k] : 1.0f;
                q.in[i][k] = i < q.nv ? q.in[i][k] : 0.0f;
                q.uv[i][k] = i < q.nv ? q.uv[i][k] : 0.0f;
            }
    }
}

// Two channels of one half of the tokens against one channel of both halves: of a lane's values
// v0, v1 of its two channels, the lower half of the wavefront takes the first channel's of both
// halves, the upper the second's; the same step leads back.
__device__ __forceinline__ void g_swap(float& v0, float& v1) {
    const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v0), __float_as_uint(v1), false, false);
    v0 = __uint_as_float(w[0]);
    v1 = __uint_as_float(w[1]);
}

// (A, H) of the two halves of the wavefront's tokens, of the lane's one channel
template <class S>
__device__ __forceinline__ void g_spans(const GTile<S>& q, float (&A)[2], float (&H)[2]) {
    if (q.plain) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            A[k] = q.av[0][k];
            H[k] = q.uv[0][k];
#pragma unroll
            for (int i = 1; i < kGL; ++i) {
                H[k] = q.av[i][k] * H[k] + q.uv[i][k];
                A[k] *= q.av[i][k];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            A[k] = 1.0f;
            H[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < kGL; ++i) {
                H[k] = (q.st >> i) & 1 ? q.uv[i][k] : q.av[i][k] * H[k] + q.uv[i][k];
                A[k] *= q.av[i][k];
            }
            if (q.st) A[k] = -1.0f;
        }
    }
    g_swap(A[0], A[1]);
    g_swap(H[0], H[1]);
}

// E that the two halves hand to the token before them, with E = 0 behind them
template <class S, class R>
__device__ __forceinline__ void g_backs(const R& r, const GTile<S>& q, float (&E)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float e = 0.0f;
        if (q.plain) {
#pragma unroll
            for (int i = kGL - 1; i >= 0; --i) e = q.av[i][k] * (Two<S>::get(r.d[i], k) + e);
        } else {
#pragma unroll
            for (int i = kGL - 1; i >= 0; --i) {
                const float d = (i < q.nv ? Two<S>::get(r.d[i], k) : 0.0f) + e;
                e = (q.st >> i) & 1 ? 0.0f : q.av[i][k] * d;
            }
        }
        E[k] = e;
    }
    g_swap(E[0], E[1]);
}

// the wavefront's (A, H) from its halves'
template <bool SEQ>
__device__ __forceinline__ float2 g_wave(const float (&A)[2], const float (&H)[2]) {
    return make_float2(fold_mark<SEQ>(A[1], A[0]), fold<SEQ>(A[1], H[1], H[0]));
}

// stores the lane's tokens; FULL as for the loads
template <bool FULL, class S>
__device__ __forceinline__ void g_put(const GArgs& a, const GPos& p, void* base, int64_t tile, int64_t row, int nv,
                                      const float (&v)[kGL][2]) {
    using T = typename S::T;
    const int64_t t0 = p.b * a.L + tile * kGTile + p.wave * kGT;
    if constexpr (FULL) {
        char* q = reinterpret_cast<char*>(static_cast<T*>(base) + t0 * row);
        const uint32_t off = here(g_offset<S>(p, row));
#pragma unroll
        for (int i = 0; i < kGL; ++i, q += row * sizeof(T))
            *reinterpret_cast<typename Two<S>::M*>(q + off) = Two<S>::round(v[i][0], v[i][1]);
    } else {
        T* q = static_cast<T*>(base) + (t0 + here(p.half * kGL)) * row + p.c0;
#pragma unroll
        for (int i = 0; i < kGL; ++i, q += row)
            if (i < nv) {
                S::store(q, 0, v[i][0]);
                if (p.c0 + 1 < a.C) S::store(q, 1, v[i][1]);
            }
    }
}

// whether any span of the tile is marked (uniform); A as stored by the wavefronts
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
    const int64_t full = g_full(a, first, last);
    GRaw<S, false, SEQ> cur, other;
    if (full > first) g_load<true>(a, p, first, cur);
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
        // wavefront 0 stores the final state, which may lie in the same place; no other block reads
        // these channels' state (cut rows take it from the workspace)
        asm volatile("" : "+v"(carry));
    }
    auto step = [&](int64_t tile, const GRaw<S, false, SEQ>& cur, auto whole) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(whole)::value;
        GTile<S> q;
        g_terms<FULL, S, SIG>(a, p, tile, cur, q);
        float A[2], H[2];
        g_spans(q, A, H);
        float2(*s2)[64] = sp[tile & 1];
        s2[p.wave][p.lane] = g_wave<SEQ>(A, H);
        __syncthreads();
        float h[2] = {carry, carry};  // before each half
        auto join = [&](auto marks) __attribute__((always_inline)) {
            constexpr bool M = decltype(marks)::value;
#pragma unroll
            for (int w = 0; w < kGW; ++w) {
                if (w == p.wave) h[0] = carry;
                const float2 s = s2[w][p.lane];
                carry = fold<M>(s.x, s.y, carry);
                if (AGG) P = fold_mark<M>(s.x, P);
            }
            h[1] = fold<M>(A[0], H[0], h[0]);
        };
        if (g_marked<SEQ>(sp[tile & 1], p.lane) || (SEQ && AGG && P < 0.0f)) join(std::true_type{});
        else join(std::false_type{});
        if constexpr (!AGG) {
            g_swap(h[0], h[1]);
            float hv[kGL][2];
            if (q.plain) {
#pragma unroll
                for (int i = 0; i < kGL; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) hv[i][k] = h[k] = q.av[i][k] * h[k] + q.uv[i][k];
            } else {
#pragma unroll
                for (int i = 0; i < kGL; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        hv[i][k] = h[k] = (q.st >> i) & 1 ? q.uv[i][k] : q.av[i][k] * h[k] + q.uv[i][k];
            }
            g_put<FULL, S>(a, p, a.y, tile, a.y_row, q.nv, hv);
        }
    };
    for (int64_t tile = first; tile < full; tile += 2) {
        g_load<true>(a, p, tile + 1 < full ? tile + 1 : tile, other);
        step(tile, cur, std::true_type{});
        if (tile + 1 == full) break;
        g_load<true>(a, p, tile + 2 < full ? tile + 2 : tile + 1, cur);
        step(tile + 1, other, std::true_type{});
    }
    for (int64_t tile = full; tile < last; ++tile) {
        g_load<false>(a, p, tile, cur);
        step(tile, cur, std::false_type{});
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
    const int64_t full = g_full(a, first, last);
    GRaw<S, SEG, SEQ> cur, other;
    if (full > first) g_load<true>(a, p, first, cur);
    float H = 0.0f, P = 1.0f, E = 0.0f;
    auto step = [&](int64_t tile, const GRaw<S, SEG, SEQ>& cur, auto whole) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(whole)::value;
        GTile<S> q;
        g_terms<FULL, S, SIG>(a, p, tile, cur, q);
        if (p.wave == 0 && p.live) {
            float* o = a.ckpt + (p.b * a.tiles + tile) * 2 * a.C + p.c;
            o[0] = P;
            o[a.C] = H;
        }
        float As[2], Hs[2];
        g_spans(q, As, Hs);
        float2(*s2)[64] = sp[tile & 1];
        s2[p.wave][p.lane] = g_wave<SEQ>(As, Hs);
        if constexpr (SEG) {
            float Es[2];
            g_backs<S>(cur, q, Es);
            se[tile & 1][p.wave][p.lane] = fold<SEQ>(As[0], Es[0], Es[1]);
        }
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
    for (int64_t tile = first; tile < full; tile += 2) {
        g_load<true>(a, p, tile + 1 < full ? tile + 1 : tile, other);
        step(tile, cur, std::true_type{});
        if (tile + 1 == full) break;
        g_load<true>(a, p, tile + 2 < full ? tile + 2 : tile + 1, cur);
        step(tile + 1, other, std::true_type{});
    }
    for (int64_t tile = full; tile < last; ++tile) {
        g_load<false>(a, p, tile, cur);
        step(tile, cur, std::false_type{});
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
    const int64_t full = g_full(a, first, last);
    GRaw<S, true, SEQ> cur, other;
    if (full > first && full == last) g_load<true>(a, p, full - 1, cur);
    float hseg = a.h0 ? a.h0[p.b * a.C + p.c] : 0.0f;
    float carry = a.dhT ? a.dhT[p.b * a.C + p.c] : 0.0f;
    if (a.nseg > 1) {
        hseg = fold_segments(a, p, sp[0], 0, 1, seg, 1, hseg);
        carry = fold_segments(a, p, sp[1], a.nseg - 1, -1, a.nseg - 1 - seg, 2, carry);
        __syncthreads();
    }
    // (A, H) of the segment's tokens before the tile
    auto before_tile = [&](int64_t tile) __attribute__((always_inline)) {
        const float* ck = a.ckpt + (p.b * a.tiles + tile) * 2 * a.C + p.c;
        return make_float2(ck[0], ck[a.C]);
    };
    auto step = [&](int64_t tile, const GRaw<S, true, SEQ>& cur, float2 ck, auto whole) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(whole)::value;
        GTile<S> q;
        g_terms<FULL, S, SIG>(a, p, tile, cur, q);
        float As[2], Hs[2], Es[2];
        g_spans(q, As, Hs);
        g_backs<S>(cur, q, Es);
        float2(*s2)[64] = sp[tile & 1];
        float(*s1)[64] = se[tile & 1];
        s2[p.wave][p.lane] = g_wave<SEQ>(As, Hs);
        s1[p.wave][p.lane] = fold<SEQ>(As[0], Es[0], Es[1]);
        __syncthreads();
        float h[2] = {fold<true>(ck.x, ck.y, hseg), 0.0f}, E[2];  // before and behind each half
        auto join = [&](auto marks) __attribute__((always_inline)) {
            constexpr bool M = decltype(marks)::value;
            // all spans are read at once: a branch around those that do not count would wait for
            // one LDS read after the other
            float A[kGW], t = h[0];
#pragma unroll
            for (int w = 0; w < kGW; ++w) {
                const float2 s = s2[w][p.lane];
                A[w] = s.x;
                if (w == p.wave) h[0] = t;
                t = fold<M>(s.x, s.y, t);
            }
            E[1] = carry;
#pragma unroll
            for (int w = kGW - 1; w >= 0; --w) {
                if (w == p.wave) E[1] = carry;
                carry = fold<M>(A[w], s1[w][p.lane], carry);
            }
            h[1] = fold<M>(As[0], Hs[0], h[0]);
            E[0] = fold<M>(As[1], Es[1], E[1]);
        };
        if (g_marked<SEQ>(sp[tile & 1], p.lane)) join(std::true_type{});
        else join(std::false_type{});
        g_swap(h[0], h[1]);
        g_swap(E[0], E[1]);
        float dx[kGL][2], dg[kGL][2];
        auto grads = [&](auto starts) __attribute__((always_inline)) {
            constexpr bool ST = decltype(starts)::value;
            float before[kGL][2];  // h_{t-1}, not used at a start
#pragma unroll
            for (int i = 0; i < kGL; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    before[i][k] = h[k];
                    h[k] = ST && (q.st >> i) & 1 ? q.uv[i][k] : q.av[i][k] * h[k] + q.uv[i][k];
                }
#pragma unroll
            for (int i = kGL - 1; i >= 0; --i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool start = ST && (q.st >> i) & 1, off = !FULL && i >= q.nv;
                    const float D = (off ? 0.0f : Two<S>::get(cur.d[i], k)) + E[k], aD = q.av[i][k] * D;
                    dx[i][k] = D;
                    dg[i][k] = start ? 0.0f : aD * before[i][k];
                    if constexpr (SIG) {
                        dx[i][k] = D * q.in[i][k];
                        dg[i][k] = q.in[i][k] * dg[i][k] - aD * q.uv[i][k];
                    }
                    E[k] = start ? 0.0f : aD;
                }
        };
        if (SEQ && !q.plain) grads(std::true_type{});
        else grads(std::false_type{});
        g_put<FULL, S>(a, p, a.dx, tile, a.dx_row, q.nv, dx);
        g_put<FULL, S>(a, p, a.dgate, tile, a.dgate_row, q.nv, dg);
    };
    for (int64_t tile = last - 1; tile >= full; --tile) {
        g_load<false>(a, p, tile, cur);
        step(tile, cur, before_tile(tile), std::false_type{});
    }
    if (full > first && full < last) g_load<true>(a, p, full - 1, cur);
    for (int64_t tile = full - 1; tile >= first; tile -= 2) {
        float2 ck = before_tile(tile);
        g_load<true>(a, p, tile > first ? tile - 1 : tile, other);
        step(tile, cur, ck, std::true_type{});
        if (tile == first) break;
        ck = before_tile(tile - 1);
        g_load<true>(a, p, tile - 1 > first ? tile - 2 : tile - 1, cur);
        step(tile - 1, other, ck, std::true_type{});
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
// kLeast tiles.  The forward's first kernel reads everything once more, so it is cut only where
// fewer than kFill / 2 blocks would run, and on more than kWhole tiles; the backward needs two
// walks in any case.  bf16, sigmoid form, forward / backward in us, cut to 256 blocks against
// other numbers:
//   1 x 8192 x 4096   53 / 98     to 128 blocks: 80 / 138
//   2 x 8192 x 4096  115 / 220    left at 128 blocks: 110 / 278
//   8 x 2048 x 1024   29 / 47     left at 128 blocks: 23 / 60
//   4 x 8192 x 4096  171 / 398    (256 blocks as it is) cut to 512: 237 / 473
//   1 x 4096 x 1024   19 / 24     segments of 8 tiles: 25 / 37
//   1 x 1024 x 1024   20 / 22     one segment of 8 tiles: 15 / 31
constexpr int64_t kFill = 256, kLeast = 4, kWhole = 8;
void g_cut(GArgs& a, bool bwd) {
    const int64_t blocks = a.B * g_groups(a.C);
    a.tiles = (a.L + kGTile - 1) / kGTile;
    int64_t want = (kFill + blocks - 1) / blocks;
    if (!bwd && (2 * blocks >= kFill || a.tiles <= kWhole)) want = 1;
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
    // a lane's tokens start up to 8 rows behind the wavefront's first: 2^31 bytes of 4-byte
    // elements at 2^26 a row
    a.pairs = c.C > 1;
    for (const int64_t row : {a.x_row, a.gate_row, a.dy_row, a.y_row, a.dx_row, a.dgate_row})
        if (row >= int64_t{1} << 26) a.pairs = false;
    return a;
}

template <class S, bool SIG, bool SEQ>
hipError_t fwd_typed(const GArgs& a, hipStream_t s) {
    const int64_t groups = a.B * g_groups(a.C);
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
    const uint32_t grid = static_cast<uint32_t>(a.B * g_groups(a.C) * a.nseg);
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
    g_cut(a, true);  // the forward has at most as many segments
    return B * g_groups(C) * a.nseg;
}

size_t gscan_workspace_bytes(int64_t B, int64_t L, int64_t C, bool bwd) {
    GArgs a{};
    a.B = B; a.L = L; a.C = C;
    g_cut(a, bwd);
    const int64_t seg = a.nseg > 1 ? B * a.nseg * 3 * C : 0;
    return static_cast<size_t>(seg + (bwd ? B * a.tiles * 2 * C : 0)) * 4;
}

hipError_t launch_gscan_fwd(const GscanCall& c, hipStream_t s) {
    GArgs a = g_args(c);
    g_cut(a, false);
    a.seg = static_cast<float*>(c.workspace);
    return g_dispatch(c, [&](auto S, auto sig, auto seq) {
        return fwd_typed<decltype(S), decltype(sig)::value, decltype(seq)::value>(a, s);
    });
}

hipError_t launch_gscan_bwd(const GscanCall& c, hipStream_t s) {
    GArgs a = g_args(c);
    g_cut(a, true);
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
