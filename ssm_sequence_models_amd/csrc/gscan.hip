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
// walks over tiles of 128 tokens, 16 wavefronts of 8 tokens each: every wavefront forms its
// (A, H), and (A, E) backward, from registers, the 16 spans are joined through LDS, and a
// second walk over the registers applies the state that comes in.  So a tile is read once.
// The next tile's loads are issued before the current one is worked on.
//
// Rows and channels too few to fill the GPU (under kFill blocks) are cut into segments of
// tiles: a first kernel joins each segment to one (A, H), which reads the inputs once more,
// and each block of the second folds the segments before (and behind) its own.
// The backward needs h before each tile: its first kernel walks forward and stores (A, H) from
// the segment's start to each tile's (8 bytes a channel and 128 tokens).
//
// A span that holds a sequence start passes nothing on; it is marked by A = -1 (a product of
// decays is never negative) and folded by a select, so a NaN or infinity of one sequence does
// not reach the next.  Everything is fp32; outputs are rounded once.
#include "internal.h"

namespace ssm {
namespace {

constexpr int kGW = 16;             // wavefronts a block
constexpr int kGT = 8;              // tokens a wavefront and tile
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

// decay a and input factor i of a gate
template <bool SIG>
__device__ __forceinline__ void gates(float g, float& a, float& i) {
    if constexpr (SIG) {
        // e = exp(-|g|) keeps both a and i = 1 - a to full relative accuracy
        const float e = __expf(-fabsf(g));
        const float r = __builtin_amdgcn_rcpf(1.0f + e), p = e * r;
        a = g >= 0.0f ? r : p;
        i = g >= 0.0f ? p : r;
        if (g != g) a = i = g;
    } else {
        a = __expf(g);
        i = 1.0f;
    }
}

__device__ __forceinline__ float fold(float A, float H, float h) { return A < 0.0f ? H : A * h + H; }
__device__ __forceinline__ float fold_mark(float A, float P) { return P < 0.0f || A < 0.0f ? -1.0f : P * A; }

// a wavefront's tokens of one tile, as loaded; token i is row tok0 + i of the row b
template <class S, bool DY>
struct GRaw {
    typename S::T x[kGT], g[kGT], d[DY ? kGT : 1];
    int32_t id;  // lane j: sequence id of token tok0 - 1 + j
};

struct GPos {
    int64_t b, c;
    int lane, wave;
    bool live;  // the lane's channel exists
};

template <class S, bool DY, bool X = true>
__device__ __forceinline__ void g_load(const GArgs& a, const GPos& p, int64_t tile, GRaw<S, DY>& r) {
    const int64_t t0 = tile * kGTile + p.wave * kGT;
    const int64_t row0 = p.b * a.L;
    using T = typename S::T;
#pragma unroll
    for (int i = 0; i < kGT; ++i) {
        const int64_t t = row0 + (t0 + i < a.L ? t0 + i : a.L - 1);  // past the end: read and not used
        if constexpr (X) r.x[i] = __builtin_nontemporal_load(static_cast<const T*>(a.x) + t * a.x_row + p.c);
        r.g[i] = __builtin_nontemporal_load(static_cast<const T*>(a.gate) + t * a.gate_row + p.c);
        if constexpr (DY) r.d[i] = __builtin_nontemporal_load(static_cast<const T*>(a.dy) + t * a.dy_row + p.c);
    }
    r.id = 0;
    if (a.seq) {
        int64_t t = t0 - 1 + p.lane;
        t = t < 0 ? 0 : t < a.L ? t : a.L - 1;
        r.id = a.seq[row0 + t];
    }
}

// bit i: token i starts a sequence (token 0 of the row never does)
template <class R>
__device__ __forceinline__ uint32_t g_starts(const GArgs& a, const GPos& p, int64_t tile, const R& r) {
    if (!a.seq) return 0;
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

// decays and inputs of the tile's tokens in this wavefront: past the row's end a = 1, u = 0
template <class S, bool SIG, class R>
__device__ __forceinline__ void g_terms(const R& r, int nv, float (&av)[kGT], float (&uv)[kGT]) {
#pragma unroll
    for (int i = 0; i < kGT; ++i) {
        float in;
        gates<SIG>(S::load(r.g, i), av[i], in);
        uv[i] = in * S::load(r.x, i);
        if (i >= nv) {
            av[i] = 1.0f;
            uv[i] = 0.0f;
        }
    }
}

// (A, H) of the wavefront's tokens
__device__ __forceinline__ void g_span(const float (&av)[kGT], const float (&uv)[kGT], uint32_t st,
                                       float& A, float& H) {
    A = 1.0f;
    H = 0.0f;
#pragma unroll
    for (int i = 0; i < kGT; ++i) {
        H = (st >> i) & 1 ? uv[i] : av[i] * H + uv[i];
        A *= av[i];
    }
    if (st) A = -1.0f;
}

// ---------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------
// AGG: only the segment's (A, H), for the join (nseg > 1); else y and the final state.
template <class S, bool SIG, bool AGG>
__global__ void __launch_bounds__(kGThreads) gscan_fwd_kernel(GArgs a) {
    __shared__ float sp[2][kGW][2][64];
    const int64_t nseg = AGG ? a.nseg - 1 : a.nseg;  // the last segment's (A, H) is not needed
    const int64_t seg = blockIdx.x % nseg;
    const GPos p = g_pos(a, blockIdx.x / nseg);
    const int64_t first = seg * a.seg_tiles;
    const int64_t last = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
    GRaw<S, false> cur;
    g_load<S, false>(a, p, first, cur);
    float carry = 0.0f, P = 1.0f;
    if (AGG) {
        // final_state may be initial_state itself: the second kernel, whose last segment writes
        // it while others may not have begun, takes the initial state from here
        if (seg == 0 && p.wave == 0 && p.live)
            a.seg[(p.b * a.nseg * 3 + 2) * a.C + p.c] = a.h0 ? a.h0[p.b * a.C + p.c] : 0.0f;
    } else {
        if (a.nseg > 1) carry = seg_at(a, p, 0, 2);
        else if (a.h0) carry = a.h0[p.b * a.C + p.c];
        for (int64_t s = 0; s < seg; ++s) carry = fold(seg_at(a, p, s, 0), seg_at(a, p, s, 1), carry);
        // every wavefront has its initial state in hand before the first barrier, hence before
        // wavefront 0 stores the final state
        asm volatile("" : "+v"(carry));
    }
    for (int64_t tile = first; tile < last; ++tile) {
        GRaw<S, false> nxt;
        g_load<S, false>(a, p, tile + 1 < last ? tile + 1 : tile, nxt);
        const int nv = g_valid(a, p, tile);
        const uint32_t st = g_starts(a, p, tile, cur);
        float av[kGT], uv[kGT], A, H;
        g_terms<S, SIG>(cur, nv, av, uv);
        g_span(av, uv, st, A, H);
        float(*s2)[2][64] = sp[tile & 1];
        s2[p.wave][0][p.lane] = A;
        s2[p.wave][1][p.lane] = H;
        __syncthreads();
        float h = carry;
#pragma unroll
        for (int w = 0; w < kGW; ++w) {
            if (w == p.wave) h = carry;
            const float Aw = s2[w][0][p.lane];
            carry = fold(Aw, s2[w][1][p.lane], carry);
            if (AGG) P = fold_mark(Aw, P);
        }
        if (!AGG) {
            using T = typename S::T;
            T* y = static_cast<T*>(a.y) + (p.b * a.L + tile * kGTile + p.wave * kGT) * a.y_row + p.c;
#pragma unroll
            for (int i = 0; i < kGT; ++i) {
                h = (st >> i) & 1 ? uv[i] : av[i] * h + uv[i];
                if (i < nv && p.live) S::store(y, i * a.y_row, h);
            }
        }
        cur = nxt;
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
template <class S, bool SIG, bool SEG>
__global__ void __launch_bounds__(kGThreads) gscan_bwd_states_kernel(GArgs a) {
    __shared__ float sp[2][kGW][SEG ? 3 : 2][64];
    const int64_t seg = blockIdx.x % a.nseg;
    const GPos p = g_pos(a, blockIdx.x / a.nseg);
    const int64_t first = seg * a.seg_tiles;
    const int64_t last = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
    GRaw<S, SEG> cur;
    g_load<S, SEG>(a, p, first, cur);
    float H = 0.0f, P = 1.0f, E = 0.0f;
    for (int64_t tile = first; tile < last; ++tile) {
        GRaw<S, SEG> nxt;
        g_load<S, SEG>(a, p, tile + 1 < last ? tile + 1 : tile, nxt);
        if (p.wave == 0 && p.live) {
            float* o = a.ckpt + (p.b * a.tiles + tile) * 2 * a.C + p.c;
            o[0] = P;
            o[a.C] = H;
        }
        const int nv = g_valid(a, p, tile);
        const uint32_t st = g_starts(a, p, tile, cur);
        float av[kGT], uv[kGT], Aw, Hw;
        g_terms<S, SIG>(cur, nv, av, uv);
        g_span(av, uv, st, Aw, Hw);
        auto s2 = sp[tile & 1];
        s2[p.wave][0][p.lane] = Aw;
        s2[p.wave][1][p.lane] = Hw;
        if constexpr (SEG) {
            float e = 0.0f;
#pragma unroll
            for (int i = kGT - 1; i >= 0; --i) {
                const float d = (i < nv ? S::load(cur.d, i) : 0.0f) + e;
                e = (st >> i) & 1 ? 0.0f : av[i] * d;
            }
            s2[p.wave][2][p.lane] = e;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kGW; ++w) {
            const float A1 = s2[w][0][p.lane];
            if constexpr (SEG) E = P < 0.0f ? E : P * s2[w][2][p.lane] + E;
            H = fold(A1, s2[w][1][p.lane], H);
            P = fold_mark(A1, P);
        }
        cur = nxt;
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
template <class S, bool SIG>
__global__ void __launch_bounds__(kGThreads) gscan_bwd_kernel(GArgs a) {
    __shared__ float sp[2][kGW][3][64];
    const int64_t seg = blockIdx.x % a.nseg;
    const GPos p = g_pos(a, blockIdx.x / a.nseg);
    const int64_t first = seg * a.seg_tiles;
    const int64_t last = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
    GRaw<S, true> cur;
    g_load<S, true>(a, p, last - 1, cur);
    float hseg = a.h0 ? a.h0[p.b * a.C + p.c] : 0.0f;
    for (int64_t s = 0; s < seg; ++s) hseg = fold(seg_at(a, p, s, 0), seg_at(a, p, s, 1), hseg);
    float carry = a.dhT ? a.dhT[p.b * a.C + p.c] : 0.0f;
    for (int64_t s = a.nseg - 1; s > seg; --s) carry = fold(seg_at(a, p, s, 0), seg_at(a, p, s, 2), carry);
    using T = typename S::T;
    for (int64_t tile = last - 1; tile >= first; --tile) {
        const float* ck = a.ckpt + (p.b * a.tiles + tile) * 2 * a.C + p.c;
        const float cA = ck[0], cH = ck[a.C];
        GRaw<S, true> nxt;
        g_load<S, true>(a, p, tile > first ? tile - 1 : tile, nxt);
        const int nv = g_valid(a, p, tile);
        const uint32_t st = g_starts(a, p, tile, cur);
        float av[kGT], uv[kGT], Aw, Hw, e = 0.0f;
        g_terms<S, SIG>(cur, nv, av, uv);
        g_span(av, uv, st, Aw, Hw);
#pragma unroll
        for (int i = kGT - 1; i >= 0; --i) {
            const float d = (i < nv ? S::load(cur.d, i) : 0.0f) + e;
            e = (st >> i) & 1 ? 0.0f : av[i] * d;
        }
        auto s3 = sp[tile & 1];
        s3[p.wave][0][p.lane] = Aw;
        s3[p.wave][1][p.lane] = Hw;
        s3[p.wave][2][p.lane] = e;
        __syncthreads();
        float h = fold(cA, cH, hseg), E = 0.0f;
#pragma unroll
        for (int w = 0; w < kGW; ++w)
            if (w < p.wave) h = fold(s3[w][0][p.lane], s3[w][1][p.lane], h);
#pragma unroll
        for (int w = kGW - 1; w >= 0; --w) {
            if (w == p.wave) E = carry;
            carry = fold(s3[w][0][p.lane], s3[w][2][p.lane], carry);
        }
        float before[kGT];  // h_{t-1}, 0 at a start
#pragma unroll
        for (int i = 0; i < kGT; ++i) {
            const bool s = (st >> i) & 1;
            before[i] = s ? 0.0f : h;
            h = s ? uv[i] : av[i] * h + uv[i];
        }
        const int64_t t0 = p.b * a.L + tile * kGTile + p.wave * kGT;
        T* dx = static_cast<T*>(a.dx) + t0 * a.dx_row + p.c;
        T* dg = static_cast<T*>(a.dgate) + t0 * a.dgate_row + p.c;
#pragma unroll
        for (int i = kGT - 1; i >= 0; --i) {
            if (i < nv) {
                const float D = S::load(cur.d, i) + E;
                float dlog = (st >> i) & 1 ? 0.0f : D * av[i] * before[i], dxv = D;
                if constexpr (SIG) {
                    float ag, in;
                    gates<SIG>(S::load(cur.g, i), ag, in);
                    dxv = D * in;
                    dlog = in * dlog - D * uv[i] * ag;
                }
                if (p.live) {
                    S::store(dx, i * a.dx_row, dxv);
                    S::store(dg, i * a.dgate_row, dlog);
                }
                E = (st >> i) & 1 ? 0.0f : av[i] * D;
            }
        }
        cur = nxt;
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

template <class S, bool SIG>
hipError_t fwd_typed(const GArgs& a, hipStream_t s) {
    const int64_t groups = a.B * ((a.C + 63) / 64);
    if (a.nseg > 1) {
        gscan_fwd_kernel<S, SIG, true><<<static_cast<uint32_t>(groups * (a.nseg - 1)), kGThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    gscan_fwd_kernel<S, SIG, false><<<static_cast<uint32_t>(groups * a.nseg), kGThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <class S, bool SIG>
hipError_t bwd_typed(const GArgs& a, hipStream_t s) {
    const uint32_t grid = static_cast<uint32_t>(a.B * ((a.C + 63) / 64) * a.nseg);
    if (a.nseg > 1) gscan_bwd_states_kernel<S, SIG, true><<<grid, kGThreads, 0, s>>>(a);
    else gscan_bwd_states_kernel<S, SIG, false><<<grid, kGThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    gscan_bwd_kernel<S, SIG><<<grid, kGThreads, 0, s>>>(a);
    return hipGetLastError();
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
    if (c.dtype == SSM_BF16) return c.sigmoid ? fwd_typed<BF16, true>(a, s) : fwd_typed<BF16, false>(a, s);
    return c.sigmoid ? fwd_typed<F32, true>(a, s) : fwd_typed<F32, false>(a, s);
}

hipError_t launch_gscan_bwd(const GscanCall& c, hipStream_t s) {
    GArgs a = g_args(c);
    g_cut(a);
    a.ckpt = static_cast<float*>(c.workspace);
    a.seg = a.ckpt + a.B * a.tiles * 2 * a.C;
    if (c.dtype == SSM_BF16) return c.sigmoid ? bwd_typed<BF16, true>(a, s) : bwd_typed<BF16, false>(a, s);
    return c.sigmoid ? bwd_typed<F32, true>(a, s) : bwd_typed<F32, false>(a, s);
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
