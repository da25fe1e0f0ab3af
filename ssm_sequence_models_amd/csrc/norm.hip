// norm.hip -- RMS / layer norm of a layer's rows with an optional SiLU gate, forward and
// backward (ssm_norm_fwd, ssm_norm_bwd).  Per row and group of m channels:
//     u = x, or x silu(z) (gate before the norm)
//     n = (u - mean) rstd,  rstd = 1 / sqrt(mean((u - mean)^2) + eps)   (mean = 0 for RMS)
//     pre = n w + b,  out = pre, or pre silu(z) (gate after the norm)
// and with d = dL/dpre w:
//     du = rstd (d - n mean(d n) - [layer] mean(d)),  dw = sum_rows dL/dpre n,  db = sum_rows dL/dpre.
//
// Both directions are bound by memory: every element is read once and written once, so a team
// of threads keeps its row's piece in registers from the load to the store, and the statistics
// (two steps for the layer norm: the mean, then the centred squares) are reductions over
// registers.  A team is one wavefront for m <= 1024 (four teams a block, no barrier) and one
// block above.  A team keeps its group and its columns while it walks over rows, so the
// weights are read once and the sums of dw and db stay in registers; each block writes one
// partial row, and a second kernel adds the partial rows in a fixed order in double
// (deterministic, no atomics).  All arithmetic is fp32; outputs are rounded once.
#include <type_traits>

#include "internal.h"

namespace ssm {
namespace {

struct NormArgs {
    const void *x, *z, *dout;
    const float *w, *b;
    void *out, *dx, *dz;
    float* part;  // [2][nb][channels]: partial sums of dw, then of db (one row a block)
    int64_t x_row, z_row, dout_row, out_row, dx_row, dz_row;
    int64_t rows, groups;
    int64_t nb;  // blocks a group
    int m;
    float eps;
    bool layer;
    bool want_dz, want_db;
};

// sum over the wavefront, in every lane
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// sum over the team, in every thread.  Block teams go through LDS: slot picks one of three
// buffers in turn, so that a buffer is written again only after a later barrier has shown
// that every thread has read it.
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float (*red)[16], int slot) {
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += red[slot][i];
    }
    return v;
}

__device__ __forceinline__ float sigmoidf(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// A thread's columns: eight consecutive ones, 16 bytes an access at any element's alignment.
// TAIL: the width is no multiple of eight, and the thread whose eight would pass the end takes the
// last eight instead.  Those it shares with the thread before it are computed twice and stored
// twice, the same values, and counted once, so that no access is under a branch of its own (bf16
// with a gate, 32768 x 2047, forward / backward: 89 / 152 us; the last few element by element
// 176 / 347; 32768 x 4097: 227 / 546, all element by element 816 / 1297).  Widths below eight go
// element by element.  Accesses are non-temporal, since nothing is used twice, but for fp32 at odd
// widths, where neighbours share lines (32768 x 4097 forward: 309 us, non-temporal 344).
constexpr int kVec = 8;
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

template <bool TAIL>
struct Cols {
    int at;     // first column
    int own;    // columns at + own .. are this thread's to count
    int width;  // the group's
    __device__ __forceinline__ Cols(int c, int m) : at(c), own(0), width(m) {
        if (TAIL && c + kVec > m && c < m) {
            at = m < kVec ? 0 : m - kVec;
            own = c - at;
        }
    }
    __device__ __forceinline__ bool counts(int e) const { return TAIL ? e >= own && at + e < width : at < width; }
};

template <class S, bool TAIL>
__device__ __forceinline__ void load_vec(const typename S::T* p, float (&v)[kVec], int m) {
    if (TAIL && m < kVec) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = i < m ? S::load(p, i < m ? i : 0) : 0.0f;
    } else if constexpr (S::kBytes == 2) {
        const u32x4_t q = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4_any* at = reinterpret_cast<const f32x4_any*>(p) + h;
            const f32x4_t q = TAIL ? static_cast<f32x4_t>(*at) : __builtin_nontemporal_load(at);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * h + i] = q[i];
        }
    }
}
template <class S, bool TAIL>
__device__ __forceinline__ void store_vec(typename S::T* p, const float (&v)[kVec], int m) {
    if (TAIL && m < kVec) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < m) S::store(p, i, v[i]);
    } else if constexpr (S::kBytes == 2) {
        u32x4_t q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4_any*>(p));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4_t q{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            f32x4_any* at = reinterpret_cast<f32x4_any*>(p) + h;
            if (TAIL) *at = q;
            else __builtin_nontemporal_store(q, at);
        }
    }
}

enum { kGateNone = 0, kGateBefore = 1, kGateAfter = 2 };

// Thread `tid` of a team of TPR holds, for j < NV, the 8 columns from 8 (j TPR + tid).
template <class S, bool TAIL, int NV, int TPR, int GATE>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_fwd_kernel(NormArgs a) {
    using T = typename S::T;
    __shared__ float red[3][16];
    constexpr int TEAMS = TPR == 64 ? 4 : 1;
    const int tid = threadIdx.x % TPR, team = threadIdx.x / TPR;
    const int64_t g = blockIdx.x % a.groups, blk = blockIdx.x / a.groups;
    const int m = a.m;
    const int64_t c0 = g * m;
    float w[NV][kVec], b[NV][kVec];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const bool in = c.at + (TAIL ? e : 0) < m;
            w[j][e] = in ? (a.w ? a.w[c0 + c.at + e] : 1.0f) : 0.0f;
            b[j][e] = in && a.b ? a.b[c0 + c.at + e] : 0.0f;
        }
    }
    const float inv_m = 1.0f / static_cast<float>(m);
    int slot = 0;
    for (int64_t r = blk * TEAMS + team; r < a.rows; r += a.nb * TEAMS) {
        const T* xr = static_cast<const T*>(a.x) + r * a.x_row + c0;
        const T* zr = GATE != kGateNone ? static_cast<const T*>(a.z) + r * a.z_row + c0 : nullptr;
        float u[NV][kVec], z[NV][kVec];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
            for (int e = 0; e < kVec; ++e) u[j][e] = z[j][e] = 0.0f;
            if (c.at < m) {
                load_vec<S, TAIL>(xr + c.at, u[j], m);
                if constexpr (GATE != kGateNone) load_vec<S, TAIL>(zr + c.at, z[j], m);
            }
        }
        float mean = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                if constexpr (GATE == kGateBefore) u[j][e] *= z[j][e] * sigmoidf(z[j][e]);
                mean += !TAIL || c.counts(e) ? u[j][e] : 0.0f;
            }
        }
        if (a.layer) {
            mean = team_sum<TPR>(mean, red, slot) * inv_m;
            slot = slot == 2 ? 0 : slot + 1;
        } else {
            mean = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float d = c.at < m ? u[j][e] - mean : 0.0f;
                u[j][e] = d;
                q += !TAIL || c.counts(e) ? d * d : 0.0f;
            }
        }
        q = team_sum<TPR>(q, red, slot) * inv_m;
        slot = slot == 2 ? 0 : slot + 1;
        const float rstd = 1.0f / sqrtf(q + a.eps);
        T* out = static_cast<T*>(a.out) + r * a.out_row + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
            float o[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                o[e] = u[j][e] * rstd * w[j][e] + b[j][e];
                if constexpr (GATE == kGateAfter) o[e] *= z[j][e] * sigmoidf(z[j][e]);
            }
            if (c.at < m) store_vec<S, TAIL>(out + c.at, o, m);
        }
    }
}

template <class S, bool TAIL, int NV, int TPR, int GATE>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_bwd_kernel(NormArgs a) {
    using T = typename S::T;
    __shared__ float red[3][16];
    constexpr int TEAMS = TPR == 64 ? 4 : 1;
    __shared__ float join[TEAMS == 4 ? 4 : 1][TEAMS == 4 ? 64 * kVec * NV : 1];
    const int tid = threadIdx.x % TPR, team = threadIdx.x / TPR;
    const int64_t g = blockIdx.x % a.groups, blk = blockIdx.x / a.groups;
    const int m = a.m;
    const int64_t c0 = g * m;
    float w[NV][kVec], b[NV][kVec], dw[NV][kVec], db[NV][kVec];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const bool in = c.at + (TAIL ? e : 0) < m;
            w[j][e] = in ? (a.w ? a.w[c0 + c.at + e] : 1.0f) : 0.0f;
            b[j][e] = GATE == kGateAfter && in && a.b ? a.b[c0 + c.at + e] : 0.0f;
            dw[j][e] = db[j][e] = 0.0f;
        }
    }
    const float inv_m = 1.0f / static_cast<float>(m);
    int slot = 0;
    for (int64_t r = blk * TEAMS + team; r < a.rows; r += a.nb * TEAMS) {
        const T* xr = static_cast<const T*>(a.x) + r * a.x_row + c0;
        const T* zr = GATE != kGateNone ? static_cast<const T*>(a.z) + r * a.z_row + c0 : nullptr;
        const T* dr = static_cast<const T*>(a.dout) + r * a.dout_row + c0;
        float x[NV][kVec], z[NV][kVec], d[NV][kVec], n[NV][kVec];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[j][e] = z[j][e] = d[j][e] = 0.0f;
            if (c.at < m) {
                load_vec<S, TAIL>(xr + c.at, x[j], m);
                if constexpr (GATE != kGateNone) load_vec<S, TAIL>(zr + c.at, z[j], m);
                load_vec<S, TAIL>(dr + c.at, d[j], m);
            }
        }
        float mean = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                n[j][e] = x[j][e];
                if constexpr (GATE == kGateBefore) n[j][e] *= z[j][e] * sigmoidf(z[j][e]);
                mean += !TAIL || c.counts(e) ? n[j][e] : 0.0f;
            }
        }
        if (a.layer) {
            mean = team_sum<TPR>(mean, red, slot) * inv_m;
            slot = slot == 2 ? 0 : slot + 1;
        } else {
            mean = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float v = c.at < m ? n[j][e] - mean : 0.0f;
                n[j][e] = v;
                q += !TAIL || c.counts(e) ? v * v : 0.0f;
            }
        }
        q = team_sum<TPR>(q, red, slot) * inv_m;
        slot = slot == 2 ? 0 : slot + 1;
        const float rstd = 1.0f / sqrtf(q + a.eps);
        T* dzr = GATE != kGateNone ? static_cast<T*>(a.dz) + r * a.dz_row + c0 : nullptr;
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
            float dzv[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                n[j][e] *= rstd;
                float dp = d[j][e];
                if constexpr (GATE == kGateAfter) {
                    const float sg = sigmoidf(z[j][e]);
                    const float pre = n[j][e] * w[j][e] + b[j][e];
                    dzv[e] = dp * pre * (sg * (1.0f + z[j][e] * (1.0f - sg)));
                    dp *= z[j][e] * sg;
                }
                dw[j][e] += dp * n[j][e];
                db[j][e] += dp;
                d[j][e] = dp * w[j][e];
                c1 += !TAIL || c.counts(e) ? d[j][e] * n[j][e] : 0.0f;
                c2 += !TAIL || c.counts(e) ? d[j][e] : 0.0f;
            }
            if constexpr (GATE == kGateAfter) {
                if (c.at < m && a.want_dz) store_vec<S, TAIL>(dzr + c.at, dzv, m);
            }
        }
        c1 = team_sum<TPR>(c1, red, slot) * inv_m;
        slot = slot == 2 ? 0 : slot + 1;
        if (a.layer) {
            c2 = team_sum<TPR>(c2, red, slot) * inv_m;
            slot = slot == 2 ? 0 : slot + 1;
        } else {
            c2 = 0.0f;
        }
        T* dxr = static_cast<T*>(a.dx) + r * a.dx_row + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Cols<TAIL> c((j * TPR + tid) * kVec, m);
            float dxv[kVec], dzv[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float du = rstd * (d[j][e] - n[j][e] * c1 - c2);
                dxv[e] = du;
                if constexpr (GATE == kGateBefore) {
                    const float sg = sigmoidf(z[j][e]);
                    dxv[e] = du * (z[j][e] * sg);
                    dzv[e] = du * x[j][e] * (sg * (1.0f + z[j][e] * (1.0f - sg)));
                }
            }
            if (c.at < m) {
                store_vec<S, TAIL>(dxr + c.at, dxv, m);
                if constexpr (GATE == kGateBefore)
                    if (a.want_dz) store_vec<S, TAIL>(dzr + c.at, dzv, m);
            }
        }
    }
    // this block's partial row: teams of one wavefront are first added in LDS, in order
    if (a.part == nullptr) return;
    for (int k = 0; k < (a.want_db ? 2 : 1); ++k) {
        float* out = a.part + (static_cast<int64_t>(k) * a.nb + blk) * a.groups * m + c0;
        if constexpr (TEAMS == 4) {
            if (k > 0) __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const Cols<TAIL> c((j * 64 + tid) * kVec, m);
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (c.counts(e)) join[team][c.at + e] = k == 0 ? dw[j][e] : db[j][e];
            }
            __syncthreads();
            for (int c = threadIdx.x; c < m; c += 256)
                out[c] = (join[0][c] + join[1][c]) + (join[2][c] + join[3][c]);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const Cols<TAIL> c((j * TPR + tid) * kVec, m);
                if (c.at < m) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (c.counts(e)) out[c.at + e] = k == 0 ? dw[j][e] : db[j][e];
                }
            }
        }
    }
}

// out[c] = sum over the nb partial rows in a fixed order, in double: 16 slices of the rows by
// 64 columns a block, the slices added through LDS.  blockIdx.y = 0: dw, 1: db.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* part, float* dw, float* db,
                                                           int64_t nb, int64_t channels) {
    __shared__ double sum[16][64];
    const int col = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + col;
    float* out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr) return;  // not asked for (the same for the whole block)
    const float* p = part + blockIdx.y * nb * channels;
    double s = 0.0;
    if (c < channels)
#pragma unroll 8
        for (int64_t r = slice; r < nb; r += 16) s += static_cast<double>(p[r * channels + c]);
    sum[slice][col] = s;
    __syncthreads();
    if (slice == 0 && c < channels) {
        for (int i = 1; i < 16; ++i) s += sum[i][col];
        out[c] = static_cast<float>(s);
    }
}

__global__ void norm_zero_kernel(float* dw, float* db, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    if (dw) dw[i] = 0.0f;
    if (db) db[i] = 0.0f;
}

// Blocks a group: 1024 in all (four wavefront teams a block for m <= 1024), never more than
// there are rows for; backward, four rows a team, since every block writes a partial row
// (2048 x 4096 bf16 33 -> 26 us, 4096 x 1024 30 -> 20; 512 rows the same).  At the size above with m = 512, forward / backward: 142 / 257 us; 512
// blocks 173 / 269, 2048 blocks 153 / 251 (m = 4096: 146 / 260, 185 / 258, 147 / 267).
int64_t norm_blocks(int64_t rows, int64_t m, int64_t groups, bool bwd) {
    const int64_t per = (m <= 1024 ? 4 : 1) * (bwd ? 4 : 1);
    const int64_t need = (rows + per - 1) / per;
    const int64_t most = groups >= 1024 ? 1 : 1024 / groups;
    return need < most ? need : most;
}

template <bool BWD, class S, bool TAIL, int NV, int TPR>
void launch_one(const NormArgs& a, int gate, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(a.nb * a.groups)), block(TPR > 256 ? TPR : 256);
    auto run = [&](auto g) {
        if constexpr (BWD) norm_bwd_kernel<S, TAIL, NV, TPR, decltype(g)::value><<<grid, block, 0, s>>>(a);
        else norm_fwd_kernel<S, TAIL, NV, TPR, decltype(g)::value><<<grid, block, 0, s>>>(a);
    };
    if (gate == kGateNone) run(std::integral_constant<int, kGateNone>{});
    else if (gate == kGateBefore) run(std::integral_constant<int, kGateBefore>{});
    else run(std::integral_constant<int, kGateAfter>{});
}

// Teams by the group's width m, bf16 with a gate at 32768 rows x 4096 channels (16384 x 8192),
// forward / backward in us (the same bytes: the floor is 130 / 217):
//   m = 512   one wavefront, one vector a lane 142 / 257    four wavefronts 344 / 546
//   m = 1024  one wavefront, two vectors 138 / 251          four wavefronts, half idle, 205 / 312
//   m = 4096  four wavefronts, two vectors 146 / 260        eight, one vector 149 / 235
//   m = 8192  16 wavefronts, one vector 138 / 279           eight, two vectors 151 / 350
// Far from the floor: m = 64, 128 and 256 (8, 16 and 32 lanes of a wavefront at work) 680 / 1030,
// 347 / 533 and 185 / 294; m = 16384 171 / 551, gate before 164 / 995 (backward 17 to 125 registers are
// spilled in the loop; at 8192 with the gate before 7).
template <bool BWD, class S, bool TAIL>
void launch_typed(const NormArgs& a, int gate, hipStream_t s) {
    const int m = a.m;
    if (m <= 512) return launch_one<BWD, S, TAIL, 1, 64>(a, gate, s);
    if (m <= 1024) return launch_one<BWD, S, TAIL, 2, 64>(a, gate, s);
    if (m <= 2048) return launch_one<BWD, S, TAIL, 1, 256>(a, gate, s);
    if (m <= 4096) {
        if constexpr (BWD) return launch_one<BWD, S, TAIL, 1, 512>(a, gate, s);
        else return launch_one<BWD, S, TAIL, 2, 256>(a, gate, s);
    }
    if (m <= 8192) return launch_one<BWD, S, TAIL, 1, 1024>(a, gate, s);
    launch_one<BWD, S, TAIL, 2, 1024>(a, gate, s);
}
template <bool BWD>
void launch_norm(const NormArgs& a, ssm_dtype_t dtype, int gate, hipStream_t s) {
    const bool tail = a.m % kVec != 0;
    if (dtype == SSM_BF16) tail ? launch_typed<BWD, BF16, true>(a, gate, s) : launch_typed<BWD, BF16, false>(a, gate, s);
    else tail ? launch_typed<BWD, F32, true>(a, gate, s) : launch_typed<BWD, F32, false>(a, gate, s);
}

}  // namespace

int64_t norm_partial_rows(int64_t rows, int64_t channels, int64_t groups) {
    return norm_blocks(rows, channels / groups, groups, true);
}

hipError_t launch_norm_fwd(const NormCall& c, hipStream_t s) {
    NormArgs a{};
    a.x = c.x; a.z = c.z; a.w = c.w; a.b = c.b; a.out = c.out;
    a.x_row = c.x_row; a.z_row = c.z_row; a.out_row = c.out_row;
    a.rows = c.rows; a.groups = c.groups;
    a.m = static_cast<int>(c.channels / c.groups);
    a.nb = norm_blocks(c.rows, a.m, c.groups, false);
    a.eps = c.eps; a.layer = c.layer;
    const int gate = c.z == nullptr ? kGateNone : c.gate_after ? kGateAfter : kGateBefore;
    launch_norm<false>(a, c.dtype, gate, s);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormCall& c, hipStream_t s) {
    if (c.rows == 0) {
        norm_zero_kernel<<<static_cast<uint32_t>((c.channels + 255) / 256), 256, 0, s>>>(c.dw, c.db, c.channels);
        return hipGetLastError();
    }
    NormArgs a{};
    a.x = c.x; a.z = c.z; a.dout = c.dout; a.w = c.w; a.b = c.b; a.dx = c.dx; a.dz = c.dz;
    a.x_row = c.x_row; a.z_row = c.z_row; a.dout_row = c.dout_row;
    a.dx_row = c.dx_row; a.dz_row = c.dz_row;
    a.rows = c.rows; a.groups = c.groups;
    a.m = static_cast<int>(c.channels / c.groups);
    a.nb = norm_blocks(c.rows, a.m, c.groups, true);
    a.eps = c.eps; a.layer = c.layer;
    a.want_dz = c.dz != nullptr;
    a.want_db = c.db != nullptr;
    a.part = c.dw || c.db ? static_cast<float*>(c.workspace) : nullptr;
    const int gate = c.z == nullptr ? kGateNone : c.gate_after ? kGateAfter : kGateBefore;
    launch_norm<true>(a, c.dtype, gate, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.part == nullptr) return e;
    const dim3 grid(static_cast<uint32_t>((c.channels + 63) / 64), c.db ? 2 : 1);
    norm_reduce_kernel<<<grid, 1024, 0, s>>>(a.part, c.dw, c.db, a.nb, c.channels);
    return hipGetLastError();
}

}  // namespace ssm
