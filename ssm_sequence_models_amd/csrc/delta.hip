// delta.hip -- the gated delta rule forward (formulas in delta.h): delta_prep, the walk along the
// rows, and the token-by-token form on state slots.
#include "delta.h"

namespace ssm {
namespace {

using namespace delta;

// ---------------------------------------------------------------------------------------
// delta_prep: T, M and the factors of one chunk of one head, a block of Q / 16 wavefronts
//
// Wavefront w forms the rows 16 w .. of k . k and q . k (exact products, fp32 sums) and the
// factors r of its pairs from differences of double sums, each pair by its own exponential: no
// factor leaves the range that the pair's own decay has.  T by blocks of 16: the diagonal blocks
// by forward substitution, one column a lane; then wavefront j takes the blocks below (j, j)
// down its column, T_ij = -T_ii sum_m D_im T_mj, whose results are the next products' operands
// where they lie.  (A product form of the inverse, (I - D)(I + D^2) .., loses everything where
// keys repeat: the powers of D grow as binomials while T itself stays small.)
// ---------------------------------------------------------------------------------------
template <class MM>
__global__ __launch_bounds__(MM::Q * 4) void delta_prep_kernel(DeltaArgs a, int mparts) {
    using S = typename MM::S;
    constexpr int Q = MM::Q, RT = Q / 16, LD = Q + 4;
    __shared__ __attribute__((aligned(16))) float sd[Q * LD];       // D
    __shared__ __attribute__((aligned(16))) float st[Q * LD];       // T
    __shared__ __attribute__((aligned(16))) float sm[Q * LD];       // M
    __shared__ __attribute__((aligned(16))) float sii[RT][16 * 20];  // T's diagonal blocks
    __shared__ double sg[Q];
    __shared__ int sr[Q];
    __shared__ float sbeta[Q];
    __shared__ int sbad;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t unit = xcd_order(blockIdx.x, gridDim.x);  // (b, chunk, h): the heads of a key head are neighbours
    const int64_t h = unit % a.H, bc = unit / a.H, c = bc % a.chunks, b = bc / a.chunks;
    const int64_t g = h / (a.H / a.G), t0 = c * Q;
    const int valid = static_cast<int>(a.L - t0 < Q ? a.L - t0 : Q), N = static_cast<int>(a.N);
    const int64_t image = (b * a.H + h) * a.chunks + c;

    if (tid == 0) sbad = 0;
    if (w == 0) {
        const TokenSums s = token_sums<Q>(a, b, h, t0, valid, lane);
        const double end = __shfl(s.gates, Q - 1);
        const int rend = __shfl(s.starts, Q - 1);
        if (lane < Q) {
            sg[lane] = s.gates;
            sr[lane] = s.starts;
            sbeta[lane] = s.beta;
            float* f = a.factors + image * kFactors * Q;
            f[lane] = s.starts == 0 ? exp_of(s.gates) : 0.0f;
            f[Q + lane] = s.starts == rend ? exp_of(end - s.gates) : 0.0f;
            f[2 * Q + lane] = s.beta;
            f[3 * Q + lane] = static_cast<float>(s.starts);
        }
    }
    for (int i = tid; i < Q * LD; i += Q * 4) st[i] = sm[i] = 0.0f;
    // products of the rows 16 w ..
    f4 kk[RT], qk[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) kk[j] = qk[j] = f4{0, 0, 0, 0};
    const S* kp = static_cast<const S*>(a.k) + (b * a.L + t0) * a.k_row + g * a.N;
    const S* qp = static_cast<const S*>(a.q) + (b * a.L + t0) * a.q_row + g * a.N;
    const int rows = 16 * w + li;
    const u4 none{0, 0, 0, 0};
    bool bad = false;
    for (int n = MM::R * g4; n < N + MM::R * g4; n += MM::KB) {  // the same number of steps in every lane
        const auto fk = MM::exact(rows < valid ? MM::load_run(kp + rows * a.k_row, n, N) : none);
        const auto fq = MM::exact(rows < valid ? MM::load_run(qp + rows * a.q_row, n, N) : none);
        bad = bad || MM::not_finite(fk) || MM::not_finite(fq);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            if (j > w) continue;
            const int s = 16 * j + li;
            const auto fs = j == w ? fk : MM::exact(s < valid ? MM::load_run(kp + s * a.k_row, n, N) : none);
            MM::template mac<1, 1>(kk[j], fk, fs);
            MM::template mac<1, 1>(qk[j], fq, fs);
        }
    }
    __syncthreads();
    const bool several = sr[Q - 1] != 0;
    if (bad && several) sbad = 1;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        if (j > w) continue;
        const int s = 16 * j + li;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 16 * w + 4 * g4 + e;
            const float r = s <= t && sr[s] == sr[t] ? exp_of(sg[t] - sg[s]) : 0.0f;
            // a factor of 0 leaves nothing of what is not finite either
            sd[t * LD + s] = s < t && r != 0.0f ? r * kk[j][e] * sbeta[s] : 0.0f;
            sm[t * LD + s] = r != 0.0f ? r * qk[j][e] * a.scale : 0.0f;
        }
    }
    __syncthreads();
    {  // T_ww, column li
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == li ? 1.0f : 0.0f;
#pragma unroll
            for (int m = 0; m < i; ++m) v -= sd[(16 * w + i) * LD + 16 * w + m] * x[m];
            x[i] = v = i < li ? 0.0f : v;  // nothing above the diagonal, whatever D holds
            if (g4 == 0) sii[w][i * 20 + li] = st[(16 * w + i) * LD + 16 * w + li] = v;
        }
    }
    __syncthreads();
    {  // the blocks below (w, w)
        f4 x[RT];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[0][e] = sii[w][(4 * g4 + e) * 20 + li];
#pragma unroll
        for (int d = 1; d < RT; ++d) {
            if (w + d >= RT) continue;
            const int i = w + d;
            f4 sum{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < d; ++m) {
                const f4 l = *reinterpret_cast<const f4*>(&sd[(16 * i + li) * LD + 16 * (w + m) + 4 * g4]);
                ByF32::mac<1, 1>(sum, ByF32::Frag<1>{l}, ByF32::Frag<1>{x[m]});
            }
            if (several) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (sr[16 * i + 4 * g4 + e] != sr[16 * w + li]) sum[e] = 0.0f;
            }
            f4 out{0, 0, 0, 0};
            const f4 l = *reinterpret_cast<const f4*>(&sii[i][li * 20 + 4 * g4]);
            ByF32::mac<1, 1>(out, ByF32::Frag<1>{l}, ByF32::Frag<1>{sum});
            x[d] = -out;
#pragma unroll
            for (int e = 0; e < 4; ++e) st[(16 * i + 4 * g4 + e) * LD + 16 * w + li] = x[d][e];
        }
    }
    __syncthreads();
    if (sbad && tid < Q) a.factors[image * kFactors * Q + 3 * Q + tid] = static_cast<float>(sr[tid]) + kNotFinite;
    // out in parts, R values a piece
    uint8_t* T = a.T + image * image_bytes<MM>(MM::TP);
    uint8_t* M = a.M + image * image_bytes<MM>(mparts);
    constexpr int PIECES = Q / MM::R;
    for (int i = tid; i < Q * PIECES; i += Q * 4) {
        const int r = i / PIECES, q = i % PIECES;
        float v[MM::R], m[MM::R];
#pragma unroll
        for (int j = 0; j < MM::R; ++j) {
            const int s = MM::R * q + j;
            v[j] = sr[s] == sr[r] ? st[r * LD + s] : 0.0f;
            m[j] = sm[r * LD + s];
        }
        if constexpr (MM::TP == 1) {
            reinterpret_cast<f4*>(T)[i] = f4{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f4*>(M)[i] = f4{m[0], m[1], m[2], m[3]};
        } else {
            const auto ft = MM::template parts<3>(v);
            const auto fm = MM::template parts<3>(m);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                reinterpret_cast<bf8*>(T)[p * Q * PIECES + i] = ft.p[p];
                if (p < mparts) reinterpret_cast<bf8*>(M)[p * Q * PIECES + i] = fm.p[p];
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// The walk: 16 channels of a head a wavefront, four wavefronts a block
// ---------------------------------------------------------------------------------------
// SAVE: for the backward, the states and E in place of y
template <class MM, int NT, bool SAVE>
__global__ __launch_bounds__(256) void delta_walk_kernel(DeltaArgs a, DeltaSaved keep) {
    using S = typename MM::S;
    constexpr int Q = MM::Q, RT = Q / 16, KT = Q / MM::KB, W = 16 * NT, KN = W / MM::KB;
    constexpr int MP = m_parts<MM>(false);
    constexpr int QQ = MM::template tile_bytes<Q>(Q), QN = MM::template tile_bytes<W>(Q);
    __shared__ __attribute__((aligned(16))) uint8_t sk[QN];
    __shared__ __attribute__((aligned(16))) uint8_t sq[SAVE ? 16 : QN];
    __shared__ __attribute__((aligned(16))) uint8_t st[MM::TP * QQ];
    __shared__ __attribute__((aligned(16))) uint8_t sm[SAVE ? 16 : MP * QQ];
    __shared__ __attribute__((aligned(16))) float sf[kFactors * Q];
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t pblocks = (a.P + 63) / 64;
    const int64_t unit = xcd_order(blockIdx.x, gridDim.x);
    const int64_t pb = unit % pblocks, bh = unit / pblocks, h = bh % a.H, b = bh / a.H;
    const int64_t g = h / (a.H / a.G);
    const int64_t p0 = 64 * pb + 16 * w, p = p0 + li;
    const bool mine = p0 < a.P, have = p < a.P;
    const int N = static_cast<int>(a.N);
    const int64_t state = (bh * a.P + p) * a.N;
    f4 hs[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = 16 * i + 4 * g4;
        hs[i] = have && n < N && a.h0 ? *reinterpret_cast<const f4*>(a.h0 + state + n) : f4{0, 0, 0, 0};
    }
    for (int64_t c = 0; c < a.chunks; ++c) {
        const int64_t t0 = b * a.L + c * Q, image = bh * a.chunks + c;
        const int valid = static_cast<int>(a.L - c * Q < Q ? a.L - c * Q : Q);
        if (SAVE && have) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int n = 16 * i + 4 * g4;
                if (n < N) *reinterpret_cast<f4*>(keep.states + (image * a.P + p) * a.N + n) = hs[i];
            }
        }
        __syncthreads();
        stage_rows<MM, W, 256>(sk, static_cast<const S*>(a.k) + t0 * a.k_row + g * a.N, a.k_row, valid, N);
        if (!SAVE) stage_rows<MM, W, 256>(sq, static_cast<const S*>(a.q) + t0 * a.q_row + g * a.N, a.q_row, valid, N);
        stage_image<MM, 256>(st, a.T + image * image_bytes<MM>(MM::TP), MM::TP);
        if (!SAVE) stage_image<MM, 256>(sm, a.M + image * image_bytes<MM>(MP), MP);
        if (tid < kFactors * Q) sf[tid] = a.factors[image * kFactors * Q + tid];
        __syncthreads();
        const int begun = static_cast<int>(sf[4 * Q - 1]) % 1024;
        const bool clean = sf[4 * Q - 1] < kNotFinite;
        if (clean && !mine) continue;
        f4 z[RT], y[RT], x[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            z[i] = y[i] = x[i] = f4{0, 0, 0, 0};
            if (have) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * i + 4 * g4 + e;
                    if (t < valid) x[i][e] = MM::value(static_cast<const S*>(a.v) + (t0 + t) * a.v_row + h * a.P, p);
                }
            }
        }
        // K h^T and Q h^T
#pragma unroll
        for (int kk = 0; kk < KN; ++kk) {
            const auto s = MM::template of_tiles<3>(hs, kk);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                MM::template mac<1, 3>(z[i], MM::template rows<W>(sk, 16 * i, kk, li, g4), s);
                if (!SAVE) MM::template mac<1, 3>(y[i], MM::template rows<W>(sq, 16 * i, kk, li, g4), s);
            }
        }
        // Z = V - e^G K h^T, E = T Z
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const f4 f = lds<f4>(reinterpret_cast<const uint8_t*>(sf + 16 * i + 4 * g4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // nothing of a state that a start has cut off
                z[i][e] = x[i][e] - (f[e] != 0.0f ? f[e] * z[i][e] : 0.0f);
                y[i][e] = f[e] != 0.0f ? f[e] * a.scale * y[i][e] : 0.0f;
            }
            x[i] = f4{0, 0, 0, 0};
        }
        by_sequences(x, z, sf + 3 * Q, begun, g4, [&](f4 (&out)[RT], const f4 (&in)[RT]) {
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const auto s = MM::template of_tiles<3>(in, kk);
#pragma unroll
                for (int i = kk * MM::KB / 16; i < RT; ++i) {
                    const auto l = of_parts<MM, MM::TP>([&](int q) { return MM::template rows<Q>(st + q * QQ, 16 * i, kk, li, g4); });
                    MM::template mac<MM::TP, 3>(out[i], l, s);
                }
            }
        });
        if (SAVE && have) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * i + 4 * g4 + e;
                    if (t < valid) keep.e[((t0 + t) * a.H + h) * a.P + p] = x[i][e];
                }
        }
        // U = b E, Y += M U
#pragma unroll
        for (int i = 0; i < RT; ++i) x[i] *= lds<f4>(reinterpret_cast<const uint8_t*>(sf + 2 * Q + 16 * i + 4 * g4));
#pragma unroll
        for (int kk = 0; kk < (SAVE ? 0 : KT); ++kk) {
            const auto s = MM::template of_tiles<MP>(x, kk);
#pragma unroll
            for (int i = kk * MM::KB / 16; i < RT; ++i) {
                const auto l = of_parts<MM, MP>([&](int q) { return MM::template rows<Q>(sm + q * QQ, 16 * i, kk, li, g4); });
                MM::template mac<MP, MP>(y[i], l, s);
            }
        }
        if (!SAVE && have) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * i + 4 * g4 + e;
                    if (t < valid) MM::store(static_cast<S*>(a.y) + (t0 + t) * a.y_row + h * a.P, p, y[i][e]);
                }
        }
        // the state after the chunk
        if (!clean) {
            __syncthreads();
            clear_rows<MM, W>(sk, sf + Q);
            __syncthreads();
        }
        const float through = sf[Q - 1];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) hs[i][e] = through != 0.0f ? through * hs[i][e] : 0.0f;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const f4 f = lds<f4>(reinterpret_cast<const uint8_t*>(sf + Q + 16 * i + 4 * g4));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = f[e] != 0.0f ? f[e] * x[i][e] : 0.0f;
        }
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            const auto s = MM::template of_tiles<3>(x, kk);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                MM::template mac<1, 3>(hs[i], MM::template columns<W>(sk, kk * MM::KB, i, li, g4), s);
        }
    }
    if (!SAVE && a.final_state && have) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = 16 * i + 4 * g4;
            if (n < N) *reinterpret_cast<f4*>(a.final_state + state + n) = hs[i];
        }
    }
}

// ---------------------------------------------------------------------------------------
// Token by token: the decode step.  Eight lanes hold a channel's state, 128 bytes side by side
// of it a load, RG channels eight apart a lane; a wavefront is a unit of its own.  The state's
// one read and one write are the whole cost (256 requests of 32 heads x 128 x 128: 1 GiB).
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ float sum8(float v) {  // over the eight lanes of a channel
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));          // i ^ 1
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));          // i ^ 2
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));  // half mirror
}

template <class D>
__device__ __forceinline__ f4 four(const typename D::T* p);
template <>
__device__ __forceinline__ f4 four<BF16>(const uint16_t* p) {
    const u2 v = *reinterpret_cast<const u2any*>(p);
    return f4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
              __uint_as_float(v[1] & 0xFFFF0000u)};
}
template <>
__device__ __forceinline__ f4 four<F32>(const float* p) {
    return __builtin_bit_cast(f4, *reinterpret_cast<const u4any4*>(p));
}

template <class D, int NI, int RG>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStep s, int64_t units) {
    using S = typename D::T;
    const DeltaArgs& a = s.a;
    const int lane = threadIdx.x & 63, l8 = lane & 7;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (unit >= units) return;
    const int64_t slabs = (a.P + 8 * RG - 1) / (8 * RG);
    const int64_t slab = unit % slabs, bh = unit / slabs, h = bh % a.H, b = bh / a.H, g = h / (a.H / a.G);
    const int64_t p0 = slab * 8 * RG + (lane >> 3);
    const int N = static_cast<int>(a.N);
    const int64_t slot = s.slots ? s.slots[b] : b;
    if (slot < 0 || slot >= s.n_slots) {
        for (int64_t t = 0; t < a.L; ++t)
            for (int r = 0; r < RG; ++r)
                if (l8 == 0 && p0 + 8 * r < a.P)
                    D::store(static_cast<S*>(a.y) + (b * a.L + t) * a.y_row + h * a.P, p0 + 8 * r, 0.0f);
        return;
    }
    f4 hs[RG][NI];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = 32 * i + 4 * l8;
            hs[r][i] = f4{0, 0, 0, 0};
            if (s.state_in && n < N && p0 + 8 * r < a.P)
                hs[r][i] = __builtin_nontemporal_load(
                    reinterpret_cast<const f4*>(s.state_in + ((slot * a.H + h) * a.P + p0 + 8 * r) * a.N + n));
        }
    for (int64_t t = 0; t < a.L; ++t) {
        const int64_t row = b * a.L + t;
        const S* kp = static_cast<const S*>(a.k) + row * a.k_row + g * a.N;
        const S* qp = static_cast<const S*>(a.q) + row * a.q_row + g * a.N;
        f4 k[NI], q[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = 32 * i + 4 * l8;
            k[i] = q[i] = f4{0, 0, 0, 0};
            if (n < N) {
                k[i] = four<D>(kp + n);
                q[i] = four<D>(qp + n);
            }
        }
        float v[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r)
            v[r] = p0 + 8 * r < a.P ? D::load(static_cast<const S*>(a.v) + row * a.v_row + h * a.P, p0 + 8 * r) : 0.0f;
        const float be = a.beta[row * a.H + h];
        float f = a.gate ? exp_of(gate_of(a.gate[row * a.H + h])) : 1.0f;
        const bool cut = a.seq && t > 0 && a.seq[row] != a.seq[row - 1];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            float kh = 0.0f, y = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hs[r][i][e] = cut ? 0.0f : f * hs[r][i][e];
                    kh += hs[r][i][e] * k[i][e];
                }
            const float u = be * (v[r] - sum8(kh));
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hs[r][i][e] += u * k[i][e];
                    y += hs[r][i][e] * q[i][e];
                }
            y = sum8(y);
            if (l8 == 0 && p0 + 8 * r < a.P) D::store(static_cast<S*>(a.y) + row * a.y_row + h * a.P, p0 + 8 * r, a.scale * y);
        }
    }
    if (s.state_out) {
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int n = 32 * i + 4 * l8;
                if (n < N && p0 + 8 * r < a.P)
                    __builtin_nontemporal_store(
                        hs[r][i], reinterpret_cast<f4*>(s.state_out + ((slot * a.H + h) * a.P + p0 + 8 * r) * a.N + n));
            }
    }
}

template <class D, int NI, int RG>
hipError_t step_of(const DeltaStep& s, hipStream_t stream) {
    const int64_t units = s.a.B * s.a.H * ((s.a.P + 8 * RG - 1) / (8 * RG));
    delta_step_kernel<D, NI, RG><<<static_cast<unsigned>((units + 3) / 4), 256, 0, stream>>>(s, units);
    return hipGetLastError();
}
template <class D>
hipError_t step_by_width(const DeltaStep& s, hipStream_t stream) {
    if (s.a.N <= 32) return step_of<D, 1, 4>(s, stream);
    if (s.a.N <= 64) return step_of<D, 2, 4>(s, stream);
    if (s.a.N <= 128) return step_of<D, 4, 4>(s, stream);
    return step_of<D, 8, 2>(s, stream);
}

template <class MM, int NT, bool SAVE>
hipError_t walk_of(const DeltaArgs& a, const DeltaSaved& keep, hipStream_t stream) {
    const int64_t blocks = a.B * a.H * ((a.P + 63) / 64);
    delta_walk_kernel<MM, NT, SAVE><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a, keep);
    return hipGetLastError();
}
template <class MM, bool SAVE>
hipError_t walk_by_width(const DeltaArgs& a, const DeltaSaved& keep, hipStream_t stream) {
    if (a.N <= 64) return walk_of<MM, 4, SAVE>(a, keep, stream);
    if (a.N <= 128) return walk_of<MM, 8, SAVE>(a, keep, stream);
    return walk_of<MM, 16, SAVE>(a, keep, stream);
}
template <class MM>
hipError_t fwd_of(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream) {
    place_chunks<MM>(a, static_cast<uint8_t*>(workspace), false);
    const hipError_t e = launch_delta_prep(a, dtype, false, stream);
    return e != hipSuccess ? e : walk_by_width<MM, false>(a, DeltaSaved{}, stream);
}

}  // namespace

hipError_t launch_delta_prep(const DeltaArgs& a, ssm_dtype_t dtype, bool bwd, hipStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(a.B * a.H * a.chunks);
    if (dtype == SSM_BF16) delta_prep_kernel<ByBf16><<<blocks, 256, 0, stream>>>(a, m_parts<ByBf16>(bwd));
    else delta_prep_kernel<ByF32><<<blocks, 128, 0, stream>>>(a, m_parts<ByF32>(bwd));
    return hipGetLastError();
}

hipError_t launch_delta_walk_saved(const DeltaArgs& a, const DeltaSaved& s, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? walk_by_width<ByBf16, true>(a, s, stream) : walk_by_width<ByF32, true>(a, s, stream);
}

size_t delta_fwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype) {
    DeltaArgs a{};
    a.B = B;
    a.L = L;
    a.H = H;
    return dtype == SSM_BF16 ? place_chunks<ByBf16>(a, nullptr, false) : place_chunks<ByF32>(a, nullptr, false);
}

hipError_t launch_delta_fwd(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? fwd_of<ByBf16>(a, workspace, dtype, stream) : fwd_of<ByF32>(a, workspace, dtype, stream);
}

hipError_t launch_delta_step(const DeltaStep& s, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? step_by_width<BF16>(s, stream) : step_by_width<F32>(s, stream);
}

}  // namespace ssm
