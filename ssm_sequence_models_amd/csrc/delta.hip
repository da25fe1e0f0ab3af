// delta.hip -- the gated delta rule forward (formulas in delta.h): delta_prep, the walk along the
// rows, and the token-by-token form on state slots.
#include <type_traits>

#include "delta.h"

namespace ssm {
namespace {

using namespace delta;

// ---------------------------------------------------------------------------------------
// delta_prep: T, M and the factors of one chunk of one head, a block of Q / 16 wavefronts
//
// Wavefront w forms the rows t = 16 w .. of k . k and q . k (exact products, fp32 sums) with the keys
// s as the instruction's rows, so that lane (li, g4) holds the pairs of t = 16 w + li with four
// neighbouring s: the order of the left operands that T and M are for the walk, which leave
// from registers.  The factors r of the pairs come from differences of double sums, each by its
// own exponential: no factor leaves the range that the pair's own decay has.  T (I + D) = I by
// blocks of 16, from a row's diagonal block to the left: the diagonal block by substitution, a row
// a lane; then T_ij = -(sum_m T_im D_mj) T_jj, transposed, so that results are the next
// products' operands where they lie.  (A product form of the inverse, (I - D)(I + D^2) .., loses
// everything where keys repeat: the powers of D grow as binomials while T itself stays small.)
// The heads of a key head go through the products once, up to a wavefront's worth of them a block (4 x 8192 x
// 32 heads of 16 key heads, dstate 128: 195 to 220 us, backward 240 to 250; a head a block took 62 and 65 more).  What
// bounds it: the chain of a row's substitution and its syncs at four wavefronts a SIMD (vector instructions busy
// half of the time, matrix ones a tenth), and 0.62 GB of images written (backward 0.93).  (Six wavefronts a
// SIMD: spills, slower.)
// ---------------------------------------------------------------------------------------
template <class MM, int NT, bool BWD, bool DIRECT>
__global__ __launch_bounds__(MM::Q * 4, NT <= 8 ? 4 : 1) void delta_prep_kernel(DeltaArgs a, int heads) {
    using S = typename MM::S;
    constexpr int Q = MM::Q, RT = Q / 16, KT = Q / MM::KB, LD = Q + 4, R = MM::R, KN = 16 * NT / MM::KB;
    __shared__ __attribute__((aligned(16))) float sd[Q * LD];        // D transposed: [s][t]
    __shared__ __attribute__((aligned(16))) float sii[RT][16 * 20];  // T's diagonal blocks, transposed
    float* const so = sd;  // T and M on the way out, once D is used up
    __shared__ __attribute__((aligned(16))) double sgs[RT][Q];
    __shared__ __attribute__((aligned(16))) int sr[Q];
    __shared__ __attribute__((aligned(16))) float sbetas[RT][Q];
    __shared__ int sbad;
    const int tid = threadIdx.x, lane = tid & 63, li_ = lane & 15, g4_ = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = xcd_order(blockIdx.x, gridDim.x);  // (b, chunk, heads): those of a key head are neighbours
    const int H = static_cast<int>(a.H), ranges = H / heads, h0 = unit % ranges * heads, bc = unit / ranges;
    const int c = bc % static_cast<int>(a.chunks), b = bc / static_cast<int>(a.chunks);
    const int64_t g = h0 / (H / static_cast<int>(a.G)), t0 = static_cast<int64_t>(c) * Q;
    const int valid = static_cast<int>(a.L - t0 < Q ? a.L - t0 : Q), N = static_cast<int>(a.N);
    const int64_t first_image = (static_cast<int64_t>(b) * H + h0) * a.chunks + c;

    if (tid == 0) sbad = 0;
    if (w < heads) {
        const TokenSums s = token_sums<Q>(a, b, h0 + w, t0, valid, lane);
        const double end = __shfl(s.gates, Q - 1);
        const int rend = __shfl(s.starts, Q - 1);
        if (lane < Q) {
            const int64_t image = first_image + w * a.chunks;
            sgs[w][lane] = s.gates * kLog2e;
            sbetas[w][lane] = s.beta;
            if (w == 0) sr[lane] = s.starts;
            float* f = a.factors + image * kFactors * Q;
            f[lane] = s.starts == 0 ? exp_of(s.gates) : 0.0f;
            f[Q + lane] = s.starts == rend ? exp_of(end - s.gates) : 0.0f;
            f[2 * Q + lane] = s.beta;
            if (BWD) a.gates[image * Q + lane] = s.gates;
        }
    }
    // products of the rows 16 w ..; rows behind the row's end are 0
    f4 kk[RT], qk[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) kk[j] = qk[j] = f4{0, 0, 0, 0};
    const int64_t first = b * a.L + t0;
    const S* kp = static_cast<const S*>(a.k) + first * a.k_row + g * a.N;
    const S* qp = static_cast<const S*>(a.q) + first * a.q_row + g * a.N;
    const Buffer rk = token_buffer<S>(a.k, first, a.k_row, g * a.N, DIRECT ? valid : 1, a.N);
    const Buffer rq = token_buffer<S>(a.q, first, a.q_row, g * a.N, DIRECT ? valid : 1, a.N);
    const auto load = [&](Buffer r, const S* p, int64_t row, int t, int kb) {
        const int n = MM::KB * kb + R * g4_;
        if (DIRECT)
            return __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(
                                              r, n < N ? (t * static_cast<uint32_t>(row) + n) * sizeof(S) : kOutside, 0, 0));
        return t < valid ? MM::load_run(p + t * row, n, N) : u4{0, 0, 0, 0};
    };
    bool bad = false;
    u4 fk[KN], fq[KN];
#pragma unroll
    for (int kb = 0; kb < KN; ++kb) fk[kb] = load(rk, kp, a.k_row, 16 * w + li_, kb);
#pragma unroll
    for (int kb = 0; kb < KN; ++kb) fq[kb] = load(rq, qp, a.q_row, 16 * w + li_, kb);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        if (j > w) continue;
        u4 fs[KN];
#pragma unroll
        for (int kb = 0; kb < KN; ++kb) fs[kb] = j == w ? fk[kb] : load(rk, kp, a.k_row, 16 * j + li_, kb);
#pragma unroll
        for (int kb = 0; kb < KN; ++kb) {
            MM::template mac<1, 1>(kk[j], MM::exact(fs[kb]), MM::exact(fk[kb]));
            MM::template mac<1, 1>(qk[j], MM::exact(fs[kb]), MM::exact(fq[kb]));
        }
    }
#pragma unroll
    for (int kb = 0; kb < KN; ++kb) bad = bad || MM::not_finite(MM::exact(fk[kb])) || MM::not_finite(MM::exact(fq[kb]));
    __syncthreads();
    const bool several = sr[Q - 1] != 0;
    if (bad && several) sbad = 1;
    for (int hh = 0; hh < heads; ++hh) {
        const int li = here(li_), g4 = here(g4_);  // addresses are formed where they are used, not kept over the loop
        const int t = 16 * w + li, rt = sr[t];
        const int64_t image = first_image + hh * a.chunks;
        const double* const sg = sgs[hh];
        const float* const sbeta = sbetas[hh];
        const double gt = sg[t];
        f4 md[RT];  // M's rows t
#pragma unroll
        for (int j = 0; j < RT; ++j) md[j] = f4{0, 0, 0, 0};
        if (hh > 0) __syncthreads();  // D's place
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            if (j > w) continue;
            const f4 be = *reinterpret_cast<const f4*>(&sbeta[16 * j + 4 * g4]);
            f4 r;
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = exp2_of(gt - sg[16 * j + 4 * g4 + e]);
            if (several) {
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = sr[16 * j + 4 * g4 + e] == rt ? r[e] : 0.0f;
            }
            f4 dd = r * kk[j] * be, mm = r * qk[j] * a.scale;
            if (several) {  // another sequence's factor leaves nothing of what is not finite either
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dd[e] = r[e] != 0.0f ? dd[e] : 0.0f;
                    mm[e] = r[e] != 0.0f ? mm[e] : 0.0f;
                }
            }
            if (j == w) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dd[e] = 4 * g4 + e < li ? dd[e] : 0.0f;
                    mm[e] = 4 * g4 + e <= li ? mm[e] : 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sd[(16 * j + 4 * g4 + e) * LD + t] = dd[e];
            md[j] = mm;
        }
        __syncthreads();
        f4 x[RT];  // T's rows t: x[j][e] is T_ts of s = 16 j + 4 g4 + e
        {          // the diagonal block, row li of it in every g4
            float v[16];
#pragma unroll
            for (int j = 15; j >= 0; --j) {
                float sum = j == li ? 1.0f : 0.0f;
#pragma unroll
                for (int m = j + 1; m < 16; ++m) sum -= v[m] * sd[(16 * w + j) * LD + 16 * w + m];
                v[j] = j > li ? 0.0f : sum;  // nothing above the diagonal, whatever D holds
            }
            f4 d;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[e] = g4 == 0 ? v[e] : g4 == 1 ? v[4 + e] : g4 == 2 ? v[8 + e] : v[12 + e];
                sii[w][(4 * g4 + e) * 20 + li] = d[e];
            }
#pragma unroll
            for (int j = 0; j < RT; ++j) x[j] = j == w ? d : f4{0, 0, 0, 0};
        }
        __syncthreads();
#pragma unroll
        for (int j = RT - 2; j >= 0; --j) {
            if (j >= w) continue;
            f4 sum{0, 0, 0, 0}, out{0, 0, 0, 0};
#pragma unroll
            for (int m = j + 1; m < RT; ++m) {
                if (m > w) continue;
                const f4 l = *reinterpret_cast<const f4*>(&sd[(16 * j + li) * LD + 16 * m + 4 * g4]);
                ByF32::mac<1, 1>(sum, ByF32::Frag<1>{l}, ByF32::Frag<1>{x[m]});
            }
            if (several) {  // sequences apart: a 0 of another's is not one times what is not finite
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (sr[16 * j + 4 * g4 + e] != rt) sum[e] = 0.0f;
            }
            const f4 l = *reinterpret_cast<const f4*>(&sii[j][li * 20 + 4 * g4]);
            ByF32::mac<1, 1>(out, ByF32::Frag<1>{l}, ByF32::Frag<1>{sum});
            x[j] = -out;
        }
        if (several) {
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (sr[16 * j + 4 * g4 + e] != rt) x[j][e] = 0.0f;
        }
        if (tid < Q) a.factors[image * kFactors * Q + 3 * Q + tid] = static_cast<float>(sr[tid]) + (sbad ? kNotFinite : 0.0f);
        uint8_t* T = a.T + image * image_bytes<MM>(MM::TP);
        uint8_t* M = a.M + image * image_bytes<MM>(MM::TP);
        const auto put = [&](uint8_t* to, const auto& f) {
#pragma unroll
            for (int p = 0; p < MM::TP; ++p) {
                if constexpr (MM::TP == 1) *reinterpret_cast<f4*>(to + lane * 16) = f.v;
                else *reinterpret_cast<bf8*>(to + p * 1024 + lane * 16) = f.p[p];
            }
        };
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (i != w) continue;
#pragma unroll
            for (int kb = 0; kb <= 16 * i / MM::KB; ++kb) {
                put(T + frag_at<MM>(i, kb, false) * MM::TP * 1024, MM::template of_tiles<MM::TP>(x, kb));
                if (!BWD) put(M + frag_at<MM>(i, kb, false) * MM::TP * 1024, MM::template of_tiles<MM::TP>(md, kb));
            }
        }
        if constexpr (BWD) {  // T and M once more with rows s: their columns through LDS
            uint8_t* Tt = a.Tt + image * image_bytes<MM>(MM::TP);
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < RT; ++j) *reinterpret_cast<f4*>(&so[t * LD + 16 * j + 4 * g4]) = pass ? md[j] : x[j];
                __syncthreads();
#pragma unroll
                for (int kb = 0; kb < KT; ++kb) {
                    if ((kb + 1) * MM::KB <= 16 * w) continue;
                    float v[R];
#pragma unroll
                    for (int m = 0; m < R; ++m) v[m] = so[(MM::KB * kb + (m >> 2) * 16 + 4 * g4 + (m & 3)) * LD + t];
                    const auto f = MM::template parts<MM::TP>(v);
                    uint8_t* to = pass ? M : Tt;
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        if (i == w) put(to + frag_at<MM>(i, kb, true) * MM::TP * 1024, f);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// The walk: 16 channels of a head a wavefront, four such wavefronts a block, and a fifth that moves memory:
// the next chunk's K, Q, T, M, factors and values straight into the other half of LDS (one half only
// where dstate is over 128), and the last chunk's y out of it.  (Fetched by the four themselves, the
// loads' issue was a third of a chunk's time.)  A chunk's y goes into its values' place in LDS, which the fifth
// empties before the next values come; with one half, where LDS has room, into a place of its own.
// A block has all of a CU's LDS, so a SIMD has one of the four: the chain of a chunk's five products is what
// bounds the walk (matrix instructions busy 45 % of it, vector ones 47 %, splits and scalings; 4.0 to 5.0 us a
// chunk by the clock).  4 x 8192 x 32 heads x 128 x 128, bf16, 256 blocks of 128 chunks: 510 to 645 us.  As kSave
// 510 to 530, 29 % and 36 %: it moves 2.3 GB, half of them the states, at 4.4 TB/s.
// kSave: for the backward, the states and E in place of y.  kSpan: a segment from zero, and behind the
// channels the N unit rows without values; only the state after it.
// DIRECT: see DeltaArgs; without it tokens pass through registers
// (Registers for two blocks a CU where LDS has the place, dstate up to 64.)
// ---------------------------------------------------------------------------------------
enum { kOut, kSave, kSpan };
template <class MM, int NT, int MODE>
struct WalkLds {
    static constexpr int W = 16 * NT, HALVES = NT <= 8 ? 2 : 1;
    static constexpr int V = 0, K = V + staged_bytes<MM, 64>(), T = K + staged_bytes<MM, W>(), F = T + image_bytes<MM>(MM::TP),
                         Qq = F + 1024, M = Qq + (MODE != kOut ? 0 : staged_bytes<MM, W>()), HALF = M + (MODE != kOut ? 0 : image_bytes<MM>(MM::TP));
    // a chunk's y: in place of its values, or (one half) in two places of its own
    static constexpr int YB = MODE == kOut && HALVES == 1 ? MM::template tile_bytes<64>(MM::Q) : 0, BYTES = HALVES * HALF + 2 * YB;
};

template <class MM, int NT, int MODE, bool DIRECT>
__global__ __launch_bounds__(320, NT <= 4 && (MODE == kSpan || (MODE == kSave && DIRECT)) ? 3 : 1) void delta_walk_kernel(DeltaArgs a, DeltaSaved keep) {
    using S = typename MM::S;
    using O = WalkLds<MM, NT, MODE>;
    constexpr int Q = MM::Q, RT = Q / 16, KT = Q / MM::KB, W = 16 * NT, KN = W / MM::KB, TP = MM::TP, ES = sizeof(S);
    __shared__ __attribute__((aligned(1024))) uint8_t sm[O::BYTES];
    const int lane = threadIdx.x & 63, li = lane & 15, g4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int H = static_cast<int>(a.H), P = static_cast<int>(a.P), N = static_cast<int>(a.N);
    const int pblocks = (P + 63) / 64, all = pblocks + (MODE == kSpan ? (N + 63) / 64 : 0), segs = static_cast<int>(a.segs);
    const int unit = xcd_order(blockIdx.x, gridDim.x);
    const int pb = unit % all, seg = unit / all % segs, bh = unit / all / segs, h = bh % H, b = bh / H;
    const int g = h / (H / static_cast<int>(a.G));
    const bool rows = MODE == kSpan && pb >= pblocks;  // unit rows
    const int chunks = static_cast<int>(a.chunks), c0 = seg * static_cast<int>(a.seg_chunks);
    const int c1 = c0 + static_cast<int>(a.seg_chunks) < chunks ? c0 + static_cast<int>(a.seg_chunks) : chunks;
    const auto rows_of = [&](int c) {
        const int64_t left = a.L - static_cast<int64_t>(c) * Q;
        return static_cast<int>(left < Q ? left : Q);
    };
    const auto half_of = [&](int c) { return sm + (O::HALVES == 2 ? (c & 1) * O::HALF : 0); };
    const auto y_of = [&](int c) { return O::YB ? sm + O::HALF + (c & 1) * O::YB : half_of(c) + O::V; };
    // what the chunk's last token says: sequences begun, and whether all keys and queries are finite
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
                if (MODE == kOut) direct_rows<MM, W, true>(half + O::Qq, token_buffer<S>(a.q, t0, a.q_row, g * N, valid, N), static_cast<int>(a.q_row), N, lane);
            } else {
                stage_rows<MM, W, 64, true>(half + O::K, static_cast<const S*>(a.k) + t0 * a.k_row + g * N, a.k_row, valid, N);
                if (MODE == kOut) stage_rows<MM, W, 64, true>(half + O::Qq, static_cast<const S*>(a.q) + t0 * a.q_row + g * N, a.q_row, valid, N);
            }
            direct_image<image_bytes<MM>(TP)>(half + O::T, a.T + image * image_bytes<MM>(TP), lane);
            if (MODE == kOut) direct_image<image_bytes<MM>(TP)>(half + O::M, a.M + image * image_bytes<MM>(TP), lane);
            direct_image<kFactors * Q * 4>(half + O::F, reinterpret_cast<const uint8_t*>(a.factors + image * kFactors * Q), lane);
        };
        const auto fetch_values = [&](int c) {
            uint8_t* const half = half_of(c);
            const int64_t t0 = b * a.L + static_cast<int64_t>(c) * Q;
            const int valid = rows_of(c);
            if (rows) return;
            if (DIRECT) direct_rows<MM, 64, false>(half + O::V, token_buffer<S>(a.v, t0, a.v_row, col, valid, width), static_cast<int>(a.v_row), width, lane);
            else stage_elements<MM, 64>(half + O::V, static_cast<const S*>(a.v) + t0 * a.v_row + col, a.v_row, valid, width);
        };
        const auto store = [&](int c) {
            if (MODE != kOut || c < c0) return;
            const uint8_t* y = y_of(c);
            const int64_t t0 = b * a.L + static_cast<int64_t>(c) * Q;
            const int valid = rows_of(c);
            if (DIRECT) {
                constexpr int PIECES = 64 * ES / 16;
                const Buffer r = token_buffer<S>(a.y, t0, a.y_row, col, valid, width);
#pragma unroll
                for (int i = 0; i < Q * PIECES / 64; ++i) {
                    const int t = (64 * i + lane) / PIECES, q = lane % PIECES, n = q * (16 / ES);
                    __builtin_amdgcn_raw_buffer_store_b128(lds<u4>(y + MM::template piece_at<64>(t, q)), r,
                                                           n < width ? (t * static_cast<int>(a.y_row) + n) * ES : kOutside, 0, 0);
                }
            } else {
                for (int i = lane; i < valid * 64; i += 64)
                    if (lane < width)
                        MM::store(static_cast<S*>(a.y) + (t0 + i / 64) * a.y_row + col, lane, MM::template at<64>(y, i / 64, lane));
            }
        };
        if (O::HALVES == 2) {
            fetch(c0);
            fetch_values(c0);
        }
        for (int c = c0; c < c1; ++c) {
            if (O::HALVES == 1) {
                __syncthreads();
                fetch(c);
                fetch_values(c);
            }
            wait_loads();
            __syncthreads();
            if (O::HALVES == 2 && c + 1 < c1) fetch(c + 1);
            store(c - 1);
            if (O::HALVES == 2 && c + 1 < c1) {
                wait_lds();  // y leaves before the next values come into its place
                fetch_values(c + 1);
            }
            if (marks_of(half_of(c)) >= static_cast<int>(kNotFinite)) {
                __syncthreads();
                __syncthreads();
            }
        }
        __syncthreads();
        store(c1 - 1);
        return;
    }

    const int p0 = 64 * (rows ? pb - pblocks : pb) + 16 * w, p = p0 + li, most = rows ? N : P;
    const bool mine = p0 < most, have = p < most;
    const int64_t bhs = static_cast<int64_t>(bh) * segs + seg;
    const float* const from = MODE == kSpan ? nullptr : segs > 1 ? a.entry + (bhs * P + p) * N : a.h0 ? a.h0 + (static_cast<int64_t>(bh) * P + p) * N : nullptr;
    float* const to = MODE == kSpan ? (rows ? a.phi + (bhs * N + p) * N : a.gain + (bhs * P + p) * N)
                      : MODE == kOut && a.final_state && seg == segs - 1 ? a.final_state + (static_cast<int64_t>(bh) * P + p) * N : nullptr;
    const uint32_t eat = have ? 4 * g4 * static_cast<uint32_t>(H * P) * 4 + p * 4 : kOutside;
    f4 hs[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = MM::state_row(i, g4);
        hs[i] = have && n < N && from ? *reinterpret_cast<const f4*>(from + n) : f4{0, 0, 0, 0};
        if (rows) {
#pragma unroll
            for (int e = 0; e < 4; ++e) hs[i][e] = n + e == p ? 1.0f : 0.0f;
        }
    }
    int power = 0;
    for (int c = c0; c < c1; ++c) {
        const int64_t t0 = b * a.L + static_cast<int64_t>(c) * Q;
        const int valid = rows_of(c);
        uint8_t* const half = half_of(c);
        if (O::HALVES == 1) __syncthreads();
        __syncthreads();
        uint8_t* const sk = half + O::K;
        const float* const sf = reinterpret_cast<const float*>(half + O::F);
        if (MODE == kSave && have) {
            float* to = keep.states + (static_cast<int64_t>(bh) * chunks + c) * P * N + static_cast<int64_t>(p) * N;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int n = MM::state_row(i, g4);
                if (n < N) *reinterpret_cast<f4*>(to + n) = hs[i];
            }
        }
        const int marks = marks_of(half);
        const bool clean = marks < static_cast<int>(kNotFinite);
        if (clean && !mine) continue;
        // straight on without branches, or with what chunks with starts need
        const auto chunk = [&](auto with_starts) __attribute__((always_inline)) {
            constexpr bool STARTS = decltype(with_starts)::value;
            f4 z[RT], y[RT], x[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) z[i] = y[i] = x[i] = f4{0, 0, 0, 0};
            // K h^T and Q h^T
#pragma unroll
            for (int kk = 0; kk < KN; ++kk) {
                const auto s = MM::template of_state<3>(hs, kk, g4);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    MM::template mac<1, 3>(z[i], MM::template state_rows<W>(sk, 16 * i, kk, li, g4), s);
                    if (MODE == kOut) MM::template mac<1, 3>(y[i], MM::template state_rows<W>(half + O::Qq, 16 * i, kk, li, g4), s);
                }
            }
            // Z = V - e^G K h^T, E = T Z
            scale_rows<STARTS>(z, sf, 1.0f, g4);
            if (MODE == kOut) scale_rows<STARTS>(y, sf, a.scale, g4);
#pragma unroll
            for (int i = 0; i < RT; ++i) z[i] = (rows ? f4{0, 0, 0, 0} : MM::template four_rows<64>(half + O::V, 16 * i, w, li, g4)) - z[i];
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const auto s = finite_tiles<MM, 3, STARTS>(z, kk);
#pragma unroll
                for (int i = kk * MM::KB / 16; i < RT; ++i)
                    MM::template mac<TP, 3>(x[i], frag<MM, TP>(half + O::T, frag_at<MM>(i, kk, false), lane), s);
            }
            mark_sequences<STARTS, Q>(x, z, sf + 3 * Q, lane);
            if (MODE == kSave) {
                const Buffer r = token_buffer<float>(keep.e, t0, static_cast<int64_t>(H) * P, static_cast<int64_t>(h) * P, DIRECT ? valid : 1, P);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 16 * i + 4 * g4 + e;
                        if (DIRECT) store_at<float>(r, eat + (16 * i + e) * static_cast<uint32_t>(H * P) * 4, x[i][e]);
                        else if (have && t < valid) keep.e[((t0 + t) * H + h) * P + p] = x[i][e];
                    }
            }
            // U = b E, Y += M U
            scale_rows<false>(x, sf + 2 * Q, 1.0f, g4);
            if (MODE == kOut) {
#pragma unroll
                for (int kk = 0; kk < KT; ++kk) {
                    const auto s = finite_tiles<MM, TP, STARTS>(x, kk);
#pragma unroll
                    for (int i = kk * MM::KB / 16; i < RT; ++i)
                        MM::template mac<TP, TP>(y[i], frag<MM, TP>(half + O::M, frag_at<MM>(i, kk, false), lane), s);
                }
                mark_sequences<STARTS, Q>(y, x, sf + 3 * Q, lane);
                uint8_t* const to = y_of(c);  // (this wavefront's columns, whose values it has read)
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) MM::template put<64>(to, 16 * i + 4 * g4 + e, 16 * w + li, y[i][e]);
            }
            // the state after the chunk
            if (STARTS && !clean) {
                __syncthreads();
                clear_rows<MM, W>(sk, sf + Q);
                __syncthreads();
            }
            scale_state<STARTS>(hs, sf[Q - 1]);
            scale_rows<STARTS>(x, sf + Q, 1.0f, g4);
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const auto s = MM::template of_tiles<3>(x, kk);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    MM::template mac<1, 3>(hs[i], MM::template state_columns<W>(sk, kk * MM::KB, i, li, g4), s);
            }
        };
        if (marks != 0) chunk(std::true_type{});
        else chunk(std::false_type{});
        if (MODE == kSpan && rows) keep_in_range(hs, power);
    }
    __syncthreads();
    if (MODE == kSpan && rows && have && g4 == 0) a.power[bhs * N + p] = power;
    if (to && have) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = MM::state_row(i, g4);
            if (n < N) *reinterpret_cast<f4*>(to + n) = hs[i];
        }
    }
}

// ---------------------------------------------------------------------------------------
// The states before the segments, h = h phi + gain from the first on (BACK: the gradients after them,
// g = g phi^T + gain from the last on), with the powers of phi's rows m put to h (BACK: to the product): 16 channels of a head a block, a wavefront 16 columns a
// product of the fp32 instruction, the next segments' phi and gain loaded meanwhile.
// 2.1 us a segment at dstate 128, 1.1 at 64 (one segment's loads ahead, and the starts read by the way: twice that).
// ---------------------------------------------------------------------------------------
template <int Q, int NT, bool BACK>
__global__ __launch_bounds__(64 * NT) void delta_join_states_kernel(DeltaArgs a) {
    constexpr int LD = 16 * NT + 4, AHEAD = NT < 16 ? 2 : 1;  // segments whose phi and gain are on their way (registers)
    __shared__ __attribute__((aligned(16))) float sh[16 * LD];
    __shared__ bool cut[64];
    const int lane = threadIdx.x & 63, li = lane & 15, g4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int P = static_cast<int>(a.P), N = static_cast<int>(a.N), segs = static_cast<int>(a.segs);
    const int ptiles = (P + 15) / 16, p0 = blockIdx.x % ptiles * 16 + 4 * g4, n = 16 * w + li;  // rows p0 .., column n
    const int64_t bh = blockIdx.x / ptiles;
    const float* const first = BACK ? a.dhT : a.h0;
    const int s0 = BACK ? segs - 1 : 0, step = BACK ? -1 : 1;
    f4 h{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (first && p0 + e < P && n < N) h[e] = first[(bh * P + p0 + e) * N + n];
    // with a start in a segment nothing of the state before it is left, finite or not
    for (int s = threadIdx.x; s < segs; s += 64 * NT) cut[s] = false;
    __syncthreads();
    for (int c = threadIdx.x; c < static_cast<int>(a.chunks); c += 64 * NT)
        if (a.factors[((bh * a.chunks + c) * kFactors + 4) * Q - 1] != 0.0f) cut[c / static_cast<int>(a.seg_chunks)] = true;
    f4 phi[AHEAD][NT], gain[AHEAD];
    int power[AHEAD];  // of row n
    const auto load = [&](int i, f4 (&ph)[NT], f4& gn, int& pw) {
        if (i + 1 >= segs) return;
        const int64_t at = bh * segs + s0 + step * i;
        const Buffer r = buffer(a.phi + at * N * N, static_cast<int64_t>(N) * N * 4);
        const Buffer rg = buffer(a.gain + at * P * N, static_cast<int64_t>(P) * N * 4);
        pw = __builtin_amdgcn_raw_buffer_load_b32(buffer(a.power + at * N, N * 4), 4 * n, 0, 0);
#pragma unroll
        for (int kk = 0; kk < NT; ++kk) {
            const int m = 16 * kk + 4 * g4;
            if (BACK) {
                ph[kk] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, n < N && m < N ? (n * N + m) * 4 : kOutside, 0, 0));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) ph[kk][e] = load_at<float>(r, n < N ? ((m + e) * N + n) * 4 : kOutside);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) gn[e] = load_at<float>(rg, n < N ? ((p0 + e) * N + n) * 4 : kOutside);
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) load(d, phi[d], gain[d], power[d]);
    for (int i0 = 0; i0 < segs; i0 += AHEAD) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            const int i = i0 + d, s = s0 + step * i;
            if (i >= segs) continue;
            __syncthreads();
            float* const entry = a.entry + (bh * segs + s) * P * N;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sh[(4 * g4 + e) * LD + n] = BACK || i + 1 == segs ? h[e] : __builtin_ldexpf(h[e], power[d]);
                if (p0 + e < P && n < N) entry[static_cast<int64_t>(p0 + e) * N + n] = h[e];
            }
            __syncthreads();
            if (i + 1 == segs) continue;
            f4 sum{0, 0, 0, 0};
#pragma unroll
            for (int kk = 0; kk < NT; ++kk) {
                const f4 l = *reinterpret_cast<const f4*>(&sh[li * LD + 16 * kk + 4 * g4]);
                ByF32::mac<1, 1>(sum, ByF32::Frag<1>{l}, ByF32::Frag<1>{phi[d][kk]});
            }
            if (BACK) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = __builtin_ldexpf(sum[e], power[d]);
            }
            h = cut[s] ? gain[d] : sum + gain[d];
            load(i + AHEAD, phi[d], gain[d], power[d]);
        }
    }
}

// ---------------------------------------------------------------------------------------
// Token by token: the decode step.  Eight lanes hold a channel's state, 128 bytes side by side
// of it a load, RG channels eight apart a lane; a wavefront is a unit of its own.  The state's
// one read and one write are the whole cost (256 requests of 32 heads x 128 x 128: 1.07 GB in 199 us,
// 5.4 TB/s).
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
    const int64_t unit = long_block() * 4 + (threadIdx.x >> 6);
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
            if (n < N && p0 + 8 * r < a.P)
                hs[r][i] = __builtin_nontemporal_load(
                    reinterpret_cast<const f4*>(s.state + ((slot * a.H + h) * a.P + p0 + 8 * r) * a.N + n));
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
        const float f = a.gate ? exp_of(gate_of(a.gate[row * a.H + h])) : 1.0f;
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            float kh = 0.0f, y = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hs[r][i][e] *= f;
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
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = 32 * i + 4 * l8;
            if (n < N && p0 + 8 * r < a.P)
                __builtin_nontemporal_store(
                    hs[r][i], reinterpret_cast<f4*>(s.state + ((slot * a.H + h) * a.P + p0 + 8 * r) * a.N + n));
        }
}

template <class D, int NI, int RG>
hipError_t step_of(const DeltaStep& s, hipStream_t stream) {
    const int64_t units = s.a.B * s.a.H * ((s.a.P + 8 * RG - 1) / (8 * RG));
    delta_step_kernel<D, NI, RG><<<long_grid((units + 3) / 4), 256, 0, stream>>>(s, units);
    return hipGetLastError();
}
template <class D>
hipError_t step_by_width(const DeltaStep& s, hipStream_t stream) {
    if (s.a.N <= 32) return step_of<D, 1, 4>(s, stream);
    if (s.a.N <= 64) return step_of<D, 2, 4>(s, stream);
    if (s.a.N <= 128) return step_of<D, 4, 4>(s, stream);
    return step_of<D, 8, 2>(s, stream);
}

// a key head's heads share the products of prep: up to one a wavefront, as long as the blocks fill the GPU (fewer:
// 1024 tokens of 32 heads of 8 x 128 x 128 forward 77 us, 69 with a head a block)
template <class MM>
int prep_heads(const DeltaArgs& a) {
    int heads = 1;
    while (2 * heads <= MM::Q / 16 && a.H / a.G % (2 * heads) == 0 && a.B * a.chunks * a.H / (2 * heads) >= 1024) heads *= 2;
    return heads;
}
template <class MM, int NT>
void prep_of(const DeltaArgs& a, bool bwd, hipStream_t stream) {
    const int heads = prep_heads<MM>(a);
    const unsigned blocks = static_cast<unsigned>(a.B * a.chunks * (a.H / heads));
    if (bwd && a.direct) delta_prep_kernel<MM, NT, true, true><<<blocks, MM::Q * 4, 0, stream>>>(a, heads);
    else if (bwd) delta_prep_kernel<MM, NT, true, false><<<blocks, MM::Q * 4, 0, stream>>>(a, heads);
    else if (a.direct) delta_prep_kernel<MM, NT, false, true><<<blocks, MM::Q * 4, 0, stream>>>(a, heads);
    else delta_prep_kernel<MM, NT, false, false><<<blocks, MM::Q * 4, 0, stream>>>(a, heads);
}
template <class MM, int NT, int MODE>
hipError_t walk_of(const DeltaArgs& a, const DeltaSaved& keep, hipStream_t stream) {
    const int64_t all = (a.P + 63) / 64 + (MODE == kSpan ? (a.N + 63) / 64 : 0);
    const unsigned blocks = static_cast<unsigned>(a.B * a.H * a.segs * all);
    if (a.direct) delta_walk_kernel<MM, NT, MODE, true><<<blocks, 320, 0, stream>>>(a, keep);
    else delta_walk_kernel<MM, NT, MODE, false><<<blocks, 320, 0, stream>>>(a, keep);
    return hipGetLastError();
}
template <class MM, int NT, bool BACK>
hipError_t join_of(const DeltaArgs& a, hipStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(a.B * a.H * ((a.P + 15) / 16));
    delta_join_states_kernel<MM::Q, NT, BACK><<<blocks, 64 * NT, 0, stream>>>(a);
    return hipGetLastError();
}
template <class MM>
hipError_t join_back(const DeltaArgs& a, hipStream_t stream) {
    if (a.N <= 64) return join_of<MM, 4, true>(a, stream);
    if (a.N <= 128) return join_of<MM, 8, true>(a, stream);
    return join_of<MM, 16, true>(a, stream);
}
template <class MM, int NT, bool SAVE>
hipError_t rows_of_width(const DeltaArgs& a, const DeltaSaved& keep, hipStream_t stream) {
    prep_of<MM, NT>(a, SAVE, stream);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.segs > 1) e = walk_of<MM, NT, kSpan>(a, keep, stream);
    if (e == hipSuccess && a.segs > 1) e = join_of<MM, NT, false>(a, stream);
    if (e == hipSuccess) e = walk_of<MM, NT, SAVE ? kSave : kOut>(a, keep, stream);
    return e;
}
template <class MM, bool SAVE>
hipError_t walk_by_width(const DeltaArgs& a, const DeltaSaved& keep, hipStream_t stream) {
    if (a.N <= 64) return rows_of_width<MM, 4, SAVE>(a, keep, stream);
    if (a.N <= 128) return rows_of_width<MM, 8, SAVE>(a, keep, stream);
    return rows_of_width<MM, 16, SAVE>(a, keep, stream);
}
template <class MM>
hipError_t fwd_of(DeltaArgs a, void* workspace, hipStream_t stream) {
    place_chunks<MM>(a, static_cast<uint8_t*>(workspace), false);
    constexpr size_t es = sizeof(typename MM::S);
    const int64_t keys = a.G * a.N, values = a.H * a.P;
    a.direct = a.N % (16 / es) == 0 && a.P % (16 / es) == 0 && direct_rows_fit(a.q, a.q_row, keys, es) &&
               direct_rows_fit(a.k, a.k_row, keys, es) && direct_rows_fit(a.v, a.v_row, values, es) &&
               direct_rows_fit(a.y, a.y_row, values, es);
    return walk_by_width<MM, false>(a, DeltaSaved{}, stream);
}

// whether each launch has less than 2^32 threads
template <class MM>
bool launches_fit(DeltaArgs a, bool bwd) {
    place_chunks<MM>(a, nullptr, bwd);
    const int64_t most = int64_t{1} << 32, walk = (a.P + 63) / 64 + (a.segs > 1 ? (a.N + 63) / 64 : 0);
    return a.B * a.chunks * (a.H / prep_heads<MM>(a)) < most / (MM::Q * 4) && a.B * a.H * a.segs * walk < most / 320 &&
           (!bwd || a.B * a.chunks * a.G < most / 512);
}

}  // namespace

bool delta_launches_fit(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype, bool bwd) {
    DeltaArgs a{};
    a.B = B;
    a.L = L;
    a.H = H;
    a.P = P;
    a.G = G;
    a.N = N;
    return dtype == SSM_BF16 ? launches_fit<ByBf16>(a, bwd) : launches_fit<ByF32>(a, bwd);
}

hipError_t launch_delta_walk_saved(const DeltaArgs& a, const DeltaSaved& s, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? walk_by_width<ByBf16, true>(a, s, stream) : walk_by_width<ByF32, true>(a, s, stream);
}

hipError_t launch_delta_join_back(const DeltaArgs& a, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? join_back<ByBf16>(a, stream) : join_back<ByF32>(a, stream);
}

size_t delta_fwd_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, ssm_dtype_t dtype) {
    DeltaArgs a{};
    a.B = B;
    a.L = L;
    a.H = H;
    a.P = P;
    a.G = G;
    a.N = N;
    return dtype == SSM_BF16 ? place_chunks<ByBf16>(a, nullptr, false) : place_chunks<ByF32>(a, nullptr, false);
}

hipError_t launch_delta_fwd(DeltaArgs a, void* workspace, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? fwd_of<ByBf16>(a, workspace, stream) : fwd_of<ByF32>(a, workspace, stream);
}

hipError_t launch_delta_step(const DeltaStep& s, ssm_dtype_t dtype, hipStream_t stream) {
    return dtype == SSM_BF16 ? step_by_width<BF16>(s, stream) : step_by_width<F32>(s, stream);
}

}  // namespace ssm
