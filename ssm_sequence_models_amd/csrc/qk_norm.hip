// qk_norm.hip -- the norm of every head of the queries and keys, with the rotation of its first R
// channels by the token's position, in one pass over both; and its backward.
//
//     r = (sum x^2 + eps)^-1/2 (l2) or (mean x^2 + eps)^-1/2 (rms),  n = r x,  m = w n
//     y = m with the pairs (i, i + R/2), or (2i, 2i + 1) interleaved, turned by pos * inv_freq_i
// backward: d = dy turned back, dw = sum of d n over tokens and heads,
//     dx = r (w d - n c),  c = sum of w d n (l2) or their mean (rms)
//
// Bound by memory: q and k are read and written once.  A head takes the lanes of one wavefront
// that hold its channels in 16-byte pieces; the partners of a pair that lie in another lane's
// piece are read again (from L1) instead of exchanged, which works for any R.  The angles are per
// token: a block takes a few tokens with all their heads and forms the sines and cosines once.
// An angle is a product in double, its whole turns taken off there: positions of any int32 size
// keep the accuracy of position 0.
//
// 4 x 8192 tokens x 32 heads x 128 bf16, rotation 64, weights: forward 105 us (0.54 GB, 5.1 TB/s), backward 153 to
// 158 + 5 (0.81 GB, 5.2 TB/s).  Without the rotation's layout as a template and the next head's loads in flight these
// were 177 and 231.  In fp32, 128 channels: 213 and 315 (5.0 and 5.1 TB/s).  Layouts of the rotation outside whole
// pieces go channel by channel: 16 + 16 heads x 80, rotation 40, bf16 322 us and 417 (1.0 and 1.2 TB/s).  Up to 8 tokens a block (16: no gain; streaming stores: none either).
#include "internal.h"

namespace ssm {
namespace {

typedef uint32_t u4e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4e4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kThreads = 256;
constexpr int kMostTokens = 8;  // a block

// V channels of a head in one 16-byte piece
template <class D>
struct Piece;
template <>
struct Piece<BF16> {
    static constexpr int V = 8;
    __device__ __forceinline__ static u32x4_t raw(const uint16_t* p) { return *reinterpret_cast<const u4e2*>(p); }
    __device__ __forceinline__ static u32x4_t pack(const float (&v)[8]) {  // of values that are bf16
        return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
    __device__ __forceinline__ static void values(u32x4_t x, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(j & 1 ? x[j >> 1] & 0xFFFF0000u : x[j >> 1] << 16);
    }
    __device__ __forceinline__ static void store(uint16_t* p, const float (&v)[8]) {
        *reinterpret_cast<u4e2*>(p) = pack(v);
    }
};
template <>
struct Piece<F32> {
    static constexpr int V = 4;
    __device__ __forceinline__ static u32x4_t raw(const float* p) { return *reinterpret_cast<const u4e4*>(p); }
    __device__ __forceinline__ static u32x4_t pack(const float (&v)[4]) {
        return u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
    __device__ __forceinline__ static void values(u32x4_t x, float (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(x[j]);
    }
    __device__ __forceinline__ static void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<u4e4*>(p) = pack(v);
    }
};

// How a call's heads lie in pieces: whole ones without rotation, with the partners of a piece in a piece
// of their own (kHalves) or beside each other in it (kInterleaved), or any channels (kAny).
enum { kPlain, kHalves, kInterleaved, kAny };

// a lane's piece of a head: channels i0 .. i0 + have, and how it takes part in the rotation
template <class D, int ROT>
struct Lane {
    static constexpr int V = Piece<D>::V;
    using T = typename D::T;
    using Raw = decltype(Piece<D>::raw(nullptr));
    int i0, have, R;
    bool turned, interleaved;

    __device__ __forceinline__ Lane(const QkNormCall& c, int l) {
        i0 = l * V;
        const int left = static_cast<int>(c.D) - i0;
        have = left < 0 ? 0 : left < V ? left : V;
        R = static_cast<int>(c.R);
        interleaved = c.interleaved;
        turned = ROT != kPlain && have > 0 && i0 < R;
    }
    __device__ __forceinline__ int partner(int i) const {
        return i >= R ? i : interleaved ? i ^ 1 : i < R / 2 ? i + R / 2 : i - R / 2;
    }
    __device__ __forceinline__ bool first(int i) const { return interleaved ? !(i & 1) : i < R / 2; }
    __device__ __forceinline__ int pair(int i) const { return interleaved ? i >> 1 : i < R / 2 ? i : i - R / 2; }

    // a head's piece, and its partners', as loads in flight (kAny: values)
    __device__ __forceinline__ Raw load(const T* p) const {
        if constexpr (ROT != kAny) {
            return have ? Piece<D>::raw(p + i0) : Raw{};
        } else {
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = j < have ? D::load(p, i0 + j) : 0.0f;
            return Piece<D>::pack(v);
        }
    }
    __device__ __forceinline__ Raw load_partners(const T* p, Raw own) const {
        if constexpr (ROT == kHalves) {
            return turned ? Piece<D>::raw(p + (i0 < R / 2 ? i0 + R / 2 : i0 - R / 2)) : Raw{};
        } else if constexpr (ROT == kAny) {
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = j < have ? D::load(p, partner(i0 + j)) : 0.0f;
            return Piece<D>::pack(v);
        } else {
            return own;
        }
    }
    __device__ __forceinline__ void partners(Raw r, float (&v)[V]) const {
        float u[V];
        Piece<D>::values(r, u);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = ROT == kInterleaved ? u[j ^ 1] : u[j];
    }
    __device__ __forceinline__ void store(T* p, const float (&v)[V]) const {
        if (have == V) {
            Piece<D>::store(p + i0, v);
        } else if (ROT == kAny) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < have) D::store(p, i0 + j, v[j]);
        }
    }
    __device__ __forceinline__ static void floats(const float* p, float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const u4e4 x = *reinterpret_cast<const u4e4*>(p + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(x[j]);
        }
    }
    __device__ __forceinline__ void weights(const float* w, float (&own)[V], float (&other)[V]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) own[j] = other[j] = 1.0f;
        if (!w) return;
        if constexpr (ROT == kAny) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                own[j] = j < have ? w[i0 + j] : 1.0f;
                other[j] = j < have ? w[partner(i0 + j)] : 1.0f;
            }
        } else {  // lanes behind the head read its first piece
            floats(w + (have ? i0 : 0), own);
            if constexpr (ROT == kHalves) {
                floats(w + (turned ? partner(i0) : 0), other);
            } else if constexpr (ROT == kInterleaved) {
#pragma unroll
                for (int j = 0; j < V; ++j) other[j] = own[j ^ 1];
            }
        }
    }
    // v turned by the token's angles (dir 1) or back (dir -1); `other` holds the partners
    __device__ __forceinline__ void turn(const float2* cs, float dir, float (&v)[V], const float (&other)[V]) const {
        if constexpr (ROT == kInterleaved) {
            const float2* a = cs + i0 / 2;
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = v[j] * a[j / 2].x + other[j] * (j & 1 ? dir : -dir) * a[j / 2].y;
        } else if constexpr (ROT == kHalves) {
            const float2* a = cs + (i0 < R / 2 ? i0 : i0 - R / 2);
            const float sign = i0 < R / 2 ? -dir : dir;
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = v[j] * a[j].x + other[j] * sign * a[j].y;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int i = i0 + j;
                if (i >= R) continue;
                const float2 a = cs[pair(i)];
                v[j] = v[j] * a.x + other[j] * (first(i) ? -dir : dir) * a.y;
            }
        }
    }
};

// the next head of a block's tokens that a head's lanes take
__device__ __forceinline__ void next_head(int& token, int& head, int heads, int tokens_on, int heads_on) {
    token += tokens_on;
    head += heads_on;
    if (head >= heads) {
        head -= heads;
        ++token;
    }
}

template <int LPH>
__device__ __forceinline__ float sum_lanes(float v) {  // over a head's lanes
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// cosines and sines of `tokens` tokens from `first` on
__device__ __forceinline__ void angles(const QkNormCall& c, float2* cs, int64_t first, int tokens) {
    const int half = static_cast<int>(c.R / 2);
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int64_t t = first + i / half;
        const double pos = c.positions ? c.positions[t] : static_cast<int32_t>(t % c.L);
        const double turns = pos * static_cast<double>(c.inv_freq[i % half]) * 0.15915494309189534;  // 1 / 2 pi
        const double part = 2.0 * (turns - rint(turns));  // in half turns
        const float hi = static_cast<float>(part), lo = static_cast<float>(part - hi) * 3.14159265f;
        float s, k;
        sincospif(hi, &s, &k);
        cs[i] = float2{k - lo * s, s + lo * k};
    }
}

// A head's 1 / norm (0 for a head of zeros without eps).  Where the squares leave fp32's range, or come near its
// ends, the values and the norm are taken in units of 2^up instead of 1: v is divided by it, and what is formed of
// 1 / norm without v is to be.
template <int LPH, int V>
__device__ __forceinline__ float inverse(float (&v)[V], const QkNormCall& c, int& up) {
    const float per = c.l2 ? 1.0f : 1.0f / static_cast<float>(c.D);
    const auto squares = [&] {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += v[j] * v[j];
        return sum_lanes<LPH>(sum) * per;
    };
    float s = squares() + c.eps;
    up = 0;
    if (__float_as_uint(s) - 0x17800000u > 0x38800000u) {  // not within 2^-80 .. 2^80, for a head's lanes alike
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) most = fmaxf(most, fabsf(v[j]));
#pragma unroll
        for (int d = 1; d < LPH; d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
        if (s != s) return s;  // NaN stays one
        if (s == 0.0f && most == 0.0f) return 0.0f;
        if (most < __builtin_inff() && c.eps < __builtin_inff()) {
            const int of_eps = c.eps > 0.0f ? (__builtin_amdgcn_frexp_expf(c.eps) >> 1) + 1 : -1000;
            up = max(most > 0.0f ? __builtin_amdgcn_frexp_expf(most) : -1000, of_eps);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = __builtin_ldexpf(v[j], -up);
            s = squares() + __builtin_ldexpf(c.eps, -2 * up);
        }
    }
    return 1.0f / sqrtf(s);
}

// The next head's loads are in flight while one is computed.
template <class D, int LPH, int ROT>
__global__ __launch_bounds__(kThreads) void qk_norm_fwd_kernel(QkNormCall c, int tokens) {
    using T = typename D::T;
    using L = Lane<D, ROT>;
    constexpr int V = L::V;
    __shared__ __attribute__((aligned(16))) float2 cs[kMostTokens * 128];
    const int64_t first = long_block() * tokens;
    if (first >= c.tokens) return;
    if (c.tokens - first < tokens) tokens = static_cast<int>(c.tokens - first);
    if (c.R) {
        angles(c, cs, first, tokens);
        __syncthreads();
    }
    const L lane(c, threadIdx.x % LPH);
    const int half = static_cast<int>(c.R / 2), D_ = static_cast<int>(c.D);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int heads = static_cast<int>(c.heads[side]);
        const T* const xs = static_cast<const T*>(c.x[side]) + first * c.x_row[side];
        T* const outs = static_cast<T*>(c.out[side]) + first * c.out_row[side];
        float w[V], wo[V];
        lane.weights(c.w[side], w, wo);
        int token = threadIdx.x / LPH / heads, head = threadIdx.x / LPH % heads;
        const int tokens_on = kThreads / LPH / heads, heads_on = kThreads / LPH % heads;
        typename L::Raw x{}, o{};
        const auto load = [&] {
            if (token >= tokens) return;
            const T* p = xs + token * c.x_row[side] + head * D_;
            x = lane.load(p);
            o = lane.load_partners(p, x);
        };
        load();
        while (token < tokens) {
            const int t = token, h = head;
            float v[V], u[V];
            Piece<D>::values(x, v);
            lane.partners(o, u);
            next_head(token, head, heads, tokens_on, heads_on);
            load();
            int up;
            const float r = inverse<LPH>(v, c, up);
            if (up != 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] = __builtin_ldexpf(u[j], -up);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= r * w[j];
            if (lane.turned) {
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] *= r * wo[j];
                lane.turn(cs + t * half, 1.0f, v, u);
            }
            lane.store(outs + t * c.out_row[side] + h * D_, v);
        }
    }
}

// Blocks walk over the tokens, queries first; the sums for dw stay in the lanes of their channels to the
// end, are added over a block's heads in LDS, and go out as a row a block (qk_norm_weights_kernel adds
// those).
template <class D, int LPH, int ROT>
__global__ __launch_bounds__(kThreads) void qk_norm_bwd_kernel(QkNormCall c, int most) {
    using T = typename D::T;
    using L = Lane<D, ROT>;
    constexpr int V = L::V, HEADS = kThreads / LPH;
    __shared__ __attribute__((aligned(16))) float2 cs[kMostTokens * 128];
    __shared__ float sums[HEADS][LPH * V];
    const L lane(c, threadIdx.x % LPH);
    const int half = static_cast<int>(c.R / 2), hd = threadIdx.x / LPH, D_ = static_cast<int>(c.D);
    const float per = c.l2 ? 1.0f : 1.0f / static_cast<float>(c.D);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int heads = static_cast<int>(side ? c.heads[1] : c.heads[0]);
        const int64_t x_row = side ? c.x_row[1] : c.x_row[0], dy_row = side ? c.dy_row[1] : c.dy_row[0],
                      out_row = side ? c.out_row[1] : c.out_row[0];
        const T* const xs = static_cast<const T*>(side ? c.x[1] : c.x[0]);
        const T* const dys = static_cast<const T*>(side ? c.dy[1] : c.dy[0]);
        T* const outs = static_cast<T*>(side ? c.out[1] : c.out[0]);
        float w[V], unused[V], dw[V];
        lane.weights(side ? c.w[1] : c.w[0], w, unused);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[j] = 0.0f;
        const int tokens_on = HEADS / heads, heads_on = HEADS % heads;
        for (int64_t first = static_cast<int64_t>(blockIdx.x) * most; first < c.tokens;
             first += static_cast<int64_t>(gridDim.x) * most) {
            const int tokens = c.tokens - first < most ? static_cast<int>(c.tokens - first) : most;
            int token = hd / heads, head = hd % heads;
            typename L::Raw x{}, y{}, o{};
            const auto load = [&] {
                if (token >= tokens) return;
                const T* p = dys + (first + token) * dy_row + head * D_;
                x = lane.load(xs + (first + token) * x_row + head * D_);
                y = lane.load(p);
                o = lane.load_partners(p, y);
            };
            load();
            if (c.R) {
                __syncthreads();
                angles(c, cs, first, tokens);
                __syncthreads();
            }
            while (token < tokens) {
                const int t = token, h = head;
                float v[V], d[V], u[V];
                Piece<D>::values(x, v);
                Piece<D>::values(y, d);
                lane.partners(o, u);
                next_head(token, head, heads, tokens_on, heads_on);
                load();
                if (lane.turned) lane.turn(cs + t * half, -1.0f, d, u);
                int up;
                const float r = inverse<LPH>(v, c, up);
                float dot = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] *= r;
                    dw[j] += d[j] * v[j];
                    d[j] *= w[j];
                    dot += d[j] * v[j];
                }
                dot = sum_lanes<LPH>(dot) * per;
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = r * (d[j] - v[j] * dot);
                if (up != 0) {
#pragma unroll
                    for (int j = 0; j < V; ++j) d[j] = __builtin_ldexpf(d[j], -up);
                }
                lane.store(outs + (first + t) * out_row + h * D_, d);
            }
        }
        if (!c.partial) continue;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) sums[hd][lane.i0 + j] = dw[j];
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < D_) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < HEADS; ++i) s += sums[i][threadIdx.x];
            c.partial[(static_cast<int64_t>(blockIdx.x) * 2 + side) * D_ + threadIdx.x] = s;
        }
    }
}

// a block a channel and side: the partial rows' sum in a fixed order
__global__ __launch_bounds__(kThreads) void qk_norm_weights_kernel(QkNormCall c, int rows) {
    __shared__ double sums[kThreads];
    const int side = blockIdx.x & 1, i = blockIdx.x >> 1, D_ = static_cast<int>(c.D);
    if (!c.dw[side]) return;
    double s = 0.0;
    for (int r = threadIdx.x; r < rows; r += kThreads) s += c.partial[(static_cast<int64_t>(r) * 2 + side) * D_ + i];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d >>= 1) {
        if (static_cast<int>(threadIdx.x) < d) sums[threadIdx.x] += sums[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) c.dw[side][i] = static_cast<float>(sums[0]);
}

// tokens a block at a time: enough blocks for every CU before a block takes more than one; backward
// few partial rows and one round of blocks (3 x 1027 tokens x 8 heads x 80: 19 us for one token at a
// time in three rounds)
int tokens_a_block(int64_t tokens, bool bwd) {
    const int64_t n = bwd ? (tokens + 1023) / 1024 : tokens / 2048;
    return n < 1 ? 1 : n > kMostTokens ? kMostTokens : static_cast<int>(n);
}

template <class D, int LPH, int ROT>
void run(const QkNormCall& c, bool bwd, hipStream_t s) {
    const int n = tokens_a_block(c.tokens, bwd);
    if (bwd) qk_norm_bwd_kernel<D, LPH, ROT><<<static_cast<unsigned>(qk_norm_partial_rows(c.tokens)), kThreads, 0, s>>>(c, n);
    else qk_norm_fwd_kernel<D, LPH, ROT><<<long_grid((c.tokens + n - 1) / n), kThreads, 0, s>>>(c, n);
}
template <class D, int LPH>
hipError_t by_rotation(const QkNormCall& c, bool bwd, hipStream_t s) {
    constexpr int V = Piece<D>::V;
    if (c.D % V != 0) run<D, LPH, kAny>(c, bwd, s);
    else if (c.R == 0) run<D, LPH, kPlain>(c, bwd, s);
    else if (c.interleaved && c.R % V == 0) run<D, LPH, kInterleaved>(c, bwd, s);
    else if (!c.interleaved && c.R % (2 * V) == 0) run<D, LPH, kHalves>(c, bwd, s);
    else run<D, LPH, kAny>(c, bwd, s);
    return hipGetLastError();
}
template <class D>
hipError_t by_width(const QkNormCall& c, bool bwd, hipStream_t s) {
    const int64_t pieces = (c.D + Piece<D>::V - 1) / Piece<D>::V;
    if (pieces <= 8) return by_rotation<D, 8>(c, bwd, s);
    if (pieces <= 16) return by_rotation<D, 16>(c, bwd, s);
    if (pieces <= 32 || Piece<D>::V == 8) return by_rotation<D, 32>(c, bwd, s);
    return by_rotation<F32, 64>(c, bwd, s);  // fp32 only: D is at most 256
}

}  // namespace

int64_t qk_norm_partial_rows(int64_t tokens) {
    const int64_t n = tokens_a_block(tokens, true), blocks = (tokens + n - 1) / n;
    return blocks < 1024 ? blocks : 1024;
}
hipError_t launch_qk_norm_fwd(const QkNormCall& c, hipStream_t s) {
    return c.dtype == SSM_BF16 ? by_width<BF16>(c, false, s) : by_width<F32>(c, false, s);
}
hipError_t launch_qk_norm_bwd(const QkNormCall& c, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (c.tokens > 0) e = c.dtype == SSM_BF16 ? by_width<BF16>(c, true, s) : by_width<F32>(c, true, s);
    if (e != hipSuccess || (!c.dw[0] && !c.dw[1])) return e;
    qk_norm_weights_kernel<<<static_cast<unsigned>(2 * c.D), kThreads, 0, s>>>(
        c, c.tokens > 0 ? static_cast<int>(qk_norm_partial_rows(c.tokens)) : 0);
    return hipGetLastError();
}

}  // namespace ssm
