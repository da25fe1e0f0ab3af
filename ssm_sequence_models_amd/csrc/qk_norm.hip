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
    __device__ __forceinline__ static void load(const uint16_t* p, float (&v)[8]) {
        const u4e2 x = *reinterpret_cast<const u4e2*>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(j & 1 ? x[j >> 1] & 0xFFFF0000u : x[j >> 1] << 16);
    }
    __device__ __forceinline__ static void store(uint16_t* p, const float (&v)[8]) {
        u4e2 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<u4e2*>(p) = x;
    }
};
template <>
struct Piece<F32> {
    static constexpr int V = 4;
    __device__ __forceinline__ static void load(const float* p, float (&v)[4]) {
        const u4e4 x = *reinterpret_cast<const u4e4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(x[j]);
    }
    __device__ __forceinline__ static void store(float* p, const float (&v)[4]) {
        u4e4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __float_as_uint(v[j]);
        *reinterpret_cast<u4e4*>(p) = x;
    }
};

// a lane's piece of a head: channels i0 .. i0 + V of D, and how it takes part in the rotation
template <class D>
struct Lane {
    static constexpr int V = Piece<D>::V;
    int i0, have;     // channels of the piece (V, fewer at the end of an odd D, 0 behind it)
    bool turned;      // some of them are rotated
    bool whole;       // partners are a piece of their own (or the same, interleaved)
    int R, interleaved;

    __device__ __forceinline__ Lane(const QkNormCall& c, int l) {
        i0 = l * V;
        const int left = static_cast<int>(c.D) - i0;
        have = left < 0 ? 0 : left < V ? left : V;
        R = static_cast<int>(c.R);
        interleaved = c.interleaved;
        turned = have > 0 && i0 < R;
        whole = have == V && R % (interleaved ? V : 2 * V) == 0;
    }
    __device__ __forceinline__ int partner(int i) const {
        return i >= R ? i : interleaved ? i ^ 1 : i < R / 2 ? i + R / 2 : i - R / 2;
    }
    __device__ __forceinline__ bool first(int i) const { return interleaved ? !(i & 1) : i < R / 2; }
    __device__ __forceinline__ int pair(int i) const { return interleaved ? i >> 1 : i < R / 2 ? i : i - R / 2; }

    __device__ __forceinline__ void load(const typename D::T* p, float (&v)[V]) const {
        if (have == V) {
            Piece<D>::load(p + i0, v);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = j < have ? D::load(p, i0 + j) : 0.0f;
        }
    }
    __device__ __forceinline__ void store(typename D::T* p, const float (&v)[V]) const {
        if (have == V) {
            Piece<D>::store(p + i0, v);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < have) D::store(p, i0 + j, v[j]);
        }
    }
    __device__ __forceinline__ void load_partners(const typename D::T* p, const float (&own)[V], float (&v)[V]) const {
        if (whole && interleaved) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = own[j ^ 1];
        } else if (whole) {
            Piece<D>::load(p + partner(i0), v);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = j < have ? D::load(p, partner(i0 + j)) : 0.0f;
        }
    }
    __device__ __forceinline__ void weights(const float* w, float (&own)[V], float (&other)[V]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            own[j] = w && j < have ? w[i0 + j] : 1.0f;
            other[j] = w && j < have ? w[partner(i0 + j)] : 1.0f;
        }
    }
    // v turned by the token's angles (dir 1) or back (dir -1); `other` holds the partners
    __device__ __forceinline__ void turn(const float2* cs, float dir, float (&v)[V], const float (&other)[V]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = i0 + j;
            if (i >= R) continue;
            const float2 a = cs[pair(i)];
            v[j] = v[j] * a.x + other[j] * (first(i) ? -dir : dir) * a.y;
        }
    }
};

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

// sum of squares -> 1 / norm; 0 for a head of zeros without eps
__device__ __forceinline__ float inverse(float squares, const QkNormCall& c) {
    const float v = squares * (c.l2 ? 1.0f : 1.0f / static_cast<float>(c.D)) + c.eps;
    return v > 0.0f ? 1.0f / sqrtf(v) : v == 0.0f ? 0.0f : v;  // NaN stays one
}

template <class D, int LPH>
__global__ __launch_bounds__(kThreads) void qk_norm_fwd_kernel(QkNormCall c, int tokens) {
    using T = typename D::T;
    constexpr int V = Piece<D>::V;
    __shared__ float2 cs[kMostTokens * 128];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
    if (c.tokens - first < tokens) tokens = static_cast<int>(c.tokens - first);
    if (c.R) {
        angles(c, cs, first, tokens);
        __syncthreads();
    }
    const Lane<D> lane(c, threadIdx.x % LPH);
    const int half = static_cast<int>(c.R / 2);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int heads = static_cast<int>(c.heads[side]);
        float w[V], wo[V];
        lane.weights(c.w[side], w, wo);
        for (int u = threadIdx.x / LPH; u < tokens * heads; u += kThreads / LPH) {
            const int token = u / heads, head = u % heads;
            const T* x = static_cast<const T*>(c.x[side]) + (first + token) * c.x_row[side] + head * c.D;
            float v[V], o[V];
            lane.load(x, v);
            if (lane.turned) lane.load_partners(x, v, o);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) sum += v[j] * v[j];
            const float r = inverse(sum_lanes<LPH>(sum), c);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= r * w[j];
            if (lane.turned) {
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] *= r * wo[j];
                lane.turn(cs + token * half, 1.0f, v, o);
            }
            lane.store(static_cast<T*>(c.out[side]) + (first + token) * c.out_row[side] + head * c.D, v);
        }
    }
}

// Blocks walk over the tokens; the sums for dw stay in the lanes of their channels to the end, are
// added over a block's heads in LDS, and go out as a row a block (qk_norm_weights_kernel adds those).
template <class D, int LPH>
__global__ __launch_bounds__(kThreads) void qk_norm_bwd_kernel(QkNormCall c, int most) {
    using T = typename D::T;
    constexpr int V = Piece<D>::V, HEADS = kThreads / LPH;
    __shared__ float2 cs[kMostTokens * 128];
    __shared__ float sums[HEADS][LPH * V];
    const Lane<D> lane(c, threadIdx.x % LPH);
    const int half = static_cast<int>(c.R / 2), hd = threadIdx.x / LPH;
    const float per = c.l2 ? 1.0f : 1.0f / static_cast<float>(c.D);
    float dw[2][V];
#pragma unroll
    for (int j = 0; j < V; ++j) dw[0][j] = dw[1][j] = 0.0f;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * most; first < c.tokens;
         first += static_cast<int64_t>(gridDim.x) * most) {
        const int tokens = c.tokens - first < most ? static_cast<int>(c.tokens - first) : most;
        if (c.R) {
            __syncthreads();
            angles(c, cs, first, tokens);
            __syncthreads();
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int heads = static_cast<int>(c.heads[side]);
            float w[V], unused[V];
            lane.weights(c.w[side], w, unused);
            for (int u = hd; u < tokens * heads; u += HEADS) {
                const int token = u / heads, head = u % heads;
                const T* x = static_cast<const T*>(c.x[side]) + (first + token) * c.x_row[side] + head * c.D;
                const T* dy = static_cast<const T*>(c.dy[side]) + (first + token) * c.dy_row[side] + head * c.D;
                float v[V], d[V], o[V];
                lane.load(x, v);
                lane.load(dy, d);
                if (lane.turned) {
                    lane.load_partners(dy, d, o);
                    lane.turn(cs + token * half, -1.0f, d, o);
                }
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) sum += v[j] * v[j];
                const float r = inverse(sum_lanes<LPH>(sum), c);
                float dot = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] *= r;
                    dw[side][j] += d[j] * v[j];
                    d[j] *= w[j];
                    dot += d[j] * v[j];
                }
                dot = sum_lanes<LPH>(dot) * per;
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = r * (d[j] - v[j] * dot);
                lane.store(static_cast<T*>(c.out[side]) + (first + token) * c.out_row[side] + head * c.D, d);
            }
        }
    }
    if (!c.partial) return;
    const int D_ = static_cast<int>(c.D);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) sums[hd][lane.i0 + j] = dw[side][j];
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

// tokens a block: enough blocks for every CU before a block takes more than one
int tokens_a_block(int64_t tokens) {
    const int64_t n = tokens / 2048;
    return n < 1 ? 1 : n > kMostTokens ? kMostTokens : static_cast<int>(n);
}

template <class D, int LPH>
hipError_t fwd_of(const QkNormCall& c, hipStream_t s) {
    const int n = tokens_a_block(c.tokens);
    qk_norm_fwd_kernel<D, LPH><<<static_cast<unsigned>((c.tokens + n - 1) / n), kThreads, 0, s>>>(c, n);
    return hipGetLastError();
}
template <class D, int LPH>
hipError_t bwd_of(const QkNormCall& c, hipStream_t s) {
    qk_norm_bwd_kernel<D, LPH><<<static_cast<unsigned>(qk_norm_partial_rows(c.tokens)), kThreads, 0, s>>>(
        c, tokens_a_block(c.tokens));
    return hipGetLastError();
}
template <class D>
hipError_t by_width(const QkNormCall& c, bool bwd, hipStream_t s) {
    const int64_t pieces = (c.D + Piece<D>::V - 1) / Piece<D>::V;
    if (pieces <= 8) return bwd ? bwd_of<D, 8>(c, s) : fwd_of<D, 8>(c, s);
    if (pieces <= 16) return bwd ? bwd_of<D, 16>(c, s) : fwd_of<D, 16>(c, s);
    if (pieces <= 32) return bwd ? bwd_of<D, 32>(c, s) : fwd_of<D, 32>(c, s);
    return bwd ? bwd_of<F32, 64>(c, s) : fwd_of<F32, 64>(c, s);  // fp32 only: D is at most 256
}

}  // namespace

int64_t qk_norm_partial_rows(int64_t tokens) {
    const int64_t n = tokens_a_block(tokens), blocks = (tokens + n - 1) / n;
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
