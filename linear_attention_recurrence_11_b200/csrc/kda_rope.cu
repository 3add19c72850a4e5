// Rotary positions: the channels (a, b) of pair i of a head at position p become
//   (a cos x - b sin x, b cos x + a sin x) * mscale,   x = p * inv_freq[i]   (inverse: x = -p * inv_freq[i])
// over the first rot_dim channels; the others pass through. Pairs are (i, i + rot_dim / 2), or
// (2i, 2i + 1) when interleaved. The transposed rotation (inverse, same mscale) is the gradient.
//
// Bound by HBM bandwidth: every element is read and written once. A CTA takes a tile of tokens (of
// all heads of q and k, or a share of them when tokens are few): the angles of its tokens are
// computed once, into shared memory, and used by every head. The angle is reduced in fp64, as
// p * (inv_freq / 2 pi) minus its nearest integer, so that positions of millions keep fp32's full
// precision; sine and cosine are then taken of at most half a turn. One thread moves vectors of VE
// elements, the widest of up to 16 bytes that the pair halves, the rotated part and the head all
// divide into.
#include "kda_hla.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 4096;  // (token, pair) angles of a CTA: 32 KB of shared memory

template <typename T, int VE>
struct alignas(sizeof(T) * VE) Vec {
    T x[VE];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &y, float x) { y = __float2bfloat16_rn(x); }

template <typename T, int VE, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs p, int tile, int share) {
    extern __shared__ float2 cs[];  // [token of the tile][pair]: cos, sin, times mscale
    using V = Vec<T, VE>;
    const int half = p.rot_dim >> 1;
    const long long tok0 = (long long)blockIdx.x * tile;
    const int nt = (int)(p.tokens - tok0 < tile ? p.tokens - tok0 : tile);
    const double turn = 0.15915494309189535;  // 1 / (2 pi)

    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const long long tok = tok0 + t;
        const long long pos = !p.positions ? tok % p.T
                              : p.pos64    ? static_cast<const long long *>(p.positions)[tok]
                                           : (long long)static_cast<const int *>(p.positions)[tok];
        double x = (double)pos * ((double)p.inv_freq[f] * turn);
        x -= rint(x);
        float s, c;
        sincospif(2.f * (float)x, &s, &c);
        cs[i] = make_float2(p.mscale * c, p.mscale * (p.inverse ? -s : s));
    }
    __syncthreads();

    // a row is one head of one token: `per` threads each take one of its vectors (a pair of vectors in the
    // half layout), and the CTA `lanes` rows at a time; q's heads come first, then k's
    const int heads = p.Hq + p.Hk, h0 = blockIdx.y * share, h1 = min(heads, h0 + share), hs = h1 - h0;
    const int nrot = kInter ? p.rot_dim / VE : half / VE, per = nrot + (p.d - p.rot_dim) / VE;
    const int lanes = max(1, kThreads / per);
    const int r0 = threadIdx.x / per;
    const int rows = nt * hs;
    for (int j = threadIdx.x - r0 * per; j < per; j += kThreads) {
        if (r0 >= lanes) break;
        for (int r = r0; r < rows; r += lanes) {
            const int t = r / hs, h = h0 + (r - t * hs);
            const bool isq = h < p.Hq;
            const size_t row = isq ? ((size_t)(tok0 + t) * p.Hq + h) : ((size_t)(tok0 + t) * p.Hk + (h - p.Hq));
            const T *src = static_cast<const T *>(isq ? p.q : p.k) + row * p.d;
            T *dst = static_cast<T *>(isq ? p.q_out : p.k_out) + row * p.d;
            if (j >= nrot) {  // channels that are not rotated
                if (src != dst) {
                    const int c = p.rot_dim + (j - nrot) * VE;
                    *reinterpret_cast<V *>(dst + c) = *reinterpret_cast<const V *>(src + c);
                }
                continue;
            }
            const float2 *ang = cs + t * half;
            if (kInter) {
                V x = *reinterpret_cast<const V *>(src + j * VE);
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    const float2 w = ang[(j * VE + e) >> 1];
                    const float a = to_f(x.x[e]), b = to_f(x.x[e + 1]);
                    from_f(x.x[e], a * w.x - b * w.y);
                    from_f(x.x[e + 1], b * w.x + a * w.y);
                }
                *reinterpret_cast<V *>(dst + j * VE) = x;
            } else {
                V x = *reinterpret_cast<const V *>(src + j * VE), y = *reinterpret_cast<const V *>(src + half + j * VE);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float2 w = ang[j * VE + e];
                    const float a = to_f(x.x[e]), b = to_f(y.x[e]);
                    from_f(x.x[e], a * w.x - b * w.y);
                    from_f(y.x[e], b * w.x + a * w.y);
                }
                *reinterpret_cast<V *>(dst + j * VE) = x;
                *reinterpret_cast<V *>(dst + half + j * VE) = y;
            }
        }
    }
}

template <typename T, int VE>
cudaError_t launch_ve(const RopeArgs &a) {
    const int heads = a.Hq + a.Hk, half = a.rot_dim / 2;
    // tiles of about 16 KB of rows, so that few angles are computed per byte and many CTAs remain
    long long tile = (16384 + (long long)heads * a.d * sizeof(T) - 1) / ((long long)heads * a.d * sizeof(T));
    if (tile * half > kMaxAngles) tile = kMaxAngles / half;
    if (tile < 1) tile = 1;
    if (tile > a.tokens) tile = a.tokens;
    const long long tiles = (a.tokens + tile - 1) / tile;
    // few tokens: a token's heads are shared out over CTAs
    int splits = 1;
    while (splits < heads && tiles * splits < 2LL * device_sm_count() && (long long)tile * heads * a.d * sizeof(T) / splits > 4096)
        splits *= 2;
    const int share = (heads + splits - 1) / splits;
    const dim3 grid((unsigned)tiles, (unsigned)((heads + share - 1) / share));
    const size_t smem = sizeof(float2) * (size_t)(tile * half);
    if (a.interleaved) rope_kernel<T, VE, true><<<grid, kThreads, smem, a.stream>>>(a, (int)tile, share);
    else rope_kernel<T, VE, false><<<grid, kThreads, smem, a.stream>>>(a, (int)tile, share);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs &a) {
    // every vector of a row starts at a multiple of VE: heads (d), the rotated part, and in the half
    // layout its halves; the tensors themselves are 16-byte aligned
    const int unit = a.interleaved ? a.rot_dim : a.rot_dim / 2;
    const auto fits = [&](int ve) { return a.d % ve == 0 && a.rot_dim % ve == 0 && unit % ve == 0; };
    if (sizeof(T) == 2 && fits(8)) return launch_ve<T, 16 / sizeof(T)>(a);
    if (fits(4)) return launch_ve<T, 4>(a);
    if (fits(2)) return launch_ve<T, 2>(a);
    // an odd head dimension, or (half layout) an odd number of pairs: single elements
    return a.interleaved ? cudaErrorInvalidValue : launch_ve<T, 1>(a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a) {
    if (a.tokens == 0) return cudaSuccess;
    return a.dtype == KDA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace kda
