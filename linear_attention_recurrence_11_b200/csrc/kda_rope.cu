// Rotary positions: the channels (a, b) of pair i of a head at position p become
//   (a cos x - b sin x, b cos x + a sin x) * mscale,   x = p * inv_freq[i]   (inverse: x = -p * inv_freq[i])
// over the first rot_dim channels; the others pass through. Pairs are (i, i + rot_dim / 2), or
// (2i, 2i + 1) when interleaved. The transposed rotation (inverse, same mscale) is the gradient.
//
// Bound by HBM bandwidth: every element is read and written once. A CTA takes a tile of tokens (of
// all heads of q and k, or a share of them when tokens are few): the angles of its tokens are
// computed once, into shared memory, and used by every head. The angle is reduced in fp64, as
// p * (inv_freq / 2 pi) minus its nearest integer, so that positions of millions keep fp32's full
// precision; sine and cosine are then taken of at most half a turn, for bf16 by the special-function
// unit (2^-21 of a pair's length, where a result's own rounding is up to 2^-8).
//
// Two forms. Where pairs stay within a 16-byte vector (interleaved) or their halves divide into vectors of 16 or 8
// bytes, a thread turns whole vectors in registers. Else (an odd number of pairs, say) the rows are staged in shared
// memory, so that HBM still sees 16-byte accesses, and the elements are turned from there. Measured on q and k of 96
// heads x 8192 tokens of 128 channels in bf16: all rotated 126 us (6.4 TB/s); 86 of them rotated in halves of 43, by
// single elements 512, staged 278.
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

// a / b as a product, for a b < 2^32: m = ceil(2^32 / b) (b > 1) is off by less than 1, a m / 2^32 by less than 1 / b
struct Div {
    uint32_t b, m;
    explicit Div(uint32_t x) : b(x), m(x > 1 ? (uint32_t)((0x100000000ull + x - 1) / x) : 0) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t a) const { return b > 1 ? __umulhi(a, m) : a; }
};

struct RopeTile {
    int tile, share;      // tokens, heads of a CTA
    Div half, heads, per;  // pairs; `share`; threads (vectors) of a row
};

// cos and sin, times mscale, of the tile's tokens and pairs
template <typename T>
__device__ __forceinline__ void angles(const RopeArgs &p, const RopeTile &k, long long tok0, int nt, float2 *cs) {
    const int half = p.rot_dim >> 1;
    const double turn = 0.15915494309189535;  // 1 / (2 pi)
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = (int)k.half(i), f = i - t * half;
        const long long tok = tok0 + t;
        const long long pos = !p.positions ? tok % p.T
                              : p.pos64    ? static_cast<const long long *>(p.positions)[tok]
                                           : (long long)static_cast<const int *>(p.positions)[tok];
        double x = (double)pos * ((double)p.inv_freq[f] * turn);
        x -= rint(x);
        float s, c;
        if (sizeof(T) == 2) {
            const float y = 6.28318531f * (float)x;
            s = __sinf(y);
            c = __cosf(y);
        } else {
            sincospif(2.f * (float)x, &s, &c);
        }
        cs[i] = make_float2(p.mscale * c, p.mscale * (p.inverse ? -s : s));
    }
}

// row r of the CTA: its token in the tile, and where it is (q's heads come first, then k's)
template <typename T>
__device__ __forceinline__ int locate(const RopeArgs &p, const RopeTile &k, long long tok0, int h0, int r, const T *&src, T *&dst) {
    const int t = (int)k.heads(r), h = h0 + (r - t * k.heads.b);
    const bool isq = h < p.Hq;
    const size_t row = isq ? ((size_t)(tok0 + t) * p.Hq + h) : ((size_t)(tok0 + t) * p.Hk + (h - p.Hq));
    src = static_cast<const T *>(isq ? p.q : p.k) + row * p.d;
    dst = static_cast<T *>(isq ? p.q_out : p.k_out) + row * p.d;
    return t;
}

// kTail (interleaved): the last rotated vector ends in channels that are not
template <typename T, int VE, bool kInter, bool kTail>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs p, const RopeTile k) {
    extern __shared__ __align__(16) uint8_t smem[];
    float2 *cs = reinterpret_cast<float2 *>(smem);  // [token of the tile][pair]
    using V = Vec<T, VE>;
    const int half = p.rot_dim >> 1;
    const long long tok0 = (long long)blockIdx.x * k.tile;
    const int nt = (int)(p.tokens - tok0 < k.tile ? p.tokens - tok0 : k.tile);
    angles<T>(p, k, tok0, nt, cs);
    __syncthreads();

    // `per` threads take a row's vectors (a pair of vectors in the half layout); a CTA's last share may be smaller
    const int h0 = blockIdx.y * k.share, hs = min(k.share, p.Hq + p.Hk - h0);
    const int nrot = kInter ? (p.rot_dim + VE - 1) / VE : half / VE, per = (int)k.per.b;
    const int items = nt * (int)k.heads.b * per;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int r = (int)k.per(i), j = i - r * per;
        const T *src;
        T *dst;
        const int t = locate(p, k, tok0, h0, r, src, dst);
        if (r - t * (int)k.heads.b >= hs) continue;
        if (j >= nrot) {  // channels that are not rotated
            if (src != dst) {
                const int c = (kInter ? 0 : nrot * VE) + j * VE;
                *reinterpret_cast<V *>(dst + c) = *reinterpret_cast<const V *>(src + c);
            }
            continue;
        }
        const float2 *ang = cs + t * half;
        if (kInter) {
            V x = *reinterpret_cast<const V *>(src + j * VE);
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                if (kTail && j * VE + e >= p.rot_dim) continue;
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

// VE: elements of a vector of a whole row (any alignment of the pairs within it); kStage rows at a time
constexpr int kStageBytes = 16384;

template <typename T, int VE>
__global__ void __launch_bounds__(kThreads) rope_staged_kernel(const RopeArgs p, const RopeTile k, int rows_at_once, int angle_bytes) {
    extern __shared__ __align__(16) uint8_t smem[];
    float2 *cs = reinterpret_cast<float2 *>(smem);
    T *stage = reinterpret_cast<T *>(smem + angle_bytes);
    using V = Vec<T, VE>;
    const int half = p.rot_dim >> 1, per = (int)k.per.b;
    const long long tok0 = (long long)blockIdx.x * k.tile;
    const int nt = (int)(p.tokens - tok0 < k.tile ? p.tokens - tok0 : k.tile);
    angles<T>(p, k, tok0, nt, cs);
    const int h0 = blockIdx.y * k.share, hs = min(k.share, p.Hq + p.Hk - h0);
    const int rows = nt * (int)k.heads.b, lanes = max(1, kThreads / per), first = threadIdx.x / per;
    for (int r0 = 0; r0 < rows; r0 += rows_at_once) {
        const int n = min(rows_at_once, rows - r0), items = n * per;
        __syncthreads();  // the rows before have been turned (or the angles are there)
        for (int i = threadIdx.x; i < items; i += kThreads) {
            const int r = (int)k.per(i), j = i - r * per;
            const T *src;
            T *dst;
            const int t = locate(p, k, tok0, h0, r0 + r, src, dst);
            if (r0 + r - t * (int)k.heads.b < hs) *reinterpret_cast<V *>(stage + i * VE) = *reinterpret_cast<const V *>(src + j * VE);
        }
        __syncthreads();
        // a thread keeps its vector's place in the row, so that its partners' places and, while the token stays, its
        // angles stay in registers
        for (int j = threadIdx.x - first * per; first < lanes && j < per; j += kThreads) {
            int other[VE], pair[VE];
            float sign[VE];
            float2 w[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int c = j * VE + e;  // the first of a pair: a cos - b sin; the second: b cos + a sin
                const bool second = p.interleaved ? (c & 1) : c >= half, turned = c < p.rot_dim;
                other[e] = !turned ? c : p.interleaved ? c ^ 1 : second ? c - half : c + half;
                pair[e] = !turned ? -1 : p.interleaved ? c >> 1 : second ? c - half : c;
                sign[e] = second ? 1.f : -1.f;
            }
            int at = -1;  // the token whose angles are held
            for (int r = first; r < n; r += lanes) {
                const T *src;
                T *dst;
                const int t = locate(p, k, tok0, h0, r0 + r, src, dst);
                if (r0 + r - t * (int)k.heads.b >= hs) continue;
                if (t != at) {
                    at = t;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        w[e] = pair[e] < 0 ? make_float2(1.f, 0.f) : cs[t * half + pair[e]];
                        w[e].y *= sign[e];
                    }
                }
                const T *row = stage + r * p.d;
                V x = *reinterpret_cast<const V *>(row + j * VE);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (pair[e] >= 0) from_f(x.x[e], to_f(x.x[e]) * w[e].x + to_f(row[other[e]]) * w[e].y);
                *reinterpret_cast<V *>(dst + j * VE) = x;
            }
        }
    }
}

template <typename T>
RopeTile tile_of(const RopeArgs &a, int per, unsigned &tiles, unsigned &shares) {
    const int heads = a.Hq + a.Hk, half = a.rot_dim / 2;
    const long long row = (long long)a.d * sizeof(T);
    // tiles of about 16 KB of rows, so that few angles are computed per byte and many CTAs remain
    long long tile = (16384 + heads * row - 1) / (heads * row);
    if (tile * half > kMaxAngles) tile = kMaxAngles / half;
    if (tile < 1) tile = 1;
    if (tile > a.tokens) tile = a.tokens;
    const long long n = (a.tokens + tile - 1) / tile;
    // few tokens: a token's heads are shared out over CTAs; and a CTA's items stay below 2^20
    int splits = 1;
    while (splits < heads && ((n * splits < 2LL * device_sm_count() && tile * heads * row / splits > 4096) || tile * heads / splits * per >= (1 << 19)))
        splits *= 2;
    const int share = (heads + splits - 1) / splits;
    tiles = (unsigned)n;
    shares = (unsigned)((heads + share - 1) / share);
    return RopeTile{(int)tile, share, Div(half), Div(share), Div(per)};
}

template <typename T, int VE>
cudaError_t launch_ve(const RopeArgs &a) {
    // threads of a row: its vectors, or (half layout) pairs of vectors and the vectors that are not rotated
    const int per = a.interleaved ? a.d / VE : a.rot_dim / 2 / VE + (a.d - a.rot_dim) / VE;
    unsigned tiles, shares;
    const RopeTile k = tile_of<T>(a, per, tiles, shares);
    const size_t smem = sizeof(float2) * (size_t)k.tile * (a.rot_dim / 2);
    const auto kern = !a.interleaved ? rope_kernel<T, VE, false, false> : a.rot_dim % VE == 0 ? rope_kernel<T, VE, true, false> : rope_kernel<T, VE, true, true>;
    kern<<<dim3(tiles, shares), kThreads, smem, a.stream>>>(a, k);
    return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t launch_staged(const RopeArgs &a) {
    unsigned tiles, shares;
    const RopeTile k = tile_of<T>(a, a.d / VE, tiles, shares);
    const int rows = kStageBytes / (int)(a.d * sizeof(T)) > 0 ? kStageBytes / (int)(a.d * sizeof(T)) : 1;
    const int angle_bytes = (int)((sizeof(float2) * (size_t)k.tile * (a.rot_dim / 2) + 15) & ~(size_t)15);
    rope_staged_kernel<T, VE><<<dim3(tiles, shares), kThreads, angle_bytes + rows * a.d * sizeof(T), a.stream>>>(a, k, rows, angle_bytes);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs &a) {
    // Interleaved pairs stay within a vector. In the half layout, vectors of 16 or 8 bytes in registers where the pairs'
    // halves divide into them (and so the rotated part does); else the rows are staged, in 16 bytes, or in the widest
    // pieces that the head divides into (d is even).
    constexpr int W = 16 / sizeof(T);
    const int half = a.rot_dim / 2;
    if (a.d % W == 0) {
        if (a.interleaved || half % W == 0) return launch_ve<T, W>(a);
        return half % (W / 2) == 0 ? launch_ve<T, W / 2>(a) : launch_staged<T, W>(a);
    }
    if (a.d % 4 == 0) return a.interleaved || half % 4 == 0 ? launch_ve<T, 4>(a) : launch_staged<T, 4>(a);
    return a.interleaved || half % 2 == 0 ? launch_ve<T, 2>(a) : launch_staged<T, 2>(a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a) {
    if (a.tokens == 0) return cudaSuccess;
    return a.dtype == KDA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace kda
