// Linear attention with one decay per head on CUDA cores (fp32 arithmetic, fp32 or bf16 storage,
// any of the head sizes): prefill and its backward pass, in chunks of 64 tokens.
//
// Three kernels. The state kernel walks the chunks of a (sequence, head, 32 rows of dv) in order
// and writes the state before each chunk (or, from the last chunk to the first, the state's
// gradient behind it); the rows of S^T evolve independently, so the split over dv is exact. The
// output and gradient kernels then take every chunk on its own, so that a few long sequences fill
// the GPU. The chunked form is in kda_hla.cuh. What bounds them: the FFMA rate, fed from shared
// memory by 4 x 8 (4 x 4, 4 x 2) register tiles of 16 x 16 threads.
#include "kda_hla.cuh"

namespace kda {
namespace {

constexpr int C = 64;
constexpr int NT = 256;
constexpr int JB = 32;  // dv rows of a state tile
constexpr int LP = C + 4;

// ------------------------------------------------------ register-tiled products
// c[i][j] += sum_k A(m, k) B(k, n) with m = ty + 16 i, n = tx + 16 j (tx, ty: this thread of 16 x 16).
// nt: A[m][k], B[n][k] rows; nn: A[m][k], B[k][n]; tn: A[k][m], B[k][n]. Row strides are multiples
// of four floats that are 4 mod 32, so that the 128-bit reads of eight consecutive rows hit all banks.
template <int K, int NI, int NJ>
__device__ __forceinline__ void mm_nt(float (&c)[NI][NJ], const float *A, int lda, const float *B, int ldb) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float4 a[NI], b[NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * lda + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * ldb + k);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                c[i][j] = fmaf(a[i].x, b[j].x, c[i][j]);
                c[i][j] = fmaf(a[i].y, b[j].y, c[i][j]);
                c[i][j] = fmaf(a[i].z, b[j].z, c[i][j]);
                c[i][j] = fmaf(a[i].w, b[j].w, c[i][j]);
            }
    }
}
template <int K, int NI, int NJ>
__device__ __forceinline__ void mm_nn(float (&c)[NI][NJ], const float *A, int lda, const float *B, int ldb) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * lda + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float b[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) b[j] = B[(k + kk) * ldb + tx + 16 * j];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float x = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
#pragma unroll
                for (int j = 0; j < NJ; ++j) c[i][j] = fmaf(x, b[j], c[i][j]);
            }
        }
    }
}
template <int K, int NI, int NJ>
__device__ __forceinline__ void mm_tn(float (&c)[NI][NJ], const float *A, int lda, const float *B, int ldb) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float a[NI], b[NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i) a[i] = A[k * lda + ty + 16 * i];
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = B[k * ldb + tx + 16 * j];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) c[i][j] = fmaf(a[i], b[j], c[i][j]);
    }
}
template <int NI, int NJ>
__device__ __forceinline__ void zero(float (&c)[NI][NJ]) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) c[i][j] = 0.f;
}

// four consecutive elements (8- or 16-byte aligned)
__device__ __forceinline__ float4 ld4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&r.x));
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&r.y));
    return make_float4(x.x, x.y, y.x, y.y);
}

// rows [row0, row0 + Lc) of columns [c0, c0 + W) of a [tokens, H, D] tensor, times `scale`; zeros from Lc on
template <typename Tin, int D, int W>
__device__ __forceinline__ void load_tile(float *s, int lds, const void *src, long long row0, int H, int h, int c0, int Lc,
                                          float scale = 1.f) {
    const Tin *p = static_cast<const Tin *>(src);
#pragma unroll 4
    for (int idx = threadIdx.x; idx < C * (W / 4); idx += NT) {
        const int r = idx / (W / 4), c = 4 * (idx % (W / 4));
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < Lc) x = ld4(p + ((size_t)(row0 + r) * H + h) * D + c0 + c);
        *reinterpret_cast<float4 *>(s + r * lds + c) = make_float4(scale * x.x, scale * x.y, scale * x.z, scale * x.w);
    }
}

// ------------------------------------------------------------------- states
// kRev = false: X = the state; a = k, b = v, row weights e^{G_C - G_s}; chunks in order; start S0, end S_T.
// kRev = true:  X = its gradient; a = q, b = dO, row weights scale e^{G_r}; chunks from the last to the
//               first; start dS_T, end dS0.
// X before each step goes to Xc [slot][H][DV][DK]. One CTA: 32 rows of dv; thread (lane, warp) holds
// rows 4 warp .. + 3 and columns lane + 32 c.
template <typename Tin, int DK, int DV, bool kRev>
__global__ void __launch_bounds__(NT) hla_state_simt_kernel(const HlaArgs p, float *__restrict__ Xc) {
    constexpr int NC = DK / 32;
    __shared__ __align__(16) float sA[C * DK];
    __shared__ __align__(16) float sB[C * JB];
    __shared__ float2 G[C];
    const int h = blockIdx.x % p.H, n = blockIdx.x / p.H, j0 = blockIdx.y * JB;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const HlaSpan sp = hla_span(p, n, C);
    const float *start = kRev ? p.dST : p.S0;
    float *end = kRev ? p.dS0 : p.ST;
    const size_t sbase = ((size_t)n * p.H + h) * (size_t)(DV * DK);

    float x[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            x[i][c] = start ? start[sbase + (size_t)(j0 + 4 * warp + i) * DK + lane + 32 * c] : 0.f;

    for (int cc = 0; cc < sp.nch; ++cc) {
        const int c = kRev ? sp.nch - 1 - cc : cc;
        const long long row0 = sp.t0 + (long long)c * C;
        const int Lc = min(C, sp.len - c * C);
        float *dst = Xc + ((size_t)(sp.slot + c) * p.H + h) * (size_t)(DV * DK);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int cx = 0; cx < NC; ++cx) dst[(size_t)(j0 + 4 * warp + i) * DK + lane + 32 * cx] = x[i][cx];
        __syncthreads();  // the previous chunk's tiles are consumed
        if (warp == 0) hla_load_scan_gate<Tin, C>(p, row0, h, Lc, G);
        load_tile<Tin, DK, DK>(sA, DK, kRev ? p.q : p.k, row0, p.H, h, 0, Lc);
        load_tile<Tin, DV, JB>(sB, JB, kRev ? p.dO : p.v, row0, p.H, h, j0, Lc);
        __syncthreads();
        const float2 gC = G[C - 1];
        const float2 g0 = make_float2(0.f, 0.f);
        for (int idx = threadIdx.x; idx < C * JB; idx += NT) {
            const float2 gr = G[idx / JB];
            sB[idx] *= kRev ? p.scale * hla_decay(gr, g0) : hla_decay(gC, gr);
        }
        __syncthreads();
        const float keep = hla_decay(gC, g0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int cx = 0; cx < NC; ++cx) x[i][cx] *= keep;
#pragma unroll 8
        for (int s = 0; s < C; ++s) {
            const float4 b = *reinterpret_cast<const float4 *>(sB + s * JB + 4 * warp);
#pragma unroll
            for (int cx = 0; cx < NC; ++cx) {
                const float a = sA[s * DK + lane + 32 * cx];
                x[0][cx] = fmaf(b.x, a, x[0][cx]);
                x[1][cx] = fmaf(b.y, a, x[1][cx]);
                x[2][cx] = fmaf(b.z, a, x[2][cx]);
                x[3][cx] = fmaf(b.w, a, x[3][cx]);
            }
        }
    }
    if (end) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) end[sbase + (size_t)(j0 + 4 * warp + i) * DK + lane + 32 * c] = x[i][c];
    }
}

// ------------------------------------------------------------------ outputs
template <int DK, int DV>
struct OutSmem {
    static constexpr int KP = DK + 4, VP = DV + 4;
    // K's tile takes the state's tiles (JB rows of DK) once Q K^T is done
    static constexpr int floats = 2 * C * KP + C * VP + C * LP;
    static constexpr size_t bytes = sizeof(float) * floats + sizeof(float2) * C;
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(NT) hla_out_simt_kernel(const HlaArgs p, const float *__restrict__ Sc) {
    using L = OutSmem<DK, DV>;
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem, *sK = sQ + C * L::KP, *sV = sK + C * L::KP, *sP = sV + C * L::VP;
    float2 *G = reinterpret_cast<float2 *>(sP + C * LP);
    const int h = blockIdx.x % p.H;
    const long long slot = blockIdx.x / p.H;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    const long long row0 = sp.t0 + (long long)c * C;
    const int Lc = min(C, sp.len - c * C);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const bool has_state = c > 0 || p.S0 != nullptr;

    if (threadIdx.x < 32) hla_load_scan_gate<Tin, C>(p, row0, h, Lc, G);
    load_tile<Tin, DK, DK>(sQ, L::KP, p.q, row0, p.H, h, 0, Lc, p.scale);
    load_tile<Tin, DK, DK>(sK, L::KP, p.k, row0, p.H, h, 0, Lc);
    load_tile<Tin, DV, DV>(sV, L::VP, p.v, row0, p.H, h, 0, Lc);
    __syncthreads();
    {
        float a[4][4];
        zero(a);
        mm_nt<DK>(a, sQ, L::KP, sK, L::KP);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, s = tx + 16 * j;
                sP[r * LP + s] = s <= r ? a[i][j] * hla_decay(G[r], G[s]) : 0.f;
            }
    }
    __syncthreads();  // P is written, K's tile is free
    float acc[4][DV / 16];
    zero(acc);
    if (has_state) {
        const float *S = Sc + ((size_t)slot * p.H + h) * (size_t)(DV * DK);
#pragma unroll
        for (int jb = 0; jb < DV / JB; ++jb) {
            for (int idx = threadIdx.x; idx < JB * (DK / 4); idx += NT) {
                const int r = idx / (DK / 4), cc = 4 * (idx % (DK / 4));
                *reinterpret_cast<float4 *>(sK + r * L::KP + cc) = ld4(S + (size_t)(jb * JB + r) * DK + cc);
            }
            __syncthreads();
            float part[4][2];
            zero(part);
            mm_nt<DK>(part, sQ, L::KP, sK, L::KP);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][2 * jb] = part[i][0];
                acc[i][2 * jb + 1] = part[i][1];
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float since = hla_decay(G[ty + 16 * i], make_float2(0.f, 0.f));
#pragma unroll
            for (int j = 0; j < DV / 16; ++j) acc[i][j] *= since;
        }
    }
    mm_nn<C>(acc, sP, LP, sV, L::VP);
    Tin *o = static_cast<Tin *>(p.o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= Lc) continue;
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) st_elem(o, ((size_t)(row0 + r) * p.H + h) * DV + tx + 16 * j, acc[i][j]);
    }
}

// ---------------------------------------------------------------- gradients
template <int DK, int DV>
struct GradSmem {
    static constexpr int KP = DK + 4, VP = DV + 4;
    // the last C x LP tile holds the state's tiles (JB x KP each) first, then the terms of dg
    static constexpr int XT = (2 * JB * KP > C * LP) ? 2 * JB * KP : C * LP;
    static constexpr int floats = 2 * C * KP + 2 * C * VP + 2 * C * LP + XT + 4 * C + 32;
    static constexpr size_t bytes = sizeof(float) * floats + sizeof(float2) * C;
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(NT) hla_grad_simt_kernel(const HlaArgs p, const float *__restrict__ Sc,
                                                           const float *__restrict__ Rc) {
    using L = GradSmem<DK, DV>;
    constexpr int KJ = DK / 16, VJ = DV / 16;
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem, *sK = sQ + C * L::KP, *sV = sK + C * L::KP, *sO = sV + C * L::VP;
    float *sA = sO + C * L::VP, *sD = sA + C * LP, *sX = sD + C * LP;
    float *sRead = sX + L::XT, *sWrit = sRead + C, *sWith = sWrit + C, *sThr = sWith + C;
    float2 *G = reinterpret_cast<float2 *>(sThr + C + 32);
    const int h = blockIdx.x % p.H;
    const long long slot = blockIdx.x / p.H;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    const long long row0 = sp.t0 + (long long)c * C;
    const int Lc = min(C, sp.len - c * C);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2 g0 = make_float2(0.f, 0.f);

    if (threadIdx.x < 32) hla_load_scan_gate<Tin, C>(p, row0, h, Lc, G);
    load_tile<Tin, DK, DK>(sQ, L::KP, p.q, row0, p.H, h, 0, Lc);
    load_tile<Tin, DK, DK>(sK, L::KP, p.k, row0, p.H, h, 0, Lc);
    load_tile<Tin, DV, DV>(sV, L::VP, p.v, row0, p.H, h, 0, Lc);
    load_tile<Tin, DV, DV>(sO, L::VP, p.dO, row0, p.H, h, 0, Lc, p.scale);
    __syncthreads();

    // the parts that go through the states: dQ from S_in, dK and dV from R, and their terms of dg
    float dq[4][KJ], dk[4][KJ];
    zero(dq);
    zero(dk);
    float thr = 0.f;
    const size_t xb = ((size_t)slot * p.H + h) * (size_t)(DV * DK);
    float *sS = sX, *sR = sX + JB * L::KP;
    Tin *out_v = static_cast<Tin *>(p.dv_);
    float dv[4][VJ];
#pragma unroll
    for (int jb = 0; jb < DV / JB; ++jb) {
        for (int idx = threadIdx.x; idx < JB * (DK / 4); idx += NT) {
            const int r = idx / (DK / 4), cc = 4 * (idx % (DK / 4));
            const float4 s4 = ld4(Sc + xb + (size_t)(jb * JB + r) * DK + cc), r4 = ld4(Rc + xb + (size_t)(jb * JB + r) * DK + cc);
            *reinterpret_cast<float4 *>(sS + r * L::KP + cc) = s4;
            *reinterpret_cast<float4 *>(sR + r * L::KP + cc) = r4;
            thr = fmaf(s4.x, r4.x, fmaf(s4.y, r4.y, fmaf(s4.z, r4.z, fmaf(s4.w, r4.w, thr))));
        }
        __syncthreads();
        mm_nn<JB>(dq, sO + jb * JB, L::VP, sS, L::KP);
        mm_nn<JB>(dk, sV + jb * JB, L::VP, sR, L::KP);
        float part[4][2];
        zero(part);
        mm_nt<DK>(part, sK, L::KP, sR, L::KP);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dv[i][2 * jb] = part[i][0];
            dv[i][2 * jb + 1] = part[i][1];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        const float since = hla_decay(G[r], g0), until = hla_decay(G[C - 1], G[r]);
        float rd = 0.f, wr = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            dq[i][j] *= since;
            dk[i][j] *= until;
            rd = fmaf(dq[i][j], sQ[r * L::KP + tx + 16 * j], rd);
            wr = fmaf(dk[i][j], sK[r * L::KP + tx + 16 * j], wr);
        }
#pragma unroll
        for (int j = 0; j < VJ; ++j) dv[i][j] *= until;
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) {
            rd += __shfl_xor_sync(0xffffffffu, rd, off);
            wr += __shfl_xor_sync(0xffffffffu, wr, off);
        }
        if (tx == 0) {
            sRead[r] = rd;
            sWrit[r] = wr;
        }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) thr += __shfl_xor_sync(0xffffffffu, thr, off);
    if (lane == 0) sThr[warp] = thr;

    // A = Q K^T . D, dA = dO' V^T . D, and the pairs within the chunk E = A . dO' V^T below the diagonal
    {
        float a[4][4], da[4][4];
        zero(a);
        zero(da);
        mm_nt<DK>(a, sQ, L::KP, sK, L::KP);
        mm_nt<DV>(da, sO, L::VP, sV, L::VP);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, s = tx + 16 * j;
                const float d = hla_decay(G[r], G[s]);
                const float x = s <= r ? a[i][j] * d : 0.f;
                sA[r * LP + s] = x;
                sD[r * LP + s] = s <= r ? da[i][j] * d : 0.f;
                sX[r * LP + s] = s < r ? x * da[i][j] : 0.f;
            }
    }
    __syncthreads();
    mm_nn<C>(dq, sD, LP, sK, L::KP);
    mm_tn<C>(dk, sD, LP, sQ, L::KP);
    mm_tn<C>(dv, sA, LP, sO, L::VP);
    Tin *out_q = static_cast<Tin *>(p.dq), *out_k = static_cast<Tin *>(p.dk_);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= Lc) continue;
        const size_t row = (size_t)(row0 + r) * p.H + h;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            st_elem(out_q, row * DK + tx + 16 * j, dq[i][j]);
            st_elem(out_k, row * DK + tx + 16 * j, dk[i][j]);
        }
#pragma unroll
        for (int j = 0; j < VJ; ++j) st_elem(out_v, row * DV + tx + 16 * j, dv[i][j]);
    }
    if (!p.dg) return;

    // dg: suffix sums of E down each column, then row sums left of the diagonal; plus the suffix sums of
    // the reads of S_in, the prefix sums of the writes that R sees, and what passes through
    if (threadIdx.x < C) {
        const int s = threadIdx.x;
        float u = 0.f;
        for (int r = C - 1; r > s; --r) {
            u += sX[r * LP + s];
            sX[r * LP + s] = u;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ty + 16 * i;
        float u = 0.f;
        for (int s = tx; s < t; s += 16) u += sX[t * LP + s];
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
        if (tx == 0) sWith[t] = u;
    }
    __syncthreads();
    if (threadIdx.x < C) {
        const int t = threadIdx.x;
        float rd = 0.f, wr = 0.f, through = 0.f;
        for (int r = C - 1; r >= t; --r) rd += sRead[r];
        for (int s = 0; s < t; ++s) wr += sWrit[s];
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) through += sThr[w];
        if (t < Lc)
            st_elem(static_cast<Tin *>(p.dg), (size_t)(row0 + t) * p.H + h,
                    (sWith[t] + rd) + fmaf(hla_decay(G[C - 1], g0), through, wr));
    }
}

// Rows of a packed batch that belong to no sequence (before the first, behind the last) have no part in
// the result: their gradients are zero.
template <typename Tin>
__global__ void __launch_bounds__(NT) hla_clear_outside_kernel(const HlaArgs p) {
    const int first = min(max(p.cu_seqlens[0], 0), p.T), last = min(max(p.cu_seqlens[p.N], first), p.T);
    const int outside = p.T - (last - first);
    for (int i = blockIdx.x; i < outside; i += gridDim.x) {
        const size_t row = i < first ? i : last + (i - first);
        const auto clear = [&](void *x, int d) {
            if (!x) return;
            Tin *y = static_cast<Tin *>(x) + row * p.H * d;
            for (int c = threadIdx.x; c < p.H * d; c += NT) st_elem(y, c, 0.f);
        };
        clear(p.dq, p.dk);
        clear(p.dk_, p.dk);
        clear(p.dv_, p.dv);
        clear(p.dg, 1);
    }
}

// ----------------------------------------------------------------- launches
template <typename F>
cudaError_t with_smem(F kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename Tin, int DK, int DV>
cudaError_t forward_t(const HlaArgs &a) {
    float *Sc = static_cast<float *>(a.workspace);
    const long long slots = hla_slots(a.cu_seqlens != nullptr, a.N, a.T, C);
    hla_state_simt_kernel<Tin, DK, DV, false><<<dim3((unsigned)(a.N * a.H), DV / JB), NT, 0, a.stream>>>(a, Sc);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || slots == 0 || a.T == 0) return e;
    const auto kern = hla_out_simt_kernel<Tin, DK, DV>;
    constexpr size_t bytes = OutSmem<DK, DV>::bytes;
    if ((e = with_smem(kern, bytes)) != cudaSuccess) return e;
    kern<<<(unsigned)(slots * a.H), NT, bytes, a.stream>>>(a, Sc);
    return cudaGetLastError();
}

template <typename Tin, int DK, int DV>
cudaError_t backward_t(const HlaArgs &a) {
    const long long slots = hla_slots(a.cu_seqlens != nullptr, a.N, a.T, C);
    float *Sc = static_cast<float *>(a.workspace), *Rc = Sc + (size_t)slots * a.H * DV * DK;
    const dim3 grid((unsigned)(a.N * a.H), DV / JB);
    HlaArgs f = a;
    f.ST = nullptr;
    hla_state_simt_kernel<Tin, DK, DV, false><<<grid, NT, 0, a.stream>>>(f, Sc);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    hla_state_simt_kernel<Tin, DK, DV, true><<<grid, NT, 0, a.stream>>>(a, Rc);
    e = cudaGetLastError();
    if (e != cudaSuccess || slots == 0 || a.T == 0) return e;
    const auto kern = hla_grad_simt_kernel<Tin, DK, DV>;
    constexpr size_t bytes = GradSmem<DK, DV>::bytes;
    if ((e = with_smem(kern, bytes)) != cudaSuccess) return e;
    kern<<<(unsigned)(slots * a.H), NT, bytes, a.stream>>>(a, Sc, Rc);
    return cudaGetLastError();
}

template <typename Tin, int DK>
cudaError_t pass_dv(const HlaArgs &a, bool back) {
    switch (a.dv) {
        case 32: return back ? backward_t<Tin, DK, 32>(a) : forward_t<Tin, DK, 32>(a);
        case 64: return back ? backward_t<Tin, DK, 64>(a) : forward_t<Tin, DK, 64>(a);
        case 128: return back ? backward_t<Tin, DK, 128>(a) : forward_t<Tin, DK, 128>(a);
        default: return cudaErrorInvalidValue;
    }
}
template <typename Tin>
cudaError_t pass_t(const HlaArgs &a, bool back) {
    switch (a.dk) {
        case 32: return pass_dv<Tin, 32>(a, back);
        case 64: return pass_dv<Tin, 64>(a, back);
        case 128: return pass_dv<Tin, 128>(a, back);
        default: return cudaErrorInvalidValue;
    }
}
cudaError_t pass(const HlaArgs &a, bool back) {
    return a.dtype == KDA_DTYPE_BF16 ? pass_t<__nv_bfloat16>(a, back) : pass_t<float>(a, back);
}

}  // namespace

size_t hla_forward_simt_workspace(const HlaArgs &a) {
    return sizeof(float) * (size_t)hla_slots(a.cu_seqlens != nullptr, a.N, a.T, C) * a.H * a.dk * a.dv;
}
cudaError_t launch_hla_clear_outside(const HlaArgs &a) {
    const unsigned grid = (unsigned)(a.T < 1024 ? a.T : 1024);
    if (a.dtype == KDA_DTYPE_BF16) hla_clear_outside_kernel<__nv_bfloat16><<<grid, NT, 0, a.stream>>>(a);
    else hla_clear_outside_kernel<float><<<grid, NT, 0, a.stream>>>(a);
    return cudaGetLastError();
}
size_t hla_backward_simt_workspace(const HlaArgs &a) { return 2 * hla_forward_simt_workspace(a); }
cudaError_t launch_hla_forward_simt(const HlaArgs &a) { return pass(a, false); }
cudaError_t launch_hla_backward_simt(const HlaArgs &a) { return pass(a, true); }

}  // namespace kda
