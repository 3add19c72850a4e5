// Linear attention with one decay per head in fp32 accuracy (fp32 or bf16 storage, any of the head sizes):
// prefill and its backward pass, in chunks of 64 tokens. The chunked form is in kda_hla.cuh.
//
// Three kernels. The state kernel walks the chunks of a (sequence, head, 64 rows of dv) in order and writes the
// state before each chunk (or, from the last chunk to the first, the state's gradient behind it); the rows of S^T
// evolve independently, so the split over dv is exact, and where chains are few the sequences are cut into
// segments. The output and gradient kernels then take every chunk on its own.
//
// Products: warp-level TF32 matrix instructions on operands split into two TF32 numbers each, x = hi + lo with 11 + 11
// bits, as lo hi + hi lo + hi hi with fp32 accumulation: what is dropped is below 2^-21 of a product, the order of
// fp32's own rounding. Measured against FFMA register tiles (4 x 8 per thread), the gradients of 16 heads x 2099
// tokens take 0.4 of the time: a fragment's element is read from shared memory once for 8 to 32 products. For 2 x 1000
// tokens, 16 heads of 128: states 30 us (in two segments), outputs 51, gradients 158 (0.45 of the instructions' rate: a
// fragment's element costs a load and three operations for every instruction, and a tile's 194 KB arrive before it begins,
// since one tile fills the SM).
#include "kda_hla.cuh"
#include "kda_hla_gate.cuh"

namespace kda {
namespace {

constexpr int C = 64;
constexpr int NT = 256;
constexpr int NG = 512;     // of the gradients: one CTA per SM, 4 x 4 warps
constexpr int JB = 32;      // dv rows of a state tile of the gradients
constexpr uint32_t GATE = kHlaGateBytes<C>;
constexpr int LP = C + 4;   // row strides are 4 mod 32 floats, but where a comment says otherwise: no bank conflicts along rows

// ------------------------------------------------------------------ products
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;   // to nearest, in magnitude
    lo = __float_as_uint(x - __uint_as_float(hi));       // (its low bits are ignored: 2^-10 of it)
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Rows of 16 bytes of shared memory, eight (or four times eight) by the lanes' addresses: lane 4 g + t gets word t of the
// g-th row of each eight.
__device__ __forceinline__ void ld_rows2(const float *p, float &a, float &b) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"((uint32_t)__cvta_generic_to_shared(p)) : "memory");
}
__device__ __forceinline__ void ld_rows4(const float *p, float (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"((uint32_t)__cvta_generic_to_shared(p)) : "memory");
}

// A warp's part of a product: 16 or 32 rows from m0 on, and of every `step` columns 8 from n0 on. With g = lane / 4 and
// t = lane % 4, c[i][j] holds rows m0 + 16 i + g (elements 0, 1) and + 8 (2, 3), columns n0 + step j + 2 t and + 1.
struct WarpTile {
    int m0, n0, g, t;
    __device__ __forceinline__ int row(int i, int e) const { return m0 + 16 * i + g + 8 * (e >> 1); }
    template <int kStep>
    __device__ __forceinline__ int col(int j, int e) const { return n0 + kStep * j + 2 * t + (e & 1); }
};
// over 64 rows, and columns in steps of 32: 2 x 4 warps of 32 rows, or 4 x 4 of 16
template <int kRows>
__device__ __forceinline__ WarpTile tile_of_warp() {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    return {kRows * (warp >> 2), 8 * (warp & 3), lane >> 2, lane & 3};
}

// c += A B over K. A is [m][k], or with kAT [k][m], the latter with kW times a weight of each k; B is [k][n], or with kBT
// [n][k]. The matrix instructions cut their
// sums off instead of rounding them: over K = 128 that alone came to 3e-6 of the result. So 16 of K at a time are summed
// by them, from zero, and added to c in fp32 (4e-7).
template <int K, int kStep, bool kAT, bool kBT, bool kW = false, int MI, int NJ>
__device__ __forceinline__ void mm(float (&c)[MI][NJ][4], const WarpTile &w, const float *A, int lda, const float *B, int ldb,
                                   const float *weight = nullptr) {
    static_assert(!kBT || NJ == 1 || NJ % 2 == 0, "column tiles are read in pairs");
    const int lane = 4 * w.g + w.t;
    // Which k of the eight is whose does not matter as long as A and B agree. Rows by matrix loads come as t and t + 4;
    // where both are read down the columns, 2 t and 2 t + 1 spread over all banks if row strides are 4 mod 32 (else 8).
    constexpr bool kCols = kAT && !kBT;
    const int kt = kCols ? 2 * w.t : w.t;
    constexpr int kNext = kCols ? 1 : 4;
#pragma unroll 1
    for (int kb = 0; kb < K; kb += 16) {
        float sum[MI][NJ][4];
#pragma unroll
        for (int kk = 0; kk < 16; kk += 8) {
            const int k0 = kb + kk;
            uint32_t ah[MI][4], al[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                float v[4];
                if (!kAT) ld_rows4(A + (w.m0 + 16 * i + (lane & 15)) * lda + k0 + 4 * (lane >> 4), v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int m = w.m0 + 16 * i + w.g + 8 * (e & 1), k = k0 + kt + kNext * (e >> 1);
                    if (kAT) v[e] = (kW ? weight[k] : 1.f) * A[k * lda + m];
                    split_tf32(v[e], ah[i][e], al[i][e]);
                }
            }
            float two[4];  // B of this column tile and the next
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                uint32_t bh[2], bl[2];
                if (kBT && NJ == 1) ld_rows2(B + (w.n0 + (lane & 7)) * ldb + k0 + 4 * ((lane >> 3) & 1), two[0], two[1]);
                if (kBT && NJ > 1 && j % 2 == 0) ld_rows4(B + (w.n0 + kStep * (j + (lane >> 4)) + (lane & 7)) * ldb + k0 + 4 * ((lane >> 3) & 1), two);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = w.n0 + kStep * j + w.g, k = k0 + kt + kNext * e;
                    split_tf32(kBT ? two[2 * (j & 1) + e] : B[k * ldb + n], bh[e], bl[e]);
                }
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    if (kk == 0) sum[i][j][0] = sum[i][j][1] = sum[i][j][2] = sum[i][j][3] = 0.f;
                    mma_tf32(sum[i][j], al[i], bh);
                    mma_tf32(sum[i][j], ah[i], bl);
                    mma_tf32(sum[i][j], ah[i], bh);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[i][j][e] += sum[i][j][e];
    }
}
template <int MI, int NJ>
__device__ __forceinline__ void zero(float (&c)[MI][NJ][4]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[i][j][e] = 0.f;
}

// this thread's G of a chunk (threads 0 .. C - 1)
__device__ __forceinline__ float2 gate_of(const uint8_t *gates, long long slot, int H, int h) {
    return __ldg(reinterpret_cast<const float2 *>(gates + ((size_t)slot * H + h) * GATE) + threadIdx.x);
}

// four consecutive elements (8-byte aligned)
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&r.x));
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&r.y));
    return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ void st2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void st2(__nv_bfloat16 *p, float x, float y) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}

// 16 bytes of fp32 to shared memory, asynchronously; zeros if not `there`
__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }  // all but the last N groups

// Columns [c0, c0 + W) of a chunk's rows of a [tokens, H, D] tensor as fp32 in shared memory, zeros from row Lc on: there
// once the thread's copies have been waited for and the block has met. fp32 is copied asynchronously (through registers,
// the state kernel's loads alone held a chunk up for 3000 of 11000 clocks); bf16 is converted on its way.
template <typename Tin, int D, int W, int kThreads = NT>
__device__ __forceinline__ void fetch_tile(float *s, int lds, const void *src, long long row0, int H, int h, int c0, int Lc) {
    constexpr int N = C * (W / 4) / kThreads;
    static_assert(N * kThreads == C * (W / 4), "whole rows of threads");
    const Tin *base = static_cast<const Tin *>(src) + ((size_t)row0 * H + h) * D + c0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int idx = threadIdx.x + kThreads * i, r = idx / (W / 4), c = 4 * (idx % (W / 4));
        const Tin *at = base + (r < Lc ? (size_t)r * H * D : 0) + c;
        if constexpr (sizeof(Tin) == 4) copy16(s + r * lds + c, at, r < Lc);
        else *reinterpret_cast<float4 *>(s + r * lds + c) = r < Lc ? ld4(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
// `rows` rows of a state
template <int D, int kThreads = NT>
__device__ __forceinline__ void fetch_state(float *s, int lds, const float *src, int rows) {
    for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kThreads) {
        const int r = idx / (D / 4), c = 4 * (idx % (D / 4));
        copy16(s + r * lds + c, src + (size_t)r * D + c, true);
    }
}

// ------------------------------------------------------------------- states
// Direction 0: X = the state; a = k, b = v, row weights e^{G_C - G_s}; chunks in order; start S0, end S_T.
// Direction 1: X = its gradient; a = q, b = dO, row weights scale e^{G_r}; chunks from the last to the first; start
// dS_T, end dS0. X before each step goes to X[dir] [slot][H][DV][DK]. With segments (sc > 0), a first launch (ends)
// writes each segment's end state from zero, and the second starts from the segments' start states.
struct StateArgs {
    HlaArgs a;
    const uint8_t *gates;
    float *X[2];
    HlaSegments seg;
    bool ends;
};

// One CTA: ROWS rows of dv; its 8 warps 2 x 4 over 64 rows, or 1 x 8 (1 x 4) over 32.
template <int DK, int DV>
struct StateTile {
    static constexpr int ROWS = DV < 64 ? 32 : 64, WN = ROWS == 64 ? 4 : DK < 64 ? 4 : 8, NJ = DK / (8 * WN);
    static constexpr int KP = DK + 4, VP = ROWS + 4;
    static constexpr size_t bytes = sizeof(float) * (2 * C * (KP + VP) + 2 * (C + 4));  // two chunks' tiles, weights and decay
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(NT, 2) hla_state_simt_kernel(const StateArgs s) {
    using L = StateTile<DK, DV>;
    constexpr int KP = L::KP, VP = L::VP, WN = L::WN, NJ = L::NJ, ROWS = L::ROWS;
    const HlaArgs &p = s.a;
    extern __shared__ __align__(16) float smem[];
    float *sA = smem, *sB = sA + 2 * C * KP, *sW = sB + 2 * C * VP;
    const int dir = blockIdx.z, j0 = blockIdx.y * ROWS, h = blockIdx.x % p.H;
    const long long su = blockIdx.x / p.H;
    int n = (int)su, sg = 0;
    HlaSpan sp;
    if (s.seg.sc && !hla_segment_of(p, su, s.seg.sc * C, n, sg)) return;
    sp = hla_span(p, n, C);
    const int nseg = s.seg.sc ? max(1, (sp.nch + s.seg.sc - 1) / s.seg.sc) : 1;
    const int c0 = s.seg.sc ? sg * s.seg.sc : 0, c1 = s.seg.sc ? min(sp.nch, c0 + s.seg.sc) : sp.nch, nc = c1 - c0;
    const bool last = dir ? sg == 0 : sg == nseg - 1;
    if (s.ends && last) return;
    const size_t base_n = ((size_t)n * p.H + h) * (size_t)(DV * DK), base_s = ((size_t)su * p.H + h) * (size_t)(DV * DK);
    const float *start = s.ends ? nullptr : s.seg.sc ? s.seg.state[dir] + base_s : dir ? p.dST : p.S0;
    if (start && !s.seg.sc) start += base_n;
    float *end = s.ends ? s.seg.state[dir] + base_s : !last ? nullptr : dir ? p.dS0 : p.ST;
    if (end && !s.ends) end += base_n;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WarpTile w{ROWS == 64 ? 32 * (warp >> 2) : 0, 8 * (warp % WN), lane >> 2, lane & 3};
    const bool active = ROWS == 64 || warp < WN;
    float x[2][NJ][4];
    const auto each = [&](auto f) {  // (pairs of columns)
        if (active)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) f((size_t)(j0 + w.row(i, e)) * DK + w.col<8 * WN>(j, e), x[i][j][e], x[i][j][e + 1]);
    };
    zero(x);
    if (start) each([&](size_t at, float &u, float &v) {
        const float2 y = *reinterpret_cast<const float2 *>(start + at);
        u = y.x;
        v = y.y;
    });
    const auto chunk = [&](int i) { return dir ? c1 - 1 - i : c0 + i; };
    const auto fetch = [&](int i) {
        if (i < nc) {
            const int c = chunk(i), Lc = min(C, sp.len - c * C);
            const long long row0 = sp.t0 + (long long)c * C;
            fetch_tile<Tin, DK, DK>(sA + (i & 1) * C * KP, KP, dir ? p.q : p.k, row0, p.H, h, 0, Lc);
            fetch_tile<Tin, DV, ROWS>(sB + (i & 1) * C * VP, VP, dir ? p.dO : p.v, row0, p.H, h, j0, Lc);
        }
        copies_commit();
    };
    const float2 g0 = make_float2(0.f, 0.f);
    float2 gate = g0, gate_end = g0;  // this thread's row's, and the chunk's
    const auto load_gate = [&](int i) {
        if (i >= nc || threadIdx.x >= C) return;
        const float2 *G = reinterpret_cast<const float2 *>(s.gates + ((size_t)(sp.slot + chunk(i)) * p.H + h) * GATE);
        gate = __ldg(G + threadIdx.x);
        gate_end = __ldg(G + C - 1);
    };
    float total = 1.f;
    fetch(0);
    load_gate(0);
    fetch(1);
    for (int i = 0; i < nc; ++i) {
        float *weight = sW + (i & 1) * (C + 4);  // of the rows; and what is kept of X
        if (threadIdx.x < C) {
            weight[threadIdx.x] = dir ? p.scale * hla_decay(gate, g0) : hla_decay(gate_end, gate);
            if (threadIdx.x == 0) weight[C] = hla_decay(gate_end, g0);
        }
        load_gate(i + 1);
        copies_wait<1>();
        __syncthreads();
        if (!s.ends) {
            float *dst = s.X[dir] + ((size_t)(sp.slot + chunk(i)) * p.H + h) * (size_t)(DV * DK);
            each([&](size_t at, float &u, float &v) { *reinterpret_cast<float2 *>(dst + at) = make_float2(u, v); });
        }
        const float keep = weight[C];
        total *= keep;
        if (active) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[a][j][e] *= keep;
            mm<C, 8 * WN, true, false, true>(x, w, sB + (i & 1) * C * VP, VP, sA + (i & 1) * C * KP, KP, weight);
        }
        __syncthreads();  // the tiles are consumed
        fetch(i + 2);
    }
    if (end) each([&](size_t at, float &u, float &v) { *reinterpret_cast<float2 *>(end + at) = make_float2(u, v); });
    if (s.ends && j0 == 0 && threadIdx.x == 0) s.seg.keep[dir][su * p.H + h] = total;
}

// End states of the segments -> their start states: start_0 = S0, start_{i+1} = keep_i start_i + end_i (in the
// direction's order), in place, one thread per four elements of a (sequence, head). `tokens` per segment.
__global__ void __launch_bounds__(256) hla_segment_scan_kernel(const HlaArgs p, const HlaSegments s, int tokens) {
    constexpr int U = 8;  // end states on their way at once
    const int dir = blockIdx.z, h = blockIdx.x % p.H, n = blockIdx.x / p.H;
    const int at = 4 * (blockIdx.y * 256 + threadIdx.x), size = p.dv * p.dk;
    if (at >= size) return;
    const HlaSpan sp = hla_span(p, n, tokens);
    const int nseg = max(1, sp.nch);
    const float *first = dir ? p.dST : p.S0;
    float4 x = first ? *reinterpret_cast<const float4 *>(first + ((size_t)n * p.H + h) * size + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    const auto where = [&](int i) { return (size_t)(sp.slot + (dir ? nseg - 1 - i : i)) * p.H + h; };
    for (int i0 = 0; i0 < nseg; i0 += U) {
        float4 e[U];
        float keep[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j + 1 < nseg) {  // (the last segment's end is the sequence's: it has no slot)
                e[j] = *reinterpret_cast<const float4 *>(s.state[dir] + where(i0 + j) * size + at);
                keep[j] = s.keep[dir][where(i0 + j)];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j < nseg) {
                *reinterpret_cast<float4 *>(s.state[dir] + where(i0 + j) * size + at) = x;
                if (i0 + j + 1 < nseg)
                    x = make_float4(fmaf(keep[j], x.x, e[j].x), fmaf(keep[j], x.y, e[j].y), fmaf(keep[j], x.z, e[j].z), fmaf(keep[j], x.w, e[j].w));
            }
    }
}

// ------------------------------------------------------------------ outputs
template <int DK, int DV>
struct OutSmem {
    static constexpr int KP = DK + 4, VP = DV + 8;
    // K's tile takes the state's tiles (64 rows of DK) once Q K^T is done, and then V: two CTAs to an SM
    static constexpr int T = KP > VP ? KP : VP;
    static constexpr int floats = C * KP + C * T + C * LP;
    static constexpr size_t bytes = sizeof(float) * floats + sizeof(float2) * C;
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(NT, 2) hla_out_simt_kernel(const HlaArgs p, const uint8_t *__restrict__ gates, const float *__restrict__ Sc) {
    using L = OutSmem<DK, DV>;
    constexpr int VJ = DV / 32;
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem, *sK = sQ + C * L::KP, *sV = sK, *sP = sK + C * L::T;
    float2 *G = reinterpret_cast<float2 *>(sP + C * LP);
    const int h = blockIdx.x % p.H;
    const long long slot = blockIdx.x / p.H;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    const long long row0 = sp.t0 + (long long)c * C;
    const int Lc = min(C, sp.len - c * C);
    const WarpTile w = tile_of_warp<32>();
    const bool has_state = c > 0 || p.S0 != nullptr;

    fetch_tile<Tin, DK, DK>(sQ, L::KP, p.q, row0, p.H, h, 0, Lc);
    fetch_tile<Tin, DK, DK>(sK, L::KP, p.k, row0, p.H, h, 0, Lc);
    copies_commit();
    if (threadIdx.x < C) G[threadIdx.x] = gate_of(gates, slot, p.H, h);
    copies_wait<0>();
    __syncthreads();
    {
        float a[2][2][4];
        zero(a);
        mm<DK, 32, false, true>(a, w, sQ, L::KP, sK, L::KP);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int r = w.row(i, e), s = w.col<32>(j, e);
                    *reinterpret_cast<float2 *>(sP + r * LP + s) =
                        make_float2(s <= r ? a[i][j][e] * (p.scale * hla_decay(G[r], G[s])) : 0.f, s + 1 <= r ? a[i][j][e + 1] * (p.scale * hla_decay(G[r], G[s + 1])) : 0.f);
                }
    }
    __syncthreads();  // P is written, K's tile is free
    float acc[2][VJ][4];
    zero(acc);
    if (has_state) {
        const float *S = Sc + ((size_t)slot * p.H + h) * (size_t)(DV * DK);
        constexpr int JT = DV < 64 ? DV : 64;  // rows of the state at a time
#pragma unroll
        for (int jb = 0; jb < DV / JT; ++jb) {
            fetch_state<DK>(sK, L::KP, S + (size_t)jb * JT * DK, JT);
            copies_commit();
            copies_wait<0>();
            __syncthreads();
            float part[2][JT / 32][4];
            zero(part);
            mm<DK, 32, false, true>(part, w, sQ, L::KP, sK, L::KP);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < JT / 32; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][jb * (JT / 32) + j][e] = part[i][j][e];
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float since = p.scale * hla_decay(G[w.row(i, e)], make_float2(0.f, 0.f));
#pragma unroll
                for (int j = 0; j < VJ; ++j) {
                    acc[i][j][e] *= since;
                    acc[i][j][e + 1] *= since;
                }
            }
    }
    fetch_tile<Tin, DV, DV>(sV, L::VP, p.v, row0, p.H, h, 0, Lc);
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    mm<C, 32, false, false>(acc, w, sP, LP, sV, L::VP);
    Tin *o = static_cast<Tin *>(p.o);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int r = w.row(i, e);
            if (r >= Lc) continue;
#pragma unroll
            for (int j = 0; j < VJ; ++j)
                st2(o + ((size_t)(row0 + r) * p.H + h) * DV + w.col<32>(j, e), acc[i][j][e], acc[i][j][e + 1]);
        }
}

// ---------------------------------------------------------------- gradients
template <int DK, int DV>
struct GradSmem {
    static constexpr int KP = DK + 4, VP = DV + 4, SP = DK + 8;  // (the states' tiles are read down the columns, beside rows)
    // the last tile holds the state's tiles (JB x SP each) first, then the pairs of dg; A's and dA's hold the next ones
    static constexpr int XT = (2 * JB * SP > C * LP) ? 2 * JB * SP : C * LP;
    static_assert(2 * JB * SP <= 2 * C * LP, "the states' tiles fit into A's and dA's");
    static constexpr int floats = 2 * C * KP + 2 * C * VP + 2 * C * LP + XT + 2 * 4 * C + C + 32;
    static constexpr size_t bytes = sizeof(float) * floats + sizeof(float2) * C;
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(NG) hla_grad_simt_kernel(const HlaArgs p, const uint8_t *__restrict__ gates, const float *__restrict__ Sc,
                                                           const float *__restrict__ Rc) {
    using L = GradSmem<DK, DV>;
    constexpr int KJ = DK / 32, VJ = DV / 32;
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem, *sK = sQ + C * L::KP, *sV = sK + C * L::KP, *sO = sV + C * L::VP;
    float *sA = sO + C * L::VP, *sD = sA + C * LP, *sX = sD + C * LP;
    float *sRead = sX + L::XT, *sWrit = sRead + 4 * C, *sWith = sWrit + 4 * C, *sThr = sWith + C;  // (read, written: by column warp)
    float2 *G = reinterpret_cast<float2 *>(sThr + 32);
    const int h = blockIdx.x % p.H;
    const long long slot = blockIdx.x / p.H;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    const long long row0 = sp.t0 + (long long)c * C;
    const int Lc = min(C, sp.len - c * C);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wn = warp & 3;
    const WarpTile w = tile_of_warp<16>();
    const float2 g0 = make_float2(0.f, 0.f);

    // the states' tiles come one ahead, into what the scores take later
    const size_t xb = ((size_t)slot * p.H + h) * (size_t)(DV * DK);
    constexpr int JN = DV / JB;
    const auto states = [&](int jb) {
        if (jb < JN) {
            float *to = jb & 1 ? sA : sX;
            fetch_state<DK, NG>(to, L::SP, Sc + xb + (size_t)jb * JB * DK, JB);
            fetch_state<DK, NG>(to + JB * L::SP, L::SP, Rc + xb + (size_t)jb * JB * DK, JB);
        }
        copies_commit();
    };
    fetch_tile<Tin, DK, DK, NG>(sQ, L::KP, p.q, row0, p.H, h, 0, Lc);
    fetch_tile<Tin, DK, DK, NG>(sK, L::KP, p.k, row0, p.H, h, 0, Lc);
    fetch_tile<Tin, DV, DV, NG>(sV, L::VP, p.v, row0, p.H, h, 0, Lc);
    fetch_tile<Tin, DV, DV, NG>(sO, L::VP, p.dO, row0, p.H, h, 0, Lc);
    states(0);
    states(1);
    if (threadIdx.x < C) G[threadIdx.x] = gate_of(gates, slot, p.H, h);

    // the parts that go through the states: dQ from S_in, dK and dV from R, and their terms of dg
    float dq[1][KJ][4], dk[1][KJ][4], dv[1][VJ][4];
    zero(dq);
    zero(dk);
    float thr = 0.f;
#pragma unroll
    for (int jb = 0; jb < JN; ++jb) {
        float *sS = jb & 1 ? sA : sX, *sR = sS + JB * L::SP;
        copies_wait<1>();
        __syncthreads();
        for (int idx = threadIdx.x; idx < JB * (DK / 4); idx += NG) {
            const int at = idx / (DK / 4) * L::SP + 4 * (idx % (DK / 4));
            const float4 s4 = *reinterpret_cast<const float4 *>(sS + at), r4 = *reinterpret_cast<const float4 *>(sR + at);
            thr = fmaf(s4.x, r4.x, fmaf(s4.y, r4.y, fmaf(s4.z, r4.z, fmaf(s4.w, r4.w, thr))));
        }
        mm<JB, 32, false, false>(dq, w, sO + jb * JB, L::VP, sS, L::SP);
        mm<JB, 32, false, false>(dk, w, sV + jb * JB, L::VP, sR, L::SP);
        float part[1][1][4];
        zero(part);
        mm<DK, 32, false, true>(part, w, sK, L::KP, sR, L::SP);
#pragma unroll
        for (int i = 0; i < 1; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dv[i][jb][e] = part[i][0][e];
        __syncthreads();
        states(jb + 2);
    }
#pragma unroll
    for (int i = 0; i < 1; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int r = w.row(i, e);
            const float since = p.scale * hla_decay(G[r], g0), until = hla_decay(G[C - 1], G[r]);
            float rd = 0.f, wr = 0.f;
#pragma unroll
            for (int j = 0; j < KJ; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float &a = dq[i][j][e + k], &b = dk[i][j][e + k];
                    a *= since;
                    b *= until;
                    rd = fmaf(a, sQ[r * L::KP + w.col<32>(j, e + k)], rd);
                    wr = fmaf(b, sK[r * L::KP + w.col<32>(j, e + k)], wr);
                }
#pragma unroll
            for (int j = 0; j < VJ; ++j) {
                dv[i][j][e] *= until;
                dv[i][j][e + 1] *= until;
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                rd += __shfl_xor_sync(0xffffffffu, rd, off);
                wr += __shfl_xor_sync(0xffffffffu, wr, off);
            }
            if (w.t == 0) {
                sRead[wn * C + r] = rd;
                sWrit[wn * C + r] = wr;
            }
        }
#pragma unroll
    for (int off = 16; off; off >>= 1) thr += __shfl_xor_sync(0xffffffffu, thr, off);
    if (lane == 0) sThr[warp] = thr;

    // A = scale Q K^T . D, dA = scale dO V^T . D, and the pairs within the chunk E = A . dO V^T below the diagonal
    {
        float a[1][2][4], da[1][2][4];
        zero(a);
        zero(da);
        mm<DK, 32, false, true>(a, w, sQ, L::KP, sK, L::KP);
        mm<DV, 32, false, true>(da, w, sO, L::VP, sV, L::VP);
#pragma unroll
        for (int i = 0; i < 1; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = w.row(i, e), s = w.col<32>(j, e);
                    const float d = hla_decay(G[r], G[s]);
                    const float x = s <= r ? a[i][j][e] * (p.scale * d) : 0.f;
                    sA[r * LP + s] = x;
                    sD[r * LP + s] = s <= r ? da[i][j][e] * (p.scale * d) : 0.f;
                    sX[r * LP + s] = s < r ? x * da[i][j][e] : 0.f;
                }
    }
    __syncthreads();
    mm<C, 32, false, false>(dq, w, sD, LP, sK, L::KP);
    mm<C, 32, true, false>(dk, w, sD, LP, sQ, L::KP);
    mm<C, 32, true, false>(dv, w, sA, LP, sO, L::VP);
    Tin *out_q = static_cast<Tin *>(p.dq), *out_k = static_cast<Tin *>(p.dk_), *out_v = static_cast<Tin *>(p.dv_);
#pragma unroll
    for (int i = 0; i < 1; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int r = w.row(i, e);
            if (r >= Lc) continue;
            const size_t row = (size_t)(row0 + r) * p.H + h;
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                st2(out_q + row * DK + w.col<32>(j, e), dq[i][j][e], dq[i][j][e + 1]);
                st2(out_k + row * DK + w.col<32>(j, e), dk[i][j][e], dk[i][j][e + 1]);
            }
#pragma unroll
            for (int j = 0; j < VJ; ++j) st2(out_v + row * DV + w.col<32>(j, e), dv[i][j][e], dv[i][j][e + 1]);
        }
    if (!p.dg) return;

    // dg: suffix sums of E down each column, then row sums left of the diagonal; plus the suffix sums of
    // the reads of S_in, the prefix sums of the writes that R sees, and what passes through
    if (threadIdx.x < C) {
        const int s = threadIdx.x;
        float u = 0.f;
#pragma unroll 8
        for (int r = C - 1; r >= 0; --r) {  // (E is zero on and above the diagonal)
            u += sX[r * LP + s];
            sX[r * LP + s] = u;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = ty + 32 * i;
        float u = 0.f;
        for (int s = tx; s < t; s += 16) u += sX[t * LP + s];
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
        if (tx == 0) sWith[t] = u;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // two tokens a lane
        const int t = 2 * lane;
        float rd[2], wr[2], through = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            rd[k] = (sRead[t + k] + sRead[C + t + k]) + (sRead[2 * C + t + k] + sRead[3 * C + t + k]);
            wr[k] = (sWrit[t + k] + sWrit[C + t + k]) + (sWrit[2 * C + t + k] + sWrit[3 * C + t + k]);
        }
        float after = rd[0] + rd[1], before = wr[0] + wr[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, after, off), z = __shfl_up_sync(0xffffffffu, before, off);
            if (lane + off < 32) after += y;
            if (lane >= off) before += z;
        }
        // (exclusive sums are shifted, not subtracted: a difference would lose what is small)
        float later = __shfl_down_sync(0xffffffffu, after, 1), earlier = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 31) later = 0.f;
        if (lane == 0) earlier = 0.f;
#pragma unroll
        for (int k = 0; k < NG / 32; ++k) through += sThr[k];
        through *= hla_decay(G[C - 1], g0);
        Tin *dg = static_cast<Tin *>(p.dg);
        if (t < Lc) st_elem(dg, (size_t)(row0 + t) * p.H + h, (sWith[t] + ((rd[0] + rd[1]) + later)) + (earlier + through));
        if (t + 1 < Lc) st_elem(dg, (size_t)(row0 + t + 1) * p.H + h, (sWith[t + 1] + (rd[1] + later)) + ((earlier + wr[0]) + through));
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
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: per direction the states at the chunks' borders, and, with segments, the segments' states and decays.
struct Layout {
    int sc;
    long long slots, seg_slots;
    size_t gates, X[2], seg[2], keep[2], bytes;
};
Layout layout(const HlaArgs &a, bool back) {
    Layout l{};
    const int dirs = back ? 2 : 1;
    const bool packed = a.cu_seqlens != nullptr;
    // two state CTAs run on an SM (its registers)
    l.sc = hla_segment_chunks(a, C, (long long)a.N * a.H * ((a.dv + 63) / 64) * dirs, 2LL * device_sm_count());
    l.slots = hla_slots(packed, a.N, a.T, C);
    l.seg_slots = l.sc ? hla_slots(packed, a.N, a.T, l.sc * C) : 0;
    size_t at = 0;
    const auto take = [&](size_t bytes) { const size_t x = at; at += align256(bytes); return x; };
    const size_t state = sizeof(float) * (size_t)a.H * a.dk * a.dv;
    l.gates = take((size_t)l.slots * a.H * GATE);
    for (int d = 0; d < dirs; ++d) {
        l.X[d] = take((size_t)l.slots * state);
        l.seg[d] = take((size_t)l.seg_slots * state);
        l.keep[d] = take((size_t)l.seg_slots * a.H * sizeof(float));
    }
    l.bytes = at;
    return l;
}

template <typename Tin, int DK, int DV>
cudaError_t states(const HlaArgs &a, const Layout &l, int dirs, StateArgs &s) {
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    s.a = a;
    if (dirs == 2) s.a.ST = nullptr;
    s.seg.sc = l.sc;
    s.gates = ws + l.gates;
    for (int d = 0; d < dirs; ++d) {
        s.X[d] = reinterpret_cast<float *>(ws + l.X[d]);
        s.seg.state[d] = reinterpret_cast<float *>(ws + l.seg[d]);
        s.seg.keep[d] = reinterpret_cast<float *>(ws + l.keep[d]);
    }
    using T = StateTile<DK, DV>;
    const auto kern = hla_state_simt_kernel<Tin, DK, DV>;
    static HlaSmem smem;
    cudaError_t e = smem.raise(kern, T::bytes);
    if (e != cudaSuccess) return e;
    if (l.slots > 0 && (e = launch_hla_gates<Tin, C>(a, l.slots, ws + l.gates)) != cudaSuccess) return e;
    const dim3 grid((unsigned)((l.sc ? l.seg_slots : a.N) * a.H), DV / T::ROWS, dirs);
    if (l.sc) {
        s.ends = true;
        kern<<<grid, NT, T::bytes, a.stream>>>(s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_hla_segment_scan(a, s.seg, l.sc * C, dirs)) != cudaSuccess) return e;
    }
    s.ends = false;
    kern<<<grid, NT, T::bytes, a.stream>>>(s);
    return cudaGetLastError();
}

template <typename Tin, int DK, int DV>
cudaError_t forward_t(const HlaArgs &a) {
    const Layout l = layout(a, false);
    StateArgs s{};
    cudaError_t e = states<Tin, DK, DV>(a, l, 1, s);
    if (e != cudaSuccess || l.slots == 0 || a.T == 0) return e;
    const auto kern = hla_out_simt_kernel<Tin, DK, DV>;
    constexpr size_t bytes = OutSmem<DK, DV>::bytes;
    static HlaSmem smem;
    if ((e = smem.raise(kern, bytes)) != cudaSuccess) return e;
    kern<<<(unsigned)(l.slots * a.H), NT, bytes, a.stream>>>(a, s.gates, s.X[0]);
    return cudaGetLastError();
}

template <typename Tin, int DK, int DV>
cudaError_t backward_t(const HlaArgs &a) {
    const Layout l = layout(a, true);
    StateArgs s{};
    cudaError_t e = states<Tin, DK, DV>(a, l, 2, s);
    if (e != cudaSuccess || l.slots == 0 || a.T == 0) return e;
    const auto kern = hla_grad_simt_kernel<Tin, DK, DV>;
    constexpr size_t bytes = GradSmem<DK, DV>::bytes;
    static HlaSmem smem;
    if ((e = smem.raise(kern, bytes)) != cudaSuccess) return e;
    kern<<<(unsigned)(l.slots * a.H), NG, bytes, a.stream>>>(a, s.gates, s.X[0], s.X[1]);
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

int hla_segment_chunks(const HlaArgs &a, int C_, long long chains, long long slots) {
    const long long chunks = ((long long)a.T + C_ - 1) / C_;  // of the longest sequence, at most
    const long long parts = slots / chains;                    // of each sequence
    if (parts < 2) return 0;
    const long long sc = (chunks + parts - 1) / parts;
    return 2 * sc + 6 < chunks ? (int)sc : 0;
}

cudaError_t launch_hla_segment_scan(const HlaArgs &a, const HlaSegments &s, int tokens, int dirs) {
    hla_segment_scan_kernel<<<dim3((unsigned)(a.N * a.H), (a.dk * a.dv + 1023) / 1024, dirs), 256, 0, a.stream>>>(a, s, tokens);
    return cudaGetLastError();
}

cudaError_t launch_hla_clear_outside(const HlaArgs &a) {
    const unsigned grid = (unsigned)(a.T < 1024 ? a.T : 1024);
    if (a.dtype == KDA_DTYPE_BF16) hla_clear_outside_kernel<__nv_bfloat16><<<grid, NT, 0, a.stream>>>(a);
    else hla_clear_outside_kernel<float><<<grid, NT, 0, a.stream>>>(a);
    return cudaGetLastError();
}
size_t hla_simt_workspace(const HlaArgs &a, bool back) { return layout(a, back).bytes; }
cudaError_t launch_hla_forward_simt(const HlaArgs &a) { return pass(a, false); }
cudaError_t launch_hla_backward_simt(const HlaArgs &a) { return pass(a, true); }

}  // namespace kda
