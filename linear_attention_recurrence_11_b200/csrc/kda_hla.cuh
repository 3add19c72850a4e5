// Linear attention with one decay per head, shared by its kernels:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t      (per sequence and head)
// with a scalar log-decay g_t. States are fp32 [N, H, dv, dk] (S^T row-major), as everywhere in
// the library.
//
// Chunked form. Within a chunk of C tokens, G_r = g_1 + .. + g_r from the chunk's start and
// D_rs = e^{G_r - G_s} for s <= r, 0 above the diagonal:
//   O   = scale [ (Q K^T . D) V + e^{G_r} Q S_in ],   S_out = e^{G_C} S_in + sum_s e^{G_C - G_s} k_s v_s^T
// and for the gradients, with dO' = scale dO and R the gradient of S_out:
//   dQ  = (dO' V^T . D) K    + e^{G_r} dO' S_in^T
//   dK  = (dO' V^T . D)^T Q  + e^{G_C - G_s} V R^T
//   dV  = (Q K^T . D)^T dO'  + e^{G_C - G_s} K R
//   R_in = e^{G_C} R + sum_r e^{G_r} q_r dO'_r^T
//   dg_t = sum_{r >= t > s} D_rs (q_r.k_s)(dO'_r.v_s) + sum_{r >= t} e^{G_r} q_r.(S_in dO'_r)
//          + sum_{s < t} e^{G_C - G_s} k_s.(R v_s) + e^{G_C} <S_in, R>
// (every term of dg is a pair of a write before t and a read from t on: nothing cancels).
//
// The decays are differences of cumulative sums. The sums are exact (integers of 2^-40) and kept as
// the sum of two floats, so that a difference of two nearby large values (strong decays earlier in
// the chunk) keeps its own precision: D_rs = 2^{(hi_r - hi_s) + (lo_r - lo_s)}. A g below -kMaxGate
// (-infinity among them) counts as -kMaxGate: e^-138 is zero in fp32.
#pragma once

#include <atomic>

#include "kda_internal.cuh"

namespace kda {

// A kernel's dynamic shared memory, raised once per device (one static object per kernel).
struct HlaSmem {
    std::atomic<unsigned long long> done{0};
    template <typename F>
    cudaError_t raise(F kern, size_t bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

struct HlaArgs {
    const void *q = nullptr, *k = nullptr, *v = nullptr, *g = nullptr;
    const float *S0 = nullptr;
    void *o = nullptr;
    float *ST = nullptr;
    // backward
    const void *dO = nullptr;
    const float *dST = nullptr;
    void *dq = nullptr, *dk_ = nullptr, *dv_ = nullptr, *dg = nullptr;  // dg null: not wanted
    float *dS0 = nullptr;                                               // null: not wanted
    int B = 0, T = 0, H = 0, dk = 0, dv = 0, dtype = 0;
    int gate = 0;      // KDA_HLA_GATE_*
    float scale = 1.f;
    const int32_t *cu_seqlens = nullptr;
    int N = 0;         // sequences
    void *workspace = nullptr;
    size_t workspace_bytes = 0;
    int *dev_status = nullptr;
    cudaStream_t stream = nullptr;
};

// Chunk slots. The chunk c of sequence n has a slot of its own in the workspace: n * ceil(T / C) + c
// for dense batches, and floor(cu[n] / C) + n + c for packed ones (a sequence of len tokens has
// ceil(len / C) <= floor(cu[n + 1] / C) - floor(cu[n] / C) + 1 chunks, so slots never meet, and no
// prefix sum over the sequences is needed).
inline __host__ __device__ long long hla_slots(bool packed, int N, int T, int C) {
    return packed ? (long long)T / C + N : (long long)N * ((T + C - 1) / C);
}

struct HlaSpan {
    long long t0;    // first token (row of the token-major tensors)
    int len;         // tokens
    int nch;         // chunks
    long long slot;  // slot of chunk 0
};

// The offsets are clamped to [0, T], and a sequence that would end before it begins is empty, so that whatever they are every
// row and slot stays inside. Offsets that fall over several sequences can give a row, or a slot, to two of them: then it is
// undefined which one's result it holds.
__device__ __forceinline__ HlaSpan hla_span(const HlaArgs &p, int n, int C) {
    HlaSpan s;
    if (p.cu_seqlens) {
        const int a = min(max(p.cu_seqlens[n], 0), p.T), b = min(max(p.cu_seqlens[n + 1], a), p.T);
        s.t0 = a;
        s.len = b - a;
        s.slot = a / C + n;
    } else {
        s.t0 = (long long)n * p.T;
        s.len = p.T;
        s.slot = (long long)n * ((p.T + C - 1) / C);
    }
    s.nch = (s.len + C - 1) / C;
    return s;
}

// Slot -> sequence and chunk; false for a slot without a chunk.
__device__ __forceinline__ bool hla_chunk_of(const HlaArgs &p, long long slot, int C, int &n, int &c, HlaSpan &s) {
    if (!p.cu_seqlens) {
        const int nch = (p.T + C - 1) / C;
        n = (int)(slot / nch);
        c = (int)(slot - (long long)n * nch);
        s = hla_span(p, n, C);
        return true;
    }
    int lo = 0, hi = p.N - 1;  // the last sequence whose first slot is at or before this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int a = min(max(p.cu_seqlens[mid], 0), p.T);
        if (a / C + mid <= slot) lo = mid; else hi = mid - 1;
    }
    n = lo;
    s = hla_span(p, n, C);
    c = (int)(slot - s.slot);
    return c >= 0 && c < s.nch;
}

constexpr float kMaxGate = 138.f;  // 2^-199 and 2^199

__device__ __forceinline__ float hla_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(a - b) for sums kept as two floats
__device__ __forceinline__ float hla_decay(float2 a, float2 b) { return hla_ex2((a.x - b.x) + (a.y - b.y)); }

// Bytes of a chunk's gates (kda_hla_gate.cuh): G as C times two floats, and C factors.
template <int C>
constexpr uint32_t kHlaGateBytes = C * 12;

// Segments. A chain's chunks run one after another; where there are too few chains to fill the GPU, sequences are
// cut into segments that run side by side, at the price of a pass for their end states, a scan over those, and two
// launches.
struct HlaSegments {
    int sc = 0;                                  // chunks per segment; 0: whole sequences
    float *state[2] = {nullptr, nullptr};        // per direction: [segment slot][H][dv][dk], end states, then start states
    float *keep[2] = {nullptr, nullptr};         // per direction: decay over each segment [segment slot][H]
};
// Segment slot -> sequence and segment; false for a slot without one (an empty sequence keeps one segment, which
// passes its state on).
__device__ __forceinline__ bool hla_segment_of(const HlaArgs &p, long long slot, int tokens, int &n, int &sg) {
    HlaSpan sp;
    hla_chunk_of(p, slot, tokens, n, sg, sp);
    return sg >= 0 && sg < max(1, sp.nch);
}
// Chunks per segment for `chains` chains on a GPU that runs `slots` of them at once. Both ways take as long as
// chunks in a row: the whole sequence's, or twice a segment's and about half a dozen for the scan and the launches.
// Measured cut and whole, prefill in bf16: 8 heads x 1152 tokens 29.5 and 39.1 us, x 65536 tokens 180 and 1530; 32 heads
// x 1536 tokens 47 and 61; in fp32, 8 heads x 1152 tokens 47 and 134.
int hla_segment_chunks(const HlaArgs &a, int C, long long chains, long long slots);
cudaError_t launch_hla_segment_scan(const HlaArgs &a, const HlaSegments &s, int tokens, int dirs);

// Launchers (return cudaSuccess or the launch error).
cudaError_t launch_hla_forward_simt(const HlaArgs &a);
cudaError_t launch_hla_backward_simt(const HlaArgs &a);
size_t hla_simt_workspace(const HlaArgs &a, bool back);
cudaError_t launch_hla_clear_outside(const HlaArgs &a);  // packed batches: zero gradients of rows of no sequence
// the tensor-core kernels: bf16, every head size
bool hla_tc_supported(const HlaArgs &a);
size_t hla_tc_workspace(const HlaArgs &a, bool back);
cudaError_t launch_hla_forward_tc(const HlaArgs &a);
cudaError_t launch_hla_backward_tc(const HlaArgs &a);

struct HlaDecodeArgs {
    const void *q, *k, *v, *g;
    float *S;
    void *o;
    int N, H, dk, dv, dtype, gate;
    float scale;
    cudaStream_t stream;
};
cudaError_t launch_hla_decode(const HlaDecodeArgs &a);

struct RopeArgs {
    const void *q, *k;        // k may be null
    const void *positions;    // device, int32 or int64 [B, T]; null: 0 .. T - 1 in every sequence
    const float *inv_freq;    // device [rot_dim / 2]
    void *q_out, *k_out;
    long long tokens;         // B * T
    int T, Hq, Hk, d, rot_dim;
    bool pos64, interleaved, inverse;
    float mscale;
    int dtype;
    cudaStream_t stream;
};
cudaError_t launch_rope(const RopeArgs &a);

}  // namespace kda
