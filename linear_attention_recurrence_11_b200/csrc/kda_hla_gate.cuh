// The decays of every chunk, summed once for all kernels.
#pragma once

#include "kda_hla.cuh"

namespace kda {
namespace {

// A log-decay in units of log2 as an integer of 2^-40, and a sum of them as two floats.
__device__ __forceinline__ long long hla_gate_fixed(float g) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2 e in two floats: the product keeps 48 bits
    g = fminf(fmaxf(g, -kMaxGate), kMaxGate);
    const float p = g * kHi, e = fmaf(g, kLo, fmaf(g, kHi, -p));
    return __float2ll_rn(p * 1099511627776.f) + __float2ll_rn(e * 1099511627776.f);  // 2^40
}
__device__ __forceinline__ float2 hla_gate_split(long long t) {
    const float hi = __ll2float_rn(t);                        // 24 bits
    const float lo = __ll2float_rn(t - __float2ll_rn(hi));    // the rest: a difference of integers
    return make_float2(hi * 9.094947017729282e-13f, lo * 9.094947017729282e-13f);  // 2^-40
}

// Of every (chunk slot, head): the cumulative log2-decays G[C] as two floats each, and the factors F[s] =
// 2^{G_e - G_s}, e the last of the 32 tokens that s is among. Rows behind a sequence's end decay by nothing, so that
// G[C - 1] is the whole chunk's; a NaN makes every sum from its row on one. The sums are integers: exact, and in any
// order. A token's log-decays of all heads are neighbours, a head's are H apart, so a block takes 32 heads and reads
// all its rows together; each kernel for itself, with its loads one behind the other, they took 5 us per chunk.
template <typename Tin, int C>
__global__ void __launch_bounds__(256) hla_gate_kernel(const HlaArgs p, uint8_t *__restrict__ gates) {
    constexpr int SEGS = 8, E = C / SEGS;
    constexpr int LG = 33;  // row stride: read down the columns
    __shared__ long long tot[SEGS][32];
    __shared__ int nans[SEGS][32];
    __shared__ float2 sG[C * LG];  // [token][head]
    const int groups = (p.H + 31) / 32, h0 = (int)(blockIdx.x % groups) * 32;  // (one axis: the second ends at 65535 blocks)
    const long long slot = blockIdx.x / groups;
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    const int Lc = min(C, sp.len - c * C);
    const size_t row0 = (size_t)(sp.t0 + (long long)c * C);
    const int hh = min(h0 + lane, p.H - 1);
    float g[E];
    if (p.gate == KDA_HLA_GATE_HEAD) {
        const float x = static_cast<const float *>(p.g)[hh];
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = x;
    } else {
        Tin raw[E];  // (read together: one wait for all)
#pragma unroll
        for (int e = 0; e < E; ++e) raw[e] = static_cast<const Tin *>(p.g)[(row0 + min(seg * E + e, Lc - 1)) * p.H + hh];
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = ld_elem(raw, e);
    }
    long long x[E];
    int first_nan = E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float v = seg * E + e < Lc ? g[e] : 0.f;
        if (v != v && first_nan == E) first_nan = e;
        x[e] = hla_gate_fixed(v) + (e ? x[e - 1] : 0);
    }
    tot[seg][lane] = x[E - 1];
    nans[seg][lane] = first_nan < E;
    __syncthreads();
    long long before = 0;
    bool nan_before = false;
#pragma unroll
    for (int k = 0; k < SEGS; ++k)
        if (k < seg) {
            before += tot[k][lane];
            nan_before |= nans[k][lane] != 0;
        }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float2 G = hla_gate_split(before + x[e]);
        if (nan_before || e >= first_nan) G.x = __int_as_float(0x7fffffff);
        sG[(seg * E + e) * LG + lane] = G;
    }
    __syncthreads();
    // out by heads, a warp each: 256 and 128 contiguous bytes at a time
    for (int i = seg; i < 32 && h0 + i < p.H; i += SEGS) {
        uint8_t *dst = gates + ((size_t)slot * p.H + h0 + i) * kHlaGateBytes<C>;
#pragma unroll
        for (int k = 0; k < C / 32; ++k) {
            const int s = 32 * k + lane;
            const float2 G = sG[s * LG + i];
            *reinterpret_cast<float2 *>(dst + s * 8) = G;
            *reinterpret_cast<float *>(dst + C * 8 + s * 4) = hla_decay(sG[(32 * k + 31) * LG + i], G);
        }
    }
}

template <typename Tin, int C>
cudaError_t launch_hla_gates(const HlaArgs &a, long long slots, uint8_t *gates) {
    hla_gate_kernel<Tin, C><<<(unsigned)(slots * ((a.H + 31) / 32)), 256, 0, a.stream>>>(a, gates);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kda
