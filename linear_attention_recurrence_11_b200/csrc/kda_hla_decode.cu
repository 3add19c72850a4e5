// One token of linear attention with one decay per head, for a batch of requests, states updated in
// place: S <- e^g S + k v^T, o = scale S^T q (kda_hla.cuh with chunks of one token).
//
// Bound by HBM bandwidth: every state is streamed once in and once out (2 x 64 KiB per head at
// dk = dv = 128) for 0.6 flop per byte. 8 lanes cover one contiguous state row (dk floats) with
// 128-bit streaming accesses, two rows per lane in flight, and the dot product over dk ends with three
// xor-shuffles. A CTA takes `rows` rows of dv of one (request, head): all of them when the batch alone
// fills the GPU, and fewer, down to one pass of 32, when it does not, so that a single request's
// states are read by every SM at once. Measured at dk = dv = 128: 256 requests x 96 heads 485 us (6.7 TB/s), 1 request x
// 32 heads 2.4 us.
#include "kda_hla.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kLanesPerRow = 8;
constexpr int kRowsPerPass = (kThreads / 32) * (32 / kLanesPerRow);  // 16
constexpr int kRowsInFlight = 2;

template <typename Tin, int DK>
__global__ void __launch_bounds__(kThreads) hla_decode_kernel(const HlaDecodeArgs p, int rows) {
    constexpr int F4 = DK / (4 * kLanesPerRow);  // float4 per lane per row
    const Tin *q = static_cast<const Tin *>(p.q), *k = static_cast<const Tin *>(p.k), *v = static_cast<const Tin *>(p.v);
    Tin *o = static_cast<Tin *>(p.o);
    const size_t unit = blockIdx.x;  // n * H + h
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & (kLanesPerRow - 1), rw = lane / kLanesPerRow;
    const int j0 = blockIdx.y * rows, j1 = min(p.dv, j0 + rows);
    float *Su = p.S + unit * (size_t)p.dv * DK;

    float kk[4 * F4], qq[4 * F4];
#pragma unroll
    for (int m = 0; m < F4; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * (sub + kLanesPerRow * m) + e;
            kk[4 * m + e] = ld_elem(k, unit * DK + i);
            qq[4 * m + e] = ld_elem(q, unit * DK + i);
        }
    const float g = p.gate == KDA_HLA_GATE_HEAD ? static_cast<const float *>(p.g)[unit % p.H]
                                                : ld_elem(static_cast<const Tin *>(p.g), unit);
    const float keep = expf(g);

    for (int jb = j0 + warp * (32 / kLanesPerRow) + rw; jb < j1; jb += kRowsPerPass * kRowsInFlight) {
        float4 s[kRowsInFlight][F4];
        float vj[kRowsInFlight];
        // every row of a pass exists: dv and `rows` are multiples of the 32 rows of a pass
#pragma unroll
        for (int r = 0; r < kRowsInFlight; ++r) {
            const int j = jb + r * kRowsPerPass;
            vj[r] = ld_elem(v, unit * p.dv + j);
#pragma unroll
            for (int m = 0; m < F4; ++m)
                s[r][m] = __ldcs(reinterpret_cast<const float4 *>(Su + (size_t)j * DK + 4 * (sub + kLanesPerRow * m)));
        }
#pragma unroll
        for (int r = 0; r < kRowsInFlight; ++r) {
            const int j = jb + r * kRowsPerPass;
            float acc = 0.f;
#pragma unroll
            for (int m = 0; m < F4; ++m) {
                float *x = reinterpret_cast<float *>(&s[r][m]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = fmaf(kk[4 * m + e], vj[r], keep * x[e]);
                    acc = fmaf(x[e], qq[4 * m + e], acc);
                }
                __stcs(reinterpret_cast<float4 *>(Su + (size_t)j * DK + 4 * (sub + kLanesPerRow * m)), s[r][m]);
            }
#pragma unroll
            for (int off = 1; off < kLanesPerRow; off <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
            if (sub == 0) st_elem(o, unit * p.dv + j, p.scale * acc);
        }
    }
}

template <typename Tin>
cudaError_t launch_t(const HlaDecodeArgs &a) {
    const long long units = (long long)a.N * a.H;
    int rows = a.dv;
    while (rows > 32 && units * (a.dv / rows) < 4LL * device_sm_count()) rows >>= 1;
    const dim3 grid((unsigned)units, (unsigned)(a.dv / rows));
    switch (a.dk) {
        case 32: hla_decode_kernel<Tin, 32><<<grid, kThreads, 0, a.stream>>>(a, rows); break;
        case 64: hla_decode_kernel<Tin, 64><<<grid, kThreads, 0, a.stream>>>(a, rows); break;
        case 128: hla_decode_kernel<Tin, 128><<<grid, kThreads, 0, a.stream>>>(a, rows); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_hla_decode(const HlaDecodeArgs &a) {
    return a.dtype == KDA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace kda
