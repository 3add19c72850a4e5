// Linear attention with one decay per head on the 5th-generation tensor cores (bf16 inputs, fp32
// states, every head size; 32 channels are padded to 64 by the copies' zero fill): prefill and its
// backward pass, in chunks of 128 tokens. The chunked form is in kda_hla.cuh.
//
// Two steps. The state kernel carries the state (and, for the backward pass, its gradient from the
// last chunk to the first) over the chunks and leaves each chunk's incoming one in the workspace as a
// bf16 operand tile. The tile kernels then take every (chunk, head) on its own.
//
// Roundings to bf16: the masked scores (as the operand of the second product), the states (as an
// operand; they are carried in fp32), and the results. The state's own update multiplies k v^T by a
// decay per token; that product is taken as the sum of two bf16 numbers (hi + lo, 16 bits of the 24),
// so that the fp32 state is good to about 2^-18 and not to 2^-9.
#include "kda_hla.cuh"
#include "kda_sm100.cuh"
#include "kda_tc_common.cuh"

namespace kda {
namespace {

using namespace sm100;
using tc::kWaitCycles;
using tc::mma_chain;
using tc::Opnd;
using tc::pack_bf2;

constexpr int C = 128;               // tokens per chunk
constexpr uint32_t KB = 1024;
constexpr uint32_t TILE = 16 * KB;   // 128 rows of 64 bf16 (128-byte swizzled rows)

__host__ __device__ constexpr int padded(int d) { return d < 64 ? 64 : d; }

// Bytes of one chunk's state operand: [dk / 64][dv rows][64 dk] bf16, swizzled as in shared memory.
__host__ __device__ inline size_t blob_bytes(int dkp, int dvp) { return (size_t)dkp * dvp * 2; }

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// ================================================================= states
// Direction 0: the state; a = k, b = v, row weights e^{G_C - G_s}, chunks in order, from S0 to S_T.
// Direction 1: its gradient; a = q, b = dO, row weights scale e^{G_r}, chunks from the last to the
// first, from dS_T to dS0. Per chunk X <- e^{G_C} X + b^T (w a), X [dv][dk].
struct StateArgs {
    HlaArgs a;
    uint8_t *blob[2];   // per direction: chunk operands [slot][H]
    float *seg[2];      // per direction: states of the segments [segment slot][H][dv][dk]
    float *seg_keep[2]; // per direction: decay over each segment [segment slot][H]
    int sc;             // chunks per segment; 0: whole sequences
    bool ends;          // first pass over segments: from zero, only the end states
};

// One CTA of 256 threads per chain. Thread: half a row of X (a TMEM lane is a row of dv), DKP / 2 columns held in
// registers; as a token it scales half a row of a. The operand tile of the incoming state is staged where the low
// halves go next, and leaves by a bulk store while the chunk's tiles arrive.
template <int DKP, int DVP>
struct StateSmem {
    static constexpr uint32_t B = 0, A = (DVP / 64) * TILE, LO = A + (DKP / 64) * TILE, MISC = LO + (DKP / 64) * TILE;
    static constexpr uint32_t G = MISC + 64;                  // 2 x 128 float2
    static constexpr uint32_t bytes = G + 2 * C * 8 + 1024;   // slack for 1024-byte alignment
};

template <int DKP, int DVP>
__global__ void __launch_bounds__(256, 2) hla_state_tc_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
                                                              const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b1,
                                                              const StateArgs s) {
    using L = StateSmem<DKP, DVP>;
    constexpr int NX = DKP / 2;  // columns of a thread
    const HlaArgs &p = s.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    uint64_t *bar_tma = reinterpret_cast<uint64_t *>(sm + L::MISC), *bar_mma = bar_tma + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bar_tma + 2);
    float2 *G = reinterpret_cast<float2 *>(sm + L::G);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, half = warp >> 2;
    const int dir = blockIdx.z;
    const int h = blockIdx.x % p.H;
    const long long su = blockIdx.x / p.H;  // sequence, or segment slot
    int n = (int)su, sg = 0;
    HlaSpan sp;
    if (s.sc) {
        hla_chunk_of(p, su, s.sc * C, n, sg, sp);
        if (sg < 0 || sg >= max(1, sp.nch)) return;  // (an empty sequence keeps one segment, which passes its state on)
    }
    sp = hla_span(p, n, C);
    const int nseg = s.sc ? max(1, (sp.nch + s.sc - 1) / s.sc) : 1;
    const int c0 = s.sc ? sg * s.sc : 0, c1 = s.sc ? min(sp.nch, c0 + s.sc) : sp.nch;
    const bool last = dir ? sg == 0 : sg == nseg - 1;  // the segment whose end is the sequence's
    if (s.ends && last) return;
    const size_t sbase_n = ((size_t)n * p.H + h) * (size_t)(p.dv * p.dk), sbase_s = ((size_t)su * p.H + h) * (size_t)(p.dv * p.dk);
    const float *start = s.ends ? nullptr : s.sc ? s.seg[dir] + sbase_s : dir ? p.dST : p.S0;
    if (start && !s.sc) start += sbase_n;
    float *end = s.ends ? s.seg[dir] + sbase_s : (!last ? nullptr : dir ? p.dS0 : p.ST);
    if (end && !s.ends) end += sbase_n;
    const auto chunk = [&](int i) { return dir ? c1 - 1 - i : c0 + i; };
    const int nc = c1 - c0;

    const auto issue = [&](int i) {  // one thread: the tiles of chunk i, and the next ones' way into L2
        const CUtensorMap *ta = dir ? &tm_a1 : &tm_a0, *tb = dir ? &tm_b1 : &tm_b0;
        const int tok = (int)(sp.t0 + (long long)chunk(i) * C);
        mbar_arrive_expect_tx(bar_tma, (DKP / 64 + DVP / 64) * TILE);
#pragma unroll
        for (int b = 0; b < DKP / 64; ++b) tma_load_3d(sm + L::A + b * TILE, ta, bar_tma, 64 * b, h, tok);
#pragma unroll
        for (int b = 0; b < DVP / 64; ++b) tma_load_3d(sm + L::B + b * TILE, tb, bar_tma, 64 * b, h, tok);
        if (i + 1 < nc) {
            const int next = (int)(sp.t0 + (long long)chunk(i + 1) * C);
#pragma unroll
            for (int b = 0; b < DKP / 64; ++b) tma_prefetch_l2_3d(ta, 64 * b, h, next);
#pragma unroll
            for (int b = 0; b < DVP / 64; ++b) tma_prefetch_l2_3d(tb, 64 * b, h, next);
        }
    };
    if (tid == 0) {
        mbar_init(bar_tma, 1);
        mbar_init(bar_mma, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        if (nc > 0) issue(0);
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(s_tmem, DKP);
        tmem_relinquish();
    }
    HlaGate<__nv_bfloat16, C> gate;  // warp 1: the next chunk's log-decays, read a chunk ahead
    const auto load_gate = [&](int i) {
        const int c = chunk(i);
        gate.load(p, sp.t0 + (long long)c * C, h, min(C, sp.len - c * C));
    };
    if (nc > 0 && warp == 1) {
        load_gate(0);
        hla_scan_gate(gate, G);
        if (nc > 1) load_gate(1);
    }

    const int row = 32 * quarter + lane, col = NX * half;  // this thread's row of X, and its first column
    const size_t row_off = (size_t)row * p.dk + col;
    float x[NX];
#pragma unroll
    for (int e = 0; e < NX; e += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (start && row < p.dv && col + e < p.dk) v = *reinterpret_cast<const float4 *>(start + row_off + e);
        x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t tlane = (uint32_t)(32 * quarter) << 16;

    constexpr uint32_t idesc = idesc_bf16_f32(128, DKP, 1, 1);
    // as a token: row `tok` of a, from its 16-byte piece `q0` of block `blk` on
    const int tok = tid & 127, blk = DKP == 128 ? tid >> 7 : 0, q0 = DKP == 128 ? 0 : 4 * (tid >> 7);
    uint32_t ph = 0;
    bool aborted = false, tma_open = nc > 0, mma_open = false;
    float total = 1.f;  // decay over the segment
    for (int i = 0; i < nc; ++i) {
        const int c = chunk(i), Lc = min(C, sp.len - c * C);
        const bool more = i + 1 < nc;
        if (!s.ends) {  // the state that this chunk starts from
            if (row < DVP) {
#pragma unroll
                for (int q = 0; q < NX / 8; ++q)
                    *reinterpret_cast<uint4 *>(sm + L::LO + (col >> 6) * (DVP * 128) + sw128_offset(row, (col & 63) + 8 * q)) =
                        make_uint4(pack_bf2(x[8 * q], x[8 * q + 1]), pack_bf2(x[8 * q + 2], x[8 * q + 3]),
                                   pack_bf2(x[8 * q + 4], x[8 * q + 5]), pack_bf2(x[8 * q + 6], x[8 * q + 7]));
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                bulk_store(s.blob[dir] + ((size_t)(sp.slot + c) * p.H + h) * blob_bytes(DKP, DVP), sm + L::LO, DKP * DVP * 2);
                bulk_commit();
                bulk_wait_read_all();
            }
            __syncwarp();
        }
        const float2 g0 = make_float2(0.f, 0.f), gC = G[(i & 1) * C + C - 1], gt = G[(i & 1) * C + tok];
        const float w = dir ? p.scale * hla_decay(gt, g0) : hla_decay(gC, gt), keep = hla_decay(gC, g0);
        total *= keep;
        const bool ok_t = mbar_wait_bounded(bar_tma, ph, kWaitCycles);
        tma_open = !ok_t;
        if (__syncthreads_or(!ok_t)) { aborted = true; break; }
        // a row times its weight, as hi + lo; a row behind the sequence's end is zero on both sides of the
        // product (what stands there may be anything)
        uint8_t *ra = sm + L::A + blk * TILE, *rl = sm + L::LO + blk * TILE;
        if (tok < Lc) {
#pragma unroll
            for (int q = 0; q < NX / 8; ++q) {
                const uint32_t off = sw128_offset(tok, 8 * (q0 + q));
                const uint4 v = *reinterpret_cast<const uint4 *>(ra + off);
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = w * bf_lo(in[e]), b = w * bf_hi(in[e]);
                    hi[e] = pack_bf2(a, b);
                    lo[e] = pack_bf2(a - bf_lo(hi[e]), b - bf_hi(hi[e]));
                }
                *reinterpret_cast<uint4 *>(ra + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(rl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        } else {
            const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < NX / 8; ++q) {
                const uint32_t off = sw128_offset(tok, 8 * (q0 + q));
                *reinterpret_cast<uint4 *>(ra + off) = z;
                *reinterpret_cast<uint4 *>(rl + off) = z;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int b = 0; b < DVP / 64; ++b)
                    *reinterpret_cast<uint4 *>(sm + L::B + b * TILE + sw128_offset(tok, 8 * (4 * (tid >> 7) + q))) = z;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {  // (a 64-row dv is read twice as the upper half of M: lanes that nothing reads)
            tc_fence_after();
            const Opnd Ab{sbase + L::B, true, 0, DVP == 128 ? TILE : 0u};
            mma_chain<C / 16>(tmem, Ab, Opnd{sbase + L::A, true, 0, TILE}, idesc, false);
            mma_chain<C / 16>(tmem, Ab, Opnd{sbase + L::LO, true, 0, TILE}, idesc, true);
            mma_commit(bar_mma);
        }
        __syncwarp();
        if (more && warp == 1) {
            hla_scan_gate(gate, G + ((i + 1) & 1) * C);
            if (i + 2 < nc) load_gate(i + 2);
        }
        const bool ok_m = mbar_wait_bounded(bar_mma, ph, kWaitCycles);
        mma_open = !ok_m;
        ph ^= 1u;
        tc_fence_after();
        if (ok_m) {
            if (more && tid == 0) {
                issue(i + 1);
                tma_open = true;
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < NX / 16; ++q) {
                float d[16];
                tmem_ld16(tmem + tlane + col + 16u * q, d);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) x[16 * q + e] = fmaf(keep, x[16 * q + e], d[e]);
            }
        }
        tc_fence_before();
        if (__syncthreads_or(!ok_m)) { aborted = true; break; }
    }
    if (aborted) {  // leave nothing in flight behind (the waits are bounded again)
        if (tid == 0) {
            if (p.dev_status) atomicExch(p.dev_status, (int)KDA_ERR_TIMEOUT);
            // a copy that is open was issued for the phase after the one that the MMA wait flipped to
            if (tma_open) mbar_wait_bounded(bar_tma, ph, kWaitCycles);
            if (mma_open) mbar_wait_bounded(bar_mma, ph ^ 1u, kWaitCycles);
        }
    } else if (end && row < p.dv) {
#pragma unroll
        for (int e = 0; e < NX; e += 4)
            if (col + e < p.dk) *reinterpret_cast<float4 *>(end + row_off + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        if (s.ends && tid == 0) s.seg_keep[dir][su * p.H + h] = total;
    }
    if (tid == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, DKP);
    }
}

// End states of the segments -> their start states: start_0 = S0, start_{i+1} = keep_i start_i + end_i (in the
// direction's order), in place, one thread per four elements of a (sequence, head).
__global__ void __launch_bounds__(256) hla_segment_scan_kernel(const StateArgs s) {
    constexpr int U = 8;  // end states on their way at once
    const HlaArgs &p = s.a;
    const int dir = blockIdx.z, h = blockIdx.x % p.H, n = blockIdx.x / p.H;
    const int at = 4 * (blockIdx.y * 256 + threadIdx.x), size = p.dv * p.dk;
    if (at >= size) return;
    const HlaSpan sp = hla_span(p, n, s.sc * C);
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
                e[j] = *reinterpret_cast<const float4 *>(s.seg[dir] + where(i0 + j) * size + at);
                keep[j] = s.seg_keep[dir][where(i0 + j)];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j < nseg) {
                *reinterpret_cast<float4 *>(s.seg[dir] + where(i0 + j) * size + at) = x;
                if (i0 + j + 1 < nseg)
                    x = make_float4(fmaf(keep[j], x.x, e[j].x), fmaf(keep[j], x.y, e[j].y), fmaf(keep[j], x.z, e[j].z), fmaf(keep[j], x.w, e[j].w));
            }
    }
}

// ================================================================== tiles
struct TileArgs {
    HlaArgs a;
    const uint8_t *S, *R;   // the chunks' incoming states, and the gradients of their outgoing ones
    unsigned ahead;         // CTAs that run at once: the tile this many further on is prefetched into L2
};

// ------------------------------------------------------------------ outputs
// O = scale [(Q K^T . D) V + e^{G_r} Q S]. One CTA per chunk, head and 64 columns of dv.
template <int XD>
struct OutTile {
    static constexpr uint32_t X = 0, Y = (XD / 64) * TILE, P = XD == 128 ? Y : Y + TILE;  // the scores go over K where it has room
    static constexpr uint32_t Z = P + 2 * TILE, W = Z + TILE, MISC = W + (XD / 64) * 8 * KB;
    static constexpr uint32_t G = MISC + 64;
    static constexpr uint32_t bytes = G + C * 8 + 1024;
};

template <int DKP, int DVP>
__global__ void __launch_bounds__(256, 2) hla_out_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                                                            const __grid_constant__ CUtensorMap tm_v, const TileArgs t) {
    using L = OutTile<DKP>;
    const HlaArgs &p = t.a;
    constexpr int parts = DVP / 64;
    const int z = blockIdx.x % parts;
    const unsigned u = blockIdx.x / parts;
    const long long slot = u / p.H;
    const int h = u % p.H;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    uint64_t *bar_xy = reinterpret_cast<uint64_t *>(sm + L::MISC), *bar_zw = bar_xy + 1, *bar_s = bar_xy + 2, *bar_o = bar_xy + 3;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bar_xy + 4);
    float2 *G = reinterpret_cast<float2 *>(sm + L::G);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, half = warp >> 2;
    const long long row0 = sp.t0 + (long long)c * C;
    const int Lc = min(C, sp.len - c * C);
    const bool has = p.S0 != nullptr || c > 0;  // a state that is not all zeros

    if (tid == 0) {
        mbar_init(bar_xy, 1);
        mbar_init(bar_zw, 1);
        mbar_init(bar_s, 1);
        mbar_init(bar_o, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar_xy, 2 * (DKP / 64) * TILE);
#pragma unroll
        for (int b = 0; b < DKP / 64; ++b) {
            tma_load_3d(sm + L::X + b * TILE, &tm_q, bar_xy, 64 * b, h, (int)row0);
            tma_load_3d(sm + L::Y + b * TILE, &tm_k, bar_xy, 64 * b, h, (int)row0);
        }
        mbar_arrive_expect_tx(bar_zw, TILE + (has ? (DKP / 64) * 8 * KB : 0u));
        tma_load_3d(sm + L::Z, &tm_v, bar_zw, 64 * z, h, (int)row0);
        if (has) {  // rows 64 z .. + 63 of every block of 64 dk
            const uint8_t *src = t.S + ((size_t)slot * p.H + h) * blob_bytes(DKP, DVP) + (size_t)z * 8 * KB;
#pragma unroll
            for (int b = 0; b < DKP / 64; ++b) bulk_load(sm + L::W + b * 8 * KB, src + (size_t)b * DVP * 128, 8 * KB, bar_zw);
        }
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(s_tmem, 256);
        tmem_relinquish();
    }
    if (warp == 1) hla_load_scan_gate<__nv_bfloat16, C>(p, row0, h, Lc, G);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem, tlane = (uint32_t)(32 * quarter) << 16;
    constexpr uint32_t TS = 0, T1 = 128, T2 = 192;  // scores, (scores) V, Q S

    bool ok = true;
    if (tid == 0) {
        ok = mbar_wait_bounded(bar_xy, 0, kWaitCycles);
        if (ok) {
            mma_chain<DKP / 16>(tmem + TS, Opnd{sbase + L::X, false, TILE, 0}, Opnd{sbase + L::Y, false, TILE, 0},
                                idesc_bf16_f32(128, 128, 0, 0), false);
            mma_commit(bar_s);
        }
    }
    __syncwarp();
    const bool ok_zw = mbar_wait_bounded(bar_zw, 0, kWaitCycles);
    if (tid == 0 && ok && ok_zw && has)
        mma_chain<DKP / 16>(tmem + T2, Opnd{sbase + L::X, false, TILE, 0}, Opnd{sbase + L::W, false, 8 * KB, 0},
                            idesc_bf16_f32(128, 64, 0, 0), false);
    if (Lc < C && ok_zw) {  // rows of V behind the sequence's end: zero, whatever stands there
        for (int i = tid; i < (C - Lc) * 8; i += 256)
            *reinterpret_cast<uint4 *>(sm + L::Z + sw128_offset(Lc + (i >> 3), 8 * (i & 7))) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    const bool ok_s = mbar_wait_bounded(bar_s, 0, kWaitCycles);
    tc_fence_after();

    // scores -> decayed, masked, bf16: the K-major operand of the second product
    const int r = 32 * quarter + lane;
    const float2 gr = G[r];
    if (ok_s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int s0 = 64 * half + 16 * q;
            uint32_t w[8];
            if (s0 > 32 * quarter + 31) {  // 32 rows and 16 columns that the mask leaves nothing of
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0u;
            } else {
                float v[16];
                tmem_ld16(tmem + tlane + TS + s0, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = s0 + e <= r ? v[e] * hla_decay(gr, G[s0 + e]) : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = pack_bf2(v[2 * e], v[2 * e + 1]);
            }
            uint8_t *dst = sm + L::P + half * TILE;
            *reinterpret_cast<uint4 *>(dst + sw128_offset(r, 16 * q)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(dst + sw128_offset(r, 16 * q + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    const bool bad = __syncthreads_or(!ok || !ok_zw || !ok_s);
    bool ok_o = false;
    if (!bad) {
        if (tid == 0) {
            tc_fence_after();
            mma_chain<C / 16>(tmem + T1, Opnd{sbase + L::P, false, TILE, 0}, Opnd{sbase + L::Z, true, 0, 0},
                              idesc_bf16_f32(128, 64, 0, 1), false);
            mma_commit(bar_o);
        }
        __syncwarp();
        ok_o = mbar_wait_bounded(bar_o, 0, kWaitCycles);
        tc_fence_after();
    }
    if (ok_o) {
        const float c2 = p.scale * hla_decay(gr, make_float2(0.f, 0.f));
        const int col = 64 * z + 32 * half;
        const size_t at = ((size_t)(row0 + r) * p.H + h) * p.dv + col;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v1[16], v2[16];
            tmem_ld16(tmem + tlane + T1 + 32u * half + 16u * q, v1);
            if (has) tmem_ld16(tmem + tlane + T2 + 32u * half + 16u * q, v2);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v1[e] = has ? fmaf(p.scale, v1[e], c2 * v2[e]) : p.scale * v1[e];
            if (r < Lc && col < p.dv) {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + at + 16 * q);
                dst[0] = make_uint4(pack_bf2(v1[0], v1[1]), pack_bf2(v1[2], v1[3]), pack_bf2(v1[4], v1[5]), pack_bf2(v1[6], v1[7]));
                dst[1] = make_uint4(pack_bf2(v1[8], v1[9]), pack_bf2(v1[10], v1[11]), pack_bf2(v1[12], v1[13]), pack_bf2(v1[14], v1[15]));
            }
        }
    }
    tc_fence_before();
    const bool failed = __syncthreads_or(!ok_o);
    if (failed && tid == 0) {  // leave nothing in flight behind
        if (p.dev_status) atomicExch(p.dev_status, (int)KDA_ERR_TIMEOUT);
        mbar_wait_bounded(bar_xy, 0, kWaitCycles);
        mbar_wait_bounded(bar_zw, 0, kWaitCycles);
        mma_commit(bad ? bar_o : bar_s);  // whatever products were issued (bar_s and bar_o count one arrival each)
        mbar_wait_bounded(bad ? bar_o : bar_s, bad ? 0u : 1u, kWaitCycles);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------- gradients
// All gradients of a (chunk, head), by one CTA of 512 threads. With P = Q K^T and dP = dO V^T (both [row r, column
// s], so that one decay D_rs serves both), A = scale P . D and dA = scale dP . D in bf16:
//   dQ = dA K   + scale e^{G_r} dO S      accumulators T2
//   dK = dA^T Q + e^{G_C - G_r} V R       T3
//   dV = A^T dO + e^{G_C - G_r} K R^T     T1 (dP's, once that is read)
// The product with the state comes first; the threads scale its rows in TMEM, and the other product accumulates on
// top. A and dA go over S and V, which are free by then. dg comes from row sums in fp32 (below).
template <int DKP, int DVP>
struct GradTile {
    static constexpr uint32_t QB = (DKP / 64) * TILE, VB = (DVP / 64) * TILE, SB = DKP * DVP * 2;
    static constexpr bool over = DKP == 128 && DVP == 128;
    static constexpr uint32_t Q = 0, K = QB, V = 2 * QB, O = V + VB, S = O + VB, R = S + SB;
    static constexpr uint32_t A = over ? S : R + SB, dA = over ? V : A + 2 * TILE, END = over ? R + SB : dA + 2 * TILE;
    static constexpr uint32_t G = END + 128, F = G + C * 8, RED = F + C * 4;   // RED: 3 x 4 x 128 floats, and 16
    static constexpr uint32_t bytes = RED + 12 * C * 4 + 64 + 1024;
    static_assert(bytes <= 232448, "shared memory budget");
};

template <int DKP, int DVP>
__global__ void __launch_bounds__(512, 1) hla_grad_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                                                             const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CUtensorMap tm_dk,
                                                             const __grid_constant__ CUtensorMap tm_dv, const TileArgs t) {
    using L = GradTile<DKP, DVP>;
    const HlaArgs &p = t.a;
    const long long slot = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H;
    int n, c;
    HlaSpan sp;
    if (!hla_chunk_of(p, slot, C, n, c, sp)) return;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    // loads: q k, v dO, S R; products: P, dP, dO S and V R, K R^T, dA K and dA^T Q, A^T dO
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::END);
    enum { L_QK, L_VO, L_SR, B_P, B_DP, B_SR, B_KR, B_QK, B_V, NBAR };
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + NBAR);
    float2 *G = reinterpret_cast<float2 *>(sm + L::G);
    float *F = reinterpret_cast<float *>(sm + L::F);    // 2^{G_e - G_s}, e the last of the 32 columns that s is among
    float *red = reinterpret_cast<float *>(sm + L::RED);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, grp = warp >> 2;
    const long long row0 = sp.t0 + (long long)c * C;
    const int Lc = min(C, sp.len - c * C);
    const bool hasS = p.S0 != nullptr || c > 0, hasR = p.dST != nullptr || c + 1 < sp.nch;

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) mbar_init(bars + i, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bars + L_QK, 2 * L::QB);
#pragma unroll
        for (int b = 0; b < DKP / 64; ++b) {
            tma_load_3d(sm + L::Q + b * TILE, &tm_q, bars + L_QK, 64 * b, h, (int)row0);
            tma_load_3d(sm + L::K + b * TILE, &tm_k, bars + L_QK, 64 * b, h, (int)row0);
        }
        mbar_arrive_expect_tx(bars + L_VO, 2 * L::VB);
#pragma unroll
        for (int b = 0; b < DVP / 64; ++b) {
            tma_load_3d(sm + L::V + b * TILE, &tm_v, bars + L_VO, 64 * b, h, (int)row0);
            tma_load_3d(sm + L::O + b * TILE, &tm_o, bars + L_VO, 64 * b, h, (int)row0);
        }
        mbar_arrive_expect_tx(bars + L_SR, (hasS ? L::SB : 0u) + (hasR ? L::SB : 0u));
        const size_t at = ((size_t)slot * p.H + h) * blob_bytes(DKP, DVP);
        if (hasS) bulk_load(sm + L::S, t.S + at, L::SB, bars + L_SR);
        if (hasR) bulk_load(sm + L::R, t.R + at, L::SB, bars + L_SR);
        // the tile that comes to this SM next (one CTA per SM) starts on its way from HBM now
        const unsigned nb = blockIdx.x + t.ahead;
        int n2, c2;
        HlaSpan s2;
        if (nb < gridDim.x && hla_chunk_of(p, nb / p.H, C, n2, c2, s2)) {
            const int h2 = nb % p.H, row2 = (int)(s2.t0 + (long long)c2 * C);
            const size_t at2 = ((size_t)(nb / p.H) * p.H + h2) * blob_bytes(DKP, DVP);
#pragma unroll
            for (int b = 0; b < DKP / 64; ++b) {
                tma_prefetch_l2_3d(&tm_q, 64 * b, h2, row2);
                tma_prefetch_l2_3d(&tm_k, 64 * b, h2, row2);
            }
#pragma unroll
            for (int b = 0; b < DVP / 64; ++b) {
                tma_prefetch_l2_3d(&tm_v, 64 * b, h2, row2);
                tma_prefetch_l2_3d(&tm_o, 64 * b, h2, row2);
            }
            bulk_prefetch_l2(t.S + at2, L::SB);
            bulk_prefetch_l2(t.R + at2, L::SB);
        }
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    if (warp == 1) {
        hla_load_scan_gate<__nv_bfloat16, C>(p, row0, h, Lc, G);
        __syncwarp();
#pragma unroll
        for (int s = lane; s < C; s += 32) F[s] = hla_decay(G[s | 31], G[s]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem, tlane = (uint32_t)(32 * quarter) << 16;
    constexpr uint32_t T0 = 0, T1 = 128, T2 = 256, T3 = 384;
    const int r = 32 * quarter + lane, col = 32 * grp;   // this thread's row, and its 32 columns
    const float2 g0 = make_float2(0.f, 0.f), gr = G[r];
    const auto zero16 = [&](uint32_t off) { *reinterpret_cast<uint4 *>(sm + off) = make_uint4(0, 0, 0, 0); };

    bool ok = true;
    const auto wait = [&](int b) { ok = mbar_wait_bounded(bars + b, 0, kWaitCycles) && ok; };
    if (Lc < C) {  // rows behind the sequence's end: zero in every operand, whatever stands there
        wait(L_QK);
        wait(L_VO);
        for (int i = tid; i < (C - Lc) * 8; i += 512) {
            const uint32_t off = sw128_offset(Lc + (i >> 3), 8 * (i & 7));
#pragma unroll
            for (int b = 0; b < DKP / 64; ++b) {
                zero16(L::Q + b * TILE + off);
                zero16(L::K + b * TILE + off);
            }
#pragma unroll
            for (int b = 0; b < DVP / 64; ++b) {
                zero16(L::V + b * TILE + off);
                zero16(L::O + b * TILE + off);
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
    }
    const Opnd oQ{sbase + L::Q, false, TILE, 0}, oK{sbase + L::K, false, TILE, 0}, oV{sbase + L::V, false, TILE, 0}, oO{sbase + L::O, false, TILE, 0};
    if (tid == 0) {
        wait(L_QK);
        if (ok) {
            mma_chain<DKP / 16>(tmem + T0, oQ, oK, idesc_bf16_f32(128, 128, 0, 0), false);
            mma_commit(bars + B_P);
        }
        wait(L_VO);
        if (ok) {
            mma_chain<DVP / 16>(tmem + T1, oO, oV, idesc_bf16_f32(128, 128, 0, 0), false);
            mma_commit(bars + B_DP);
        }
        wait(L_SR);
        if (ok) {  // S, R as [dv rows][dk]: dk is the result's column
            if (hasS) mma_chain<DVP / 16>(tmem + T2, oO, Opnd{sbase + L::S, true, 0, DVP * 128}, idesc_bf16_f32(128, DKP, 0, 1), false);
            if (hasR) mma_chain<DVP / 16>(tmem + T3, oV, Opnd{sbase + L::R, true, 0, DVP * 128}, idesc_bf16_f32(128, DKP, 0, 1), false);
            mma_commit(bars + B_SR);
        }
    }
    __syncwarp();
    float thr = 0.f;
    if (p.dg && hasS && hasR) {  // <S, R>
        wait(L_SR);
        if (ok) {
#pragma unroll
            for (int i = 0; i < (int)(L::SB / 16 / 512); ++i) {
                const uint32_t off = 16u * (tid + 512 * i);
                const uint4 a = *reinterpret_cast<const uint4 *>(sm + L::S + off), b = *reinterpret_cast<const uint4 *>(sm + L::R + off);
                thr = fmaf(bf_lo(a.x), bf_lo(b.x), fmaf(bf_hi(a.x), bf_hi(b.x), thr));
                thr = fmaf(bf_lo(a.y), bf_lo(b.y), fmaf(bf_hi(a.y), bf_hi(b.y), thr));
                thr = fmaf(bf_lo(a.z), bf_lo(b.z), fmaf(bf_hi(a.z), bf_hi(b.z), thr));
                thr = fmaf(bf_lo(a.w), bf_lo(b.w), fmaf(bf_hi(a.w), bf_hi(b.w), thr));
            }
        }
    }
    // A and dA of this thread's row and columns, in bf16 pairs
    uint32_t wa[16], wd[16];
    wait(B_P);
    wait(B_DP);
    tc_fence_after();
    if (col > 32 * quarter) {  // (32 columns, all behind these 32 rows)
#pragma unroll
        for (int e = 0; e < 16; ++e) wa[e] = wd[e] = 0u;
    } else if (ok && col < 32 * quarter) {
        // all columns before these rows: D_rs = 2^{G_r - G_e} 2^{G_e - G_s}, e the last of the columns. Both factors are
        // at most 1, and the second is the same for all rows: a product replaces the exponential (0.4 of the instructions)
        const float x = r < Lc ? p.scale * hla_decay(gr, G[col + 31]) : 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float a[16], d[16];
            tmem_ld16(tmem + tlane + T0 + col + 16u * q, a);
            tmem_ld16(tmem + tlane + T1 + col + 16u * q, d);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(F + col + 16 * q + e);
                const float y[4] = {x * f.x, x * f.y, x * f.z, x * f.w};
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    wa[8 * q + (e + k) / 2] = pack_bf2(y[k] * a[e + k], y[k + 1] * a[e + k + 1]);
                    wd[8 * q + (e + k) / 2] = pack_bf2(y[k] * d[e + k], y[k + 1] * d[e + k + 1]);
                }
            }
        }
    } else if (ok) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float a[16], d[16];
            tmem_ld16(tmem + tlane + T0 + col + 16u * q, a);
            tmem_ld16(tmem + tlane + T1 + col + 16u * q, d);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int s = col + 16 * q + e;
                const float x = p.scale * hla_decay(gr, G[s]);
                const bool in = s <= r && r < Lc;
                a[e] = in ? a[e] * x : 0.f;
                d[e] = in ? d[e] * x : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                wa[8 * q + e] = pack_bf2(a[2 * e], a[2 * e + 1]);
                wd[8 * q + e] = pack_bf2(d[2 * e], d[2 * e + 1]);
            }
        }
    }
    wait(B_SR);  // the products have read S and V ..
    __syncthreads();  // .. and every thread its part of S
    if (ok) {
        uint8_t *da = sm + L::A + (col >> 6) * TILE, *dd = sm + L::dA + (col >> 6) * TILE;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t off = sw128_offset(r, (col & 63) + 8 * q);
            *reinterpret_cast<uint4 *>(da + off) = make_uint4(wa[4 * q], wa[4 * q + 1], wa[4 * q + 2], wa[4 * q + 3]);
            *reinterpret_cast<uint4 *>(dd + off) = make_uint4(wd[4 * q], wd[4 * q + 1], wd[4 * q + 2], wd[4 * q + 3]);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    // the state's products scaled per row in TMEM; sums of k . dK2 on the way
    const float since = p.scale * hla_decay(gr, g0), until = hla_decay(G[C - 1], gr);
    float cs2 = 0.f, cs = 0.f, rs = 0.f;
    const auto dot16 = [&](uint32_t tile, int cl, const float (&v)[16]) {
        float x = 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint4 a = *reinterpret_cast<const uint4 *>(sm + tile + (cl >> 6) * TILE + sw128_offset(r, (cl & 63) + 8 * q));
            const uint32_t in[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) x = fmaf(bf_lo(in[e]), v[8 * q + 2 * e], fmaf(bf_hi(in[e]), v[8 * q + 2 * e + 1], x));
        }
        return x;
    };
    const auto scale_rows = [&](uint32_t T, float f) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[16];
            tmem_ld16(tmem + tlane + T + col + 16u * q, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= f;
            tmem_st16(tmem + tlane + T + col + 16u * q, v);
            if (T == T3 && p.dg) cs2 += dot16(L::K, col + 16 * q, v);
        }
        tmem_wait_st();
    };
    bool bad = __syncthreads_or(!ok);
    if (!bad) {
        if (tid == 0) {
            tc_fence_after();
            if (hasR) mma_chain<DKP / 16>(tmem + T1, oK, Opnd{sbase + L::R, false, DVP * 128, 0}, idesc_bf16_f32(128, DVP, 0, 0), false);
            mma_commit(bars + B_KR);
        }
        __syncwarp();
        tc_fence_after();
        if (hasS && col < DKP) scale_rows(T2, since);
        if (hasR && col < DKP) scale_rows(T3, until);
        tc_fence_before();
        __syncthreads();
        const Opnd aT{sbase + L::A, true, 0, TILE}, dT{sbase + L::dA, true, 0, TILE}, dN{sbase + L::dA, false, TILE, 0};
        if (tid == 0) {
            tc_fence_after();
            mma_chain<C / 16>(tmem + T2, dN, Opnd{sbase + L::K, true, 0, TILE}, idesc_bf16_f32(128, DKP, 0, 1), hasS);
            mma_chain<C / 16>(tmem + T3, dT, Opnd{sbase + L::Q, true, 0, TILE}, idesc_bf16_f32(128, DKP, 1, 1), hasR);
            mma_commit(bars + B_QK);
        }
        __syncwarp();
        wait(B_KR);
        tc_fence_after();
        if (ok && hasR && col < DVP) scale_rows(T1, until);
        tc_fence_before();
        bad = __syncthreads_or(!ok);
        if (!bad) {
            if (tid == 0) {
                tc_fence_after();
                mma_chain<C / 16>(tmem + T1, aT, Opnd{sbase + L::O, true, 0, TILE}, idesc_bf16_f32(128, DVP, 1, 1), hasR);
                mma_commit(bars + B_V);
            }
            __syncwarp();
        }
    }
    // results: staged over q, k and (dA, or v), written by tensor stores; rows of a partial chunk directly
    const auto result = [&](uint32_t T, uint32_t stage, void *out, int d, float *sum) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[16];
            const int cl = col + 16 * q;
            tmem_ld16(tmem + tlane + T + cl, v);
            tmem_wait_ld();
            if (sum && p.dg) *sum += dot16(stage, cl, v);
            const uint4 w0 = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
            const uint4 w1 = make_uint4(pack_bf2(v[8], v[9]), pack_bf2(v[10], v[11]), pack_bf2(v[12], v[13]), pack_bf2(v[14], v[15]));
            if (Lc == C) {  // (each thread replaces the elements that it alone has read)
                uint8_t *dst = sm + stage + (cl >> 6) * TILE;
                *reinterpret_cast<uint4 *>(dst + sw128_offset(r, cl & 63)) = w0;
                *reinterpret_cast<uint4 *>(dst + sw128_offset(r, (cl & 63) + 8)) = w1;
            } else if (r < Lc && cl < d) {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + ((size_t)(row0 + r) * p.H + h) * d + cl);
                dst[0] = w0;
                dst[1] = w1;
            }
        }
    };
    if (!bad) {
        wait(B_QK);
        tc_fence_after();
        if (ok && col < DKP) {
            result(T2, L::Q, p.dq, p.dk, &rs);
            result(T3, L::K, p.dk_, p.dk, &cs);
        }
        if (p.dg) {
            red[grp * C + r] = rs;
            red[(4 + grp) * C + r] = cs;
            red[(8 + grp) * C + r] = cs2;
#pragma unroll
            for (int off = 16; off; off >>= 1) thr += __shfl_xor_sync(0xffffffffu, thr, off);
            if (lane == 0) red[12 * C + warp] = thr;
        }
        fence_proxy_async_smem();
        bad = __syncthreads_or(!ok);
    }
    if (!bad) {
        if (Lc == C && tid == 0) {
#pragma unroll
            for (int b = 0; b < DKP / 64; ++b) {
                tma_store_3d(&tm_dq, sm + L::Q + b * TILE, 64 * b, h, (int)row0);
                tma_store_3d(&tm_dk, sm + L::K + b * TILE, 64 * b, h, (int)row0);
            }
            bulk_commit();
        }
        __syncwarp();
        // dg by one warp: what a token from t on reads of one before t. Within the chunk: the later rows' sums
        // q . dQ less the later columns' sums k . dK1 (pairs that both count, the diagonal among them, cancel; the
        // rows' sums hold the reads of S too); the earlier columns' k . dK2; and e^{G_C} <S, R>.
        if (p.dg && warp == 2) {
            double a[4], b[4];  // (larger terms cancel: fp64, of a few hundred numbers)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * lane + e;
                double x[3];
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    x[k] = ((double)red[(4 * k) * C + i] + (double)red[(4 * k + 1) * C + i]) + ((double)red[(4 * k + 2) * C + i] + (double)red[(4 * k + 3) * C + i]);
                a[e] = x[0] - (x[1] - x[2]);
                b[e] = x[2];
            }
            double after = (a[0] + a[1]) + (a[2] + a[3]), before = (b[0] + b[1]) + (b[2] + b[3]), fb = before, through = 0.0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double x = __shfl_down_sync(0xffffffffu, after, off), y = __shfl_up_sync(0xffffffffu, before, off);
                if (lane + off < 32) after += x;
                if (lane >= off) before += y;
            }
            fb = before - fb;
            for (int w = 0; w < 16; ++w) through += (double)red[12 * C + w];
            through *= (double)hla_decay(G[C - 1], g0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * lane + e;
                if (i < Lc) st_elem(static_cast<__nv_bfloat16 *>(p.dg), (size_t)(row0 + i) * p.H + h, (float)(after + fb + through));
                after -= a[e];
                fb += b[e];
            }
        }
        wait(B_V);
        tc_fence_after();
        const uint32_t stage = L::over ? L::dA : L::V;
        if (ok && col < DVP) result(T1, stage, p.dv_, p.dv, nullptr);
        fence_proxy_async_smem();
        bad = __syncthreads_or(!ok);
        if (!bad && Lc == C && tid == 0) {
#pragma unroll
            for (int b = 0; b < DVP / 64; ++b) tma_store_3d(&tm_dv, sm + stage + b * TILE, 64 * b, h, (int)row0);
            bulk_commit();
        }
    }
    if (tid == 0) bulk_wait_read_all();
    tc_fence_before();
    if (bad && tid == 0) {  // leave nothing in flight behind: the copies, and whatever products were issued
        if (p.dev_status) atomicExch(p.dev_status, (int)KDA_ERR_TIMEOUT);
        mbar_wait_bounded(bars + L_QK, 0, kWaitCycles);
        mbar_wait_bounded(bars + L_VO, 0, kWaitCycles);
        mbar_wait_bounded(bars + L_SR, 0, kWaitCycles);
        uint64_t *spare = bars + L_QK;  // its copies are done: a second phase, completed by the last product
        mma_commit(spare);
        mbar_wait_bounded(spare, 1, kWaitCycles);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ================================================================== host
// 3-D map over a token-major [tokens, H, d] bf16 tensor; box of 64 channels (zeros past d) and 128 tokens.
bool make_tile_map(CUtensorMap *m, const void *base, size_t tokens, int H, int d) {
    auto enc = tc::get_encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)C};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Chunks per segment (0: whole sequences). The chains run one after another; where there are too few of them to
// fill the GPU (two CTAs per SM), sequences are cut into segments that run side by side, at the price of a first
// pass for their end states.
int segment_chunks(const HlaArgs &a, int dirs) {
    const long long chains = (long long)a.N * a.H * dirs, want = 2LL * device_sm_count();
    const long long chunks = a.cu_seqlens ? (long long)a.T / C + 1 : ((long long)a.T + C - 1) / C;  // of the longest sequence, at most
    if (chains * 3 > want || chunks < 8) return 0;
    const long long total = a.cu_seqlens ? chunks * a.H * dirs : chunks * chains;
    long long sc = (total + want - 1) / want;
    if (!a.cu_seqlens) sc = (chunks + want / chains - 1) / (want / chains);  // equal parts
    return (int)(sc < 2 ? 2 : sc);
}

struct Layout {
    int sc;
    long long slots, seg_slots;
    size_t blob[2], seg[2], keep[2], bytes;
};
Layout layout(const HlaArgs &a, bool back) {
    Layout l{};
    const int dirs = back ? 2 : 1, dkp = padded(a.dk), dvp = padded(a.dv);
    const bool packed = a.cu_seqlens != nullptr;
    l.sc = segment_chunks(a, dirs);
    l.slots = hla_slots(packed, a.N, a.T, C);
    l.seg_slots = l.sc ? hla_slots(packed, a.N, a.T, l.sc * C) : 0;
    size_t at = 0;
    const auto take = [&](size_t bytes) { const size_t x = at; at += align256(bytes); return x; };
    for (int d = 0; d < dirs; ++d) {
        l.blob[d] = take((size_t)l.slots * a.H * blob_bytes(dkp, dvp));
        l.seg[d] = take((size_t)l.seg_slots * a.H * a.dk * a.dv * 4);
        l.keep[d] = take((size_t)l.seg_slots * a.H * 4);
    }
    l.bytes = at;
    return l;
}

template <typename F>
cudaError_t with_smem(F kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

struct Maps {
    CUtensorMap q, k, v, o, dq, dk, dv;
};

template <int DKP, int DVP>
cudaError_t states(const StateArgs &s0, const Maps &m, const Layout &l, int dirs) {
    const HlaArgs &a = s0.a;
    const auto kern = hla_state_tc_kernel<DKP, DVP>;
    constexpr size_t bytes = StateSmem<DKP, DVP>::bytes;
    cudaError_t e = with_smem(kern, bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((l.sc ? l.seg_slots : a.N) * a.H), 1, dirs);
    StateArgs s = s0;
    if (l.sc) {
        s.ends = true;
        kern<<<grid, 256, bytes, a.stream>>>(m.k, m.v, m.q, m.o, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        hla_segment_scan_kernel<<<dim3((unsigned)(a.N * a.H), (a.dk * a.dv + 1023) / 1024, dirs), 256, 0, a.stream>>>(s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        s.ends = false;
    }
    kern<<<grid, 256, bytes, a.stream>>>(m.k, m.v, m.q, m.o, s);
    return cudaGetLastError();
}

template <int DKP, int DVP>
cudaError_t pass_t(const HlaArgs &a, bool back) {
    const size_t tokens = (size_t)a.B * a.T;
    Maps m;
    if (!make_tile_map(&m.q, a.q, tokens, a.H, a.dk) || !make_tile_map(&m.k, a.k, tokens, a.H, a.dk) ||
        !make_tile_map(&m.v, a.v, tokens, a.H, a.dv) || !make_tile_map(&m.o, back ? a.dO : a.v, tokens, a.H, a.dv))
        return cudaErrorInvalidValue;
    if (back && (!make_tile_map(&m.dq, a.dq, tokens, a.H, a.dk) || !make_tile_map(&m.dk, a.dk_, tokens, a.H, a.dk) ||
                 !make_tile_map(&m.dv, a.dv_, tokens, a.H, a.dv)))
        return cudaErrorInvalidValue;
    const Layout l = layout(a, back);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    StateArgs s{};
    s.a = a;
    if (back) s.a.ST = nullptr;
    s.sc = l.sc;
    for (int d = 0; d < (back ? 2 : 1); ++d) {
        s.blob[d] = ws + l.blob[d];
        s.seg[d] = reinterpret_cast<float *>(ws + l.seg[d]);
        s.seg_keep[d] = reinterpret_cast<float *>(ws + l.keep[d]);
    }
    cudaError_t e = states<DKP, DVP>(s, m, l, back ? 2 : 1);
    if (e != cudaSuccess) return e;
    TileArgs t{};
    t.a = a;
    t.S = s.blob[0];
    t.R = s.blob[1];
    const unsigned units = (unsigned)(l.slots * a.H);
    if (!back) {
        const auto kern = hla_out_tc_kernel<DKP, DVP>;
        constexpr size_t bytes = OutTile<DKP>::bytes;
        if ((e = with_smem(kern, bytes)) != cudaSuccess) return e;
        kern<<<units * (DVP / 64), 256, bytes, a.stream>>>(m.q, m.k, m.v, t);
        return cudaGetLastError();
    }
    t.ahead = device_sm_count();
    const auto kern = hla_grad_tc_kernel<DKP, DVP>;
    constexpr size_t bytes = GradTile<DKP, DVP>::bytes;
    if ((e = with_smem(kern, bytes)) != cudaSuccess) return e;
    kern<<<units, 512, bytes, a.stream>>>(m.q, m.k, m.v, m.o, m.dq, m.dk, m.dv, t);
    return cudaGetLastError();
}

cudaError_t pass(const HlaArgs &a, bool back) {
    const int k = padded(a.dk), v = padded(a.dv);
    if (k == 128) return v == 128 ? pass_t<128, 128>(a, back) : pass_t<128, 64>(a, back);
    return v == 128 ? pass_t<64, 128>(a, back) : pass_t<64, 64>(a, back);
}

}  // namespace

bool hla_tc_supported(const HlaArgs &a) {
    // one tile per (chunk slot, head, slice of a result), in a 31-bit grid
    return a.dtype == KDA_DTYPE_BF16 && hla_slots(a.cu_seqlens != nullptr, a.N, a.T, C) <= 0x7fffffffLL / 2 / a.H;
}
size_t hla_tc_workspace(const HlaArgs &a, bool back) { return layout(a, back).bytes; }
cudaError_t launch_hla_forward_tc(const HlaArgs &a) { return pass(a, false); }
cudaError_t launch_hla_backward_tc(const HlaArgs &a) { return pass(a, true); }

}  // namespace kda
