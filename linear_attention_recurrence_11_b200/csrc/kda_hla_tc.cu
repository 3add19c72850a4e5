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
// decay per token; that product is taken as the sum of two bf16 numbers (hi + lo, 16 bits of the 24:
// at most 2^-16 of it is lost, where one number would lose up to 2^-8). The fp32 states and their gradients
// are off by 2.5e-6 for that, normwise; the products' own sums, by 1.2e-7.
#include "kda_hla.cuh"
#include "kda_hla_gate.cuh"
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

// 32 consecutive TMEM columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
    tmem_ld16(addr, *reinterpret_cast<float(*)[16]>(v));
    tmem_ld16(addr + 16u, *reinterpret_cast<float(*)[16]>(v + 16));
}

constexpr uint32_t GATE = kHlaGateBytes<C>;

// Masked decayed scores of one TMEM row r (in the 32 rows from R on), 16 columns at a time:
// x D_rs, D_rs = 2^{G_r - G_s} for s <= r, and 0 above. Columns that all come before these rows take D_rs as
// 2^{G_r - G_e} F_s, e the last of the 32 columns: both factors are at most 1, the second is the same for all rows, and
// a product replaces the exponential (5 instructions an element instead of 12). On the diagonal the first factor is
// 1 or more; it and F_s keep their precision as long as no sum of these 32 tokens is more than 60 away from the last one's
// (either way: a positive g grows).
struct DecayRow {
    const float2 *G;
    const float *F;
    float2 gr;
    int r, R, Lc;
    float scale;
    bool mild;  // the sums of the 32 rows are near each other
    // (by the warp of rows R ..)
    __device__ __forceinline__ DecayRow(const float2 *gates, int row, int rows, float s)
        : G(gates), F(reinterpret_cast<const float *>(gates + C)), gr(gates[row]), r(row), R(row & ~31), Lc(rows), scale(s),
          mild(__all_sync(0xffffffffu, fabsf(gr.x - gates[row | 31].x) <= 60.f)) {}
    // the decays of 16 columns, times scale; zero where masked
    __device__ __forceinline__ bool none(int col) const { return col > R + 31; }
    __device__ __forceinline__ void get(int col, float (&d)[16]) const {
        if (col < R || mild) {
            const float x = r < Lc ? scale * hla_decay(gr, G[col | 31]) : 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(F + col + e);
                d[e] = x * f.x; d[e + 1] = x * f.y; d[e + 2] = x * f.z; d[e + 3] = x * f.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) d[e] = col + e <= r && r < Lc ? scale * hla_decay(gr, G[col + e]) : 0.f;
        }
    }
    // x d with the masked elements dropped, not multiplied: they may be anything
    __device__ __forceinline__ float keep(int s, float x, float d) const { return s <= r && r < Lc ? x * d : 0.f; }
};

// ================================================================== chains
// The chunks of a sequence (or of a segment of it), one after the other, by one CTA per chain.
//   kOut:    the outputs; the state stays in the SM from chunk to chunk.
//   kStates: each chunk's incoming state as an operand tile for the gradients (or, dir 1, the gradient of its
//            outgoing state, from the last chunk to the first).
//   kEnds:   a segment's end state, from zero.
// Per chunk X <- e^{G_C} X + b^T (w a), X [dv][dk] fp32 in registers; direction 0: a = k, b = v, w = e^{G_C - G_s}, from S0
// to S_T; direction 1: a = q, b = dO, w = scale e^{G_r}, from dS_T to dS0. The increment does not depend on X, so only
// the two instructions per element of that update are serial; everything else is pipelined over the chunks:
//   warps 0-7    scale a into hi + lo; decay and mask the scores into bf16 (in TMEM)
//   warps 8-15   the state: update, operand copy; the outputs: rows of Q S scaled, result stored
//   warp 16      issues the products: Q K^T; Q S; b^T hi + b^T lo; (scores) V onto the scaled Q S
//   warp 17      the copies: a tile is requested again as soon as the last product that reads it is done
// Measured for d = 128: a chunk with outputs 3.3 us (96 heads x 8192 tokens: 210 us), 5800 clocks. By its bytes (96 KB
// copied in, 96 read and 96 written by the threads, 290 read by the products) shared memory is busy for 4500 of them, and
// every role waits for the others for a third: the operand warps 1700 to 2700 clocks (most of it for the next tiles of a and
// the gates, whose places are single), the state warps 2000, the issuing thread 2000. A chunk's states
// 2.3 us with all SMs at it (6.4 TB/s) and 1.9 us with 96, an end state 2.0 us.
enum { kOut = 0, kStates = 1, kEnds = 2 };
// 5 warpgroups launched at 96 registers a thread, 480 in all: two go down to 88, two up to 120, the last down to 64
constexpr int kChainThreads = 640;

struct ChainArgs {
    HlaArgs a;
    const uint8_t *gates;
    uint8_t *blob[2];   // kStates, per direction: chunk operands [slot][H]
    HlaSegments seg;
    const int32_t *order;  // packed batches: sequences, longest first (null: as they come)
    int h0, hn;            // heads of this launch
    unsigned *next;        // the gradients' counter of tiles, set to `first` (null: no gradients)
    unsigned first;
};

// Outputs: one tile each of a, its hi and lo halves, b, q, the state, and the outputs' staging. States: two of a, whose hi
// halves replace it, two of lo, so that a chunk is scaled while the one before is multiplied (2.0 us a chunk where one
// took 2.2), and two of b. The state before chunk i is stored from chunk i - 1's lo, which is free by then.
template <int DKP, int DVP, int kMode>
struct ChainSmem {
    static constexpr bool out = kMode == kOut;
    static constexpr uint32_t KT = (DKP / 64) * TILE, VT = (DVP / 64) * TILE;
    static constexpr int NK = out ? 1 : 2, NV = NK;  // buffers of a (and of lo), of b
    static constexpr uint32_t K = 0, HI = out ? KT : 0u, LO = 2 * KT, V = LO + NK * KT, S = V + NV * VT, Q = S + (out ? DKP * DVP * 2 : 0);
    static_assert(DKP * DVP * 2 <= KT, "a state fits into lo");
    static constexpr uint32_t O = Q + (out ? KT : 0u);             // 8 warps x 32 rows of 32 columns
    static constexpr uint32_t G = O + (out ? 16 * KB : 0u), BARS = G + 4 * GATE;  // a ring of four chunks' gates
    static constexpr uint32_t bytes = BARS + 256 + 1024;           // slack for 1024-byte alignment
    static_assert(bytes <= 232448, "shared memory budget");
};

template <int DKP, int DVP, int kMode>
__global__ void __launch_bounds__(kChainThreads, 1)
hla_chain_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_o, const ChainArgs s) {
    using L = ChainSmem<DKP, DVP, kMode>;
    constexpr int NX = DKP / 2, NO = DVP / 2;  // columns of a thread: of X, of the outputs
    const HlaArgs &p = s.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    // A barrier completes once per chunk, its phase is the chunk's parity; one that is waited for two chunks later
    // is a pair, of which a chunk takes one: a phase can only be told from the next, not from the one after.
    constexpr int NK = L::NK, NV = L::NV;
    enum { F_K, F_V = F_K + 2, F_Q = F_V + 2,   // tiles have arrived, by buffer (a's with the gates)
           D_SCALE = F_Q + 2, D_P = D_SCALE + 2, D_X, D_S, D_O, D_E,  // done: hi + lo (pair); scores; increment read; operand; Q S scaled; outputs read (pair)
           C_QK = D_E + 2, C_QS, C_PV, C_X, C_END = C_X + 2,  // products (increment: a pair)
           R_S = F_Q,                           // kStates: the operand tile has been read by its store (pair)
           NBAR = C_END + 1 };
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + NBAR);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int dir = kMode == kOut ? 0 : blockIdx.z;
    const int h = s.h0 + blockIdx.x % s.hn;
    const long long su = blockIdx.x / s.hn;  // sequence, or segment slot
    if (kMode == kStates) {
        grid_launch_dependents();  // (the gradients of another launch's heads)
        if (s.next && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) *s.next = s.first;
    }
    int n = (int)su, sg = 0;
    HlaSpan sp;
    if (s.seg.sc) {
        if (!hla_segment_of(p, su, s.seg.sc * C, n, sg)) return;
    } else if (s.order) {
        n = s.order[n];
    }
    sp = hla_span(p, n, C);
    const int nseg = s.seg.sc ? max(1, (sp.nch + s.seg.sc - 1) / s.seg.sc) : 1;
    const int c0 = s.seg.sc ? sg * s.seg.sc : 0, c1 = s.seg.sc ? min(sp.nch, c0 + s.seg.sc) : sp.nch, nc = c1 - c0;
    const bool last = dir ? sg == 0 : sg == nseg - 1;  // the segment whose end is the sequence's
    if (kMode == kEnds && last) return;
    const size_t base_n = ((size_t)n * p.H + h) * (size_t)(p.dv * p.dk), base_s = ((size_t)su * p.H + h) * (size_t)(p.dv * p.dk);
    const float *start = kMode == kEnds ? nullptr : s.seg.sc ? s.seg.state[dir] + base_s : dir ? p.dST : p.S0;
    if (start && !s.seg.sc) start += base_n;
    float *end = kMode == kEnds ? s.seg.state[dir] + base_s : (!last ? nullptr : dir ? p.dS0 : p.ST);
    if (end && kMode != kEnds) end += base_n;
    const auto chunk = [&](int i) { return dir ? c1 - 1 - i : c0 + i; };
    const auto rows_of = [&](int i) { return min(C, sp.len - chunk(i) * C); };
    const auto row_of = [&](int i) { return sp.t0 + (long long)chunk(i) * C; };
    const auto G = [&](int i) { return reinterpret_cast<const float2 *>(sm + L::G + (i & 3) * GATE); };
    const float2 g0 = make_float2(0.f, 0.f);

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) mbar_init(bars + i, i >= D_SCALE && i < C_QK ? 8 : 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 16) {
        tmem_alloc(s_tmem, kMode == kOut ? 512 : 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    // increment; outputs (of two chunks); scores, and in bf16, each half in the first half of its columns
    constexpr uint32_t TX = 0, TO = 128, TS = 384;

    bool ok = true;
    const auto wait = [&](int b, int i) {  // (by a warp that goes on or gives up as one, or by one thread)
        if (ok) ok = mbar_wait_bounded(bars + b, (uint32_t)i & 1u, kWaitCycles);
        if (warp < 16) ok = __all_sync(0xffffffffu, ok);
        return ok;
    };
    const auto wait_pair = [&](int b, int i) { return wait(b + (i & 1), i >> 1); };
    const auto wait_k = [&](int i) { return NK == 1 ? wait(F_K, i) : wait_pair(F_K, i); };
    const auto wait_v = [&](int i) { return NV == 1 ? wait(F_V, i) : wait_pair(F_V, i); };
    // buffer of chunk i
    const auto k_of = [&](int i) { return NK == 1 ? 0u : (uint32_t)(i & 1); };
    const auto v_of = [&](int i) { return NV == 1 ? 0u : (uint32_t)(i & 1); };
    // a warp's threads have done their part: their writes to shared memory and TMEM are seen by what waits on b
    const auto done = [&](int b) {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + b);
    };

    if (warp < 8) {
        // ---------------------------------------------------- operands
        regs_dec<88>();
        const int quarter = warp & 3, half = warp >> 2, R = 32 * quarter, r = R + lane;
        const uint32_t tlane = (uint32_t)R << 16;
        // as a token: row `tok` of a, from its 16-byte piece `q0` of block `blk` on
        const int tok = tid & 127, blk = DKP == 128 ? tid >> 7 : 0, q0 = DKP == 128 ? 0 : 4 * (tid >> 7);
        for (int i = 0; i < nc && ok; ++i) {
            const int Lc = rows_of(i);
            wait_k(i);
            if (NK == 1 && i > 0) wait_pair(C_X, i - 1);  // hi and lo are read (of two, since a's tile was asked for)
            if (kMode == kStates && i > 0) wait_pair(R_S, i - 1);  // and the state that lo held since
            if (Lc < C) {  // b's tile is waited for here only, so first what its buffer's load before was there for
                if (i >= NV) wait_pair(C_X, i - NV);
                wait_v(i);
            }
            if (!ok) break;
            // a row times its weight, as hi + lo; a row behind the sequence's end is zero on both sides of
            // the products (what stands there may be anything)
            const uint32_t kt = k_of(i) * L::KT;
            const uint8_t *ra = sm + L::K + kt + blk * TILE;
            uint8_t *rh = sm + L::HI + kt + blk * TILE, *rl = sm + L::LO + kt + blk * TILE;
            if (tok < Lc) {
                const float2 gt = G(i)[tok];
                const float w = dir ? p.scale * hla_decay(gt, g0) : hla_decay(G(i)[C - 1], gt);
#pragma unroll(kMode == kOut ? 1 : 2)
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
                    *reinterpret_cast<uint4 *>(rh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(rl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            } else {
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < NX / 8; ++q) {
                    const uint32_t off = sw128_offset(tok, 8 * (q0 + q));
                    *reinterpret_cast<uint4 *>(rh + off) = z;
                    *reinterpret_cast<uint4 *>(rl + off) = z;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int b = 0; b < DVP / 64; ++b)
                        *reinterpret_cast<uint4 *>(sm + L::V + v_of(i) * L::VT + b * TILE +
                                                    sw128_offset(tok, 8 * (4 * (tid >> 7) + q))) = z;
            }
            done(D_SCALE + (i & 1));
            if (kMode != kOut) continue;
            if (!wait(C_QK, i)) break;
            tc_fence_after();
            const DecayRow dr(G(i), r, Lc, p.scale);
            // (a loop of 16 columns, not unrolled: the warps' roles are long straight lines of code, and what is not
            // fetched again runs at a third of the rate)
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const int col = 64 * half + 16 * k;
                uint32_t w[8];  // bf16 pairs
                if (dr.none(col)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                } else {
                    float v[16], d[16];
                    tmem_ld16(tmem + tlane + TS + col, v);
                    dr.get(col, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_bf2(dr.keep(col + 2 * e, v[2 * e], d[2 * e]), dr.keep(col + 2 * e + 1, v[2 * e + 1], d[2 * e + 1]));
                }
                tmem_st8(tmem + tlane + TS + 64u * half + 8u * k, w);
            }
            tmem_wait_st();
            done(D_P);
        }
    } else if (warp < 16) {
        // ------------------------------------------------- state, outputs
        regs_inc<120>();
        const int quarter = warp & 3, half = (warp >> 2) & 1, r = 32 * quarter + lane, col = NX * half;
        const uint32_t tlane = (uint32_t)(32 * quarter) << 16;
        const size_t row_off = (size_t)r * p.dk + col;
        float x[NX];  // row r of X (dv), columns from col on
#pragma unroll
        for (int e = 0; e < NX; e += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (start && r < p.dv && col + e < p.dk) v = *reinterpret_cast<const float4 *>(start + row_off + e);
            x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
        }
        const auto operand = [&](uint32_t to) {  // X in bf16, as a K-major tile of dv rows
            if (r < DVP) {
#pragma unroll
                for (int q = 0; q < NX / 8; ++q)
                    *reinterpret_cast<uint4 *>(sm + to + (col >> 6) * (DVP * 128) + sw128_offset(r, (col & 63) + 8 * q)) =
                        make_uint4(pack_bf2(x[8 * q], x[8 * q + 1]), pack_bf2(x[8 * q + 2], x[8 * q + 3]),
                                   pack_bf2(x[8 * q + 4], x[8 * q + 5]), pack_bf2(x[8 * q + 6], x[8 * q + 7]));
            }
        };
        if (kMode == kOut && nc > 0) {
            operand(L::S);
            done(D_S);
        }
        float total = 1.f;  // decay over the chain
        for (int i = 0; i < nc && ok; ++i) {
            if (kMode == kStates) {
                const uint32_t at = L::LO + ((i + 1) & 1) * L::KT;
                operand(at);
                done(D_S);
                if (wait(D_S, i) && tid == 256) {
                    bulk_store(s.blob[dir] + ((size_t)(sp.slot + chunk(i)) * p.H + h) * blob_bytes(DKP, DVP), sm + at, DKP * DVP * 2);
                    bulk_commit();
                    bulk_wait_read_all();  // (the increment is not there yet)
                    mbar_arrive(bars + R_S + (i & 1));
                }
                __syncwarp();
            }
            const int oc = NO * half;
            if (kMode == kOut) {
                if (!wait(C_QS, i)) break;
                tc_fence_after();
                const float since = p.scale * hla_decay(G(i)[r], g0);
                const uint32_t to = tmem + tlane + TO + 128u * (i & 1) + oc;
#pragma unroll 1
                for (int q = 0; q < NO / 16; ++q) {
                    float v[16];
                    tmem_ld16(to + 16u * q, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] *= since;
                    tmem_st16(to + 16u * q, v);
                }
                tmem_wait_st();
                done(D_O);
            }
            if (!wait_pair(C_X, i)) break;
            tc_fence_after();
            const float keep = hla_decay(G(i)[C - 1], g0);
            total *= keep;
#pragma unroll
            for (int q = 0; q < NX / 16; ++q) {
                float d[16];
                tmem_ld16(tmem + tlane + TX + col + 16u * q, d);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) x[16 * q + e] = fmaf(keep, x[16 * q + e], d[e]);
            }
            done(D_X);
            if (kMode != kOut) continue;
            if (i + 1 < nc) {
                operand(L::S);
                done(D_S);
            }
            if (!wait(C_PV, i)) break;
            tc_fence_after();
            // a full chunk leaves through a staging tile of the warp's 32 rows and 32 columns at a time (64-byte
            // swizzled rows) by tensor stores; a partial one directly: one 16-byte piece per row and instruction, which
            // costs the LSU four times the full tile's
            const int Lc = rows_of(i);
            uint8_t *stage = sm + L::O + (warp - 8) * 2 * KB;
#pragma unroll 1
            for (int k = 0; k < NO / 32; ++k) {
                const int c = oc + 32 * k;
                float v[32];
                tmem_ld32(tmem + tlane + TO + 128u * (i & 1) + c, v);
                tmem_wait_ld();
                uint4 w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = make_uint4(pack_bf2(v[8 * e], v[8 * e + 1]), pack_bf2(v[8 * e + 2], v[8 * e + 3]),
                                      pack_bf2(v[8 * e + 4], v[8 * e + 5]), pack_bf2(v[8 * e + 6], v[8 * e + 7]));
                if (Lc == C) {
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(stage + 64 * lane + 16 * (e ^ ((lane >> 1) & 3))) = w[e];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && c < p.dv) {
                        tma_store_3d(&tm_o, stage, c, h, (int)(row_of(i) + 32 * quarter));
                        bulk_commit();
                    }
                    __syncwarp();
                } else if (r < Lc && c < p.dv) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + ((size_t)(row_of(i) + r) * p.H + h) * p.dv + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[e] = w[e];
                }
            }
            done(D_E + (i & 1));
        }
        if (ok && end && r < p.dv) {
#pragma unroll
            for (int e = 0; e < NX; e += 4)
                if (col + e < p.dk) *reinterpret_cast<float4 *>(end + row_off + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
        if (kMode == kEnds && ok && tid == 256) s.seg.keep[dir][su * p.H + h] = total;
        if (kMode != kEnds && lane == 0) bulk_wait_read_all();
    } else {
        regs_dec<64>();
        if (warp == 16 && lane == 0) {
            // ------------------------------------------------- products
            const Opnd oQ{sbase + L::Q, false, TILE, 0}, oK{sbase + L::K, false, TILE, 0}, oS{sbase + L::S, false, DVP * 128, 0};
            constexpr uint32_t idX = idesc_bf16_f32(128, DKP, 1, 1), idS = idesc_bf16_f32(128, 128, 0, 0), idO = idesc_bf16_f32(128, DVP, 0, 0),
                               idP = idesc_bf16_f32(128, DVP, 0, 1);
            for (int i = 0; i < nc && ok; ++i) {
                if (kMode == kOut) {
                    wait(F_K, i);
                    wait(F_Q, i);
                    if (i > 0) wait(C_PV, i - 1);  // the bf16 scores before, which these replace, are read
                    if (!ok) break;
                    tc_fence_after();
                    mma_chain<DKP / 16>(tmem + TS, oQ, oK, idS, false);
                    mma_commit(bars + C_QK);
                    wait(D_S, i);
                    if (i > 1) wait_pair(D_E, i - 2);
                    if (!ok) break;
                    tc_fence_after();
                    mma_chain<DKP / 16>(tmem + TO + 128u * (i & 1), oQ, oS, idO, false);
                    mma_commit(bars + C_QS);
                }
                wait_pair(D_SCALE, i);
                wait_v(i);
                if (i > 0) wait(D_X, i - 1);
                if (!ok) break;
                tc_fence_after();
                // (a 64-row dv is read twice as the upper half of M: lanes that nothing reads)
                const uint32_t kt = k_of(i) * L::KT, vb = sbase + L::V + v_of(i) * L::VT;
                const Opnd oVt{vb, true, 0, DVP == 128 ? TILE : 0u};
                mma_chain<C / 16>(tmem + TX, oVt, Opnd{sbase + L::HI + kt, true, 0, TILE}, idX, false);
                mma_chain<C / 16>(tmem + TX, oVt, Opnd{sbase + L::LO + kt, true, 0, TILE}, idX, true);
                mma_commit(bars + C_X + (i & 1));
                if (kMode == kOut) {
                    wait(D_P, i);
                    if (!wait(D_O, i)) break;
                    tc_fence_after();
                    const uint64_t dV = smem_desc_sw128(vb, TILE, 1024u);
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        mma_bf16_ts(tmem + TO + 128u * (i & 1), tmem + TS + 64u * (k >> 2) + 8u * (k & 3), dV + (uint64_t)((k * 2048u) >> 4), idP, 1u);
                    mma_commit(bars + C_PV);
                }
            }
            mma_commit(bars + C_END);  // nothing may be in flight when TMEM is freed
            ok = mbar_wait_bounded(bars + C_END, 0, kWaitCycles) && ok;
        } else if (warp == 17 && lane == 0) {
            // --------------------------------------------------- copies
            const CUtensorMap *ta = dir ? &tm_q : &tm_k, *tb = dir ? &tm_o : &tm_v;
            int nk = 0, nq = 0, nv = 0;  // loads issued
            for (int i = 0; i < nc && ok; ++i) {
                const int tok = (int)row_of(i);
                const uint32_t kb = k_of(i), vb = v_of(i);
                if (kMode == kOut) {
                    if (i > 0) {
                        wait_pair(D_SCALE, i - 1);
                        wait(C_QK, i - 1);
                    }
                } else if (i > 1) {
                    wait_pair(C_X, i - 2);
                }
                // (The gates' ring: what reads chunk i - 4's was done before D_O of chunk i - 2, which came before Q K^T of
                // chunk i - 1; or, without outputs, before D_X of chunk i - 3, which came before the increment of chunk i - 2.)
                if (!ok) break;
                mbar_arrive_expect_tx(bars + F_K + kb, L::KT + GATE);
                ++nk;
                bulk_load(sm + L::G + (i & 3) * GATE, s.gates + ((size_t)(sp.slot + chunk(i)) * p.H + h) * GATE, GATE, bars + F_K + kb);
#pragma unroll
                for (int b = 0; b < DKP / 64; ++b) {
                    tma_load_3d(sm + L::K + kb * L::KT + b * TILE, ta, bars + F_K + kb, 64 * b, h, tok);
                }
                if (kMode == kOut) {
                    if (i > 0 && !wait(C_QS, i - 1)) break;
                    mbar_arrive_expect_tx(bars + F_Q, L::KT);
                    ++nq;
#pragma unroll
                    for (int b = 0; b < DKP / 64; ++b) {
                        tma_load_3d(sm + L::Q + b * TILE, &tm_q, bars + F_Q, 64 * b, h, tok);
                    }
                    if (i > 0 && !wait(C_PV, i - 1)) break;  // (and the products before it)
                }
                mbar_arrive_expect_tx(bars + F_V + vb, L::VT);
                ++nv;
#pragma unroll
                for (int b = 0; b < DVP / 64; ++b) {
                    tma_load_3d(sm + L::V + vb * L::VT + b * TILE, tb, bars + F_V + vb, 64 * b, h, tok);
                }
            }
            // nothing may be in flight when the CTA ends: the last loads into each buffer (bounded)
            const auto drain = [&](int b, int buffers, int issued) {
                for (int st = 0; st < buffers; ++st) {
                    const int of = buffers == 1 ? issued : (issued + 1 - st) / 2;  // loads into this buffer
                    if (of > 0) mbar_wait_bounded(bars + b + st, (uint32_t)(of - 1) & 1u, kWaitCycles);
                }
            };
            drain(F_K, NK, nk);
            drain(F_V, NV, nv);
            if (nq > 0) mbar_wait_bounded(bars + F_Q, (uint32_t)(nq - 1) & 1u, kWaitCycles);
        }
        __syncwarp();
    }
    if (!ok && p.dev_status) atomicExch(p.dev_status, (int)KDA_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, kMode == kOut ? 512 : 128);
    }
}

// =============================================================== gradients
struct TileArgs {
    HlaArgs a;
    const uint8_t *gates;
    const uint8_t *S, *R;   // the chunks' incoming states, and the gradients of their outgoing ones
    unsigned tiles;         // chunk slots x heads
    unsigned split;         // of which these, of heads 0 .. h1 - 1, come first; the others' states may still be under way
    int h1;
    unsigned *next;         // the next tile that no CTA has taken
};

// All gradients of a (chunk, head), by 512 threads; one CTA per SM, which takes tiles from a counter, with the next
// one's copies under way: q and k as soon as their products are done, the rest as the places fall free. With P = Q K^T and dP = dO V^T (both [row r, column
// s], so that one decay D_rs serves both), A = scale P . D and dA = scale dP . D in bf16:
//   dQ = dA K   + scale e^{G_r} dO S      accumulators T2
//   dK = dA^T Q + e^{G_C - G_r} V R       T3
//   dV = A^T dO + e^{G_C - G_r} K R^T     T1 (dP's, once that is read)
// The product with the state comes first; the threads scale its rows in TMEM, and the other product accumulates on
// top. A and dA go over S and V, which are free by then. dg_t is a sum over pairs of a write before t and a read from t
// on, and of nothing else (an earlier form took all of q . dQ less all of k . dK, whose pairs on one side of t cancel but for
// their roundings: from g = -10 down those were larger than what was left). The pairs within the chunk E = A . dP, in fp32,
// are summed where the scores are masked, a warp's 32 x 32 block to its rows' and columns' sums; the reads of S (rows of
// q . dQ2) and what R sees of the writes (k . dK2) while those products are scaled.
// (The pairs' sums take 10 us of 687 for 96 heads x 8192 tokens; held back until the products of dQ and dK run, whose time
// they would share, they cost spills and 70 us.)
// Measured for d = 128: 10.0 us a tile, 74 heads x 8192 tokens 319 us (4.3 TB/s of its 288 KB a tile; 6.6 us at the rate
// of a copy). The phases of a tile follow each other; warps of their own for copies, products and results took longer.
template <int DKP, int DVP>
struct GradTile {
    static constexpr uint32_t QB = (DKP / 64) * TILE, VB = (DVP / 64) * TILE, SB = DKP * DVP * 2;
    static constexpr bool over = DKP == 128 && DVP == 128;
    static constexpr uint32_t Q = 0, K = QB, V = 2 * QB, O = V + VB, S = O + VB, R = S + SB;
    static constexpr uint32_t A = over ? S : R + SB, dA = over ? V : A + 2 * TILE, END = over ? R + SB : dA + 2 * TILE;
    // the results' staging: where nothing is read any more by then, and not over q and k, whose next tiles come first
    static constexpr uint32_t stQ = over ? R : S, stK = dA, stV = A;
    static constexpr uint32_t G = END + 128, RED = G + 2 * GATE;
    // RED, in floats: per column warp the reads and the writes of each token; sums of the pairs E over blocks of 32 x 32
    // below the diagonal, of a row ([column block][row]) and of a column ([row block - 1][column]); in the blocks on the
    // diagonal the pairs across each token; and each warp's part of <S, R>
    static constexpr int READS = 0, WRITES = 4 * C, ROWS = 8 * C, COLS = 11 * C, DIAG = 14 * C, THR = 15 * C;
    static constexpr uint32_t bytes = RED + (THR + 16) * 4 + 1024;
    static_assert(bytes <= 232448, "shared memory budget");
    static_assert(over || QB <= 2 * SB, "dQ is staged over S and R");
};

// Sums over a warp's lanes of 16 values each: lane l gets that of value l / 2.
__device__ __forceinline__ float lane_sums(float (&x)[16], int lane) {
#pragma unroll
    for (int n = 8; n >= 1; n >>= 1) {  // the lanes of either half keep half of the values
        const bool upper = lane & (2 * n);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[i + n], 2 * n);
            x[i] = (upper ? x[i + n] : x[i]) + other;
        }
    }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

template <int DKP, int DVP>
__global__ void __launch_bounds__(512, 1) hla_grad_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                                                             const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CUtensorMap tm_dk,
                                                             const __grid_constant__ CUtensorMap tm_dv, const TileArgs t) {
    using L = GradTile<DKP, DVP>;
    const HlaArgs &p = t.a;
    struct Tile {
        long long slot, row0;
        int h, Lc;
        bool hasS, hasR;
    };
    // tile i; false for one without a chunk
    const auto tile = [&](unsigned i, Tile &x) {
        int n, c;
        HlaSpan sp;
        const unsigned j = i < t.split ? i : i - t.split, heads = i < t.split ? t.h1 : p.H - t.h1;
        x.slot = j / heads;
        if (!hla_chunk_of(p, x.slot, C, n, c, sp)) return false;
        x.h = (i < t.split ? 0 : t.h1) + j % heads;
        x.row0 = sp.t0 + (long long)c * C;
        x.Lc = min(C, sp.len - c * C);
        x.hasS = p.S0 != nullptr || c > 0;
        x.hasR = p.dST != nullptr || c + 1 < sp.nch;
        return true;
    };
    // (by one thread) i, if it has a chunk, or else the next one taken that has
    const auto settle = [&](unsigned i) {
        for (Tile x; i < t.tiles && !tile(i, x);) i = atomicAdd(t.next, 1u);
        return i;
    };
    __shared__ unsigned s_tile[2];  // the next tile, by parity
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sm);
    // loads: q k, v dO, S R; products: P, dP, dO S and V R, K R^T, dA K and dA^T Q, A^T dO. One phase per tile.
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::END);
    enum { L_QK, L_VO, L_SR, B_P, B_DP, B_SR, B_KR, B_QK, B_V, B_END, NBAR };
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + NBAR);
    float *red = reinterpret_cast<float *>(sm + L::RED);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, grp = warp >> 2;
    const bool issuer = tid == 0, copier = tid == 96;  // the threads that issue the products, and the copies
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) mbar_init(bars + i, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    if (tid == 64) {
        s_tile[1] = settle(blockIdx.x);
        s_tile[0] = settle(atomicAdd(t.next, 1u));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem, tlane = (uint32_t)(32 * quarter) << 16;
    constexpr uint32_t T0 = 0, T1 = 128, T2 = 256, T3 = 384;
    const int r = 32 * quarter + lane, col = 32 * grp;   // this thread's row, and its 32 columns
    const float2 g0 = make_float2(0.f, 0.f);

    // the copier's loads of tile x, the it-th of this CTA
    int loads[3] = {0, 0, 0};
    const auto load_qk = [&](const Tile &x, int it) {
        mbar_arrive_expect_tx(bars + L_QK, 2 * L::QB + GATE);
        ++loads[0];
        bulk_load(sm + L::G + (it & 1) * GATE, t.gates + ((size_t)x.slot * p.H + x.h) * GATE, GATE, bars + L_QK);
#pragma unroll
        for (int b = 0; b < DKP / 64; ++b) {
            tma_load_3d(sm + L::Q + b * TILE, &tm_q, bars + L_QK, 64 * b, x.h, (int)x.row0);
            tma_load_3d(sm + L::K + b * TILE, &tm_k, bars + L_QK, 64 * b, x.h, (int)x.row0);
        }
    };
    const auto load_o = [&](const Tile &x) {
        mbar_arrive_expect_tx(bars + L_VO, 2 * L::VB);
        ++loads[1];
#pragma unroll
        for (int b = 0; b < DVP / 64; ++b) tma_load_3d(sm + L::O + b * TILE, &tm_o, bars + L_VO, 64 * b, x.h, (int)x.row0);
    };
    const auto load_vsr = [&](const Tile &x) {
#pragma unroll
        for (int b = 0; b < DVP / 64; ++b) tma_load_3d(sm + L::V + b * TILE, &tm_v, bars + L_VO, 64 * b, x.h, (int)x.row0);
        mbar_arrive_expect_tx(bars + L_SR, (x.hasS ? L::SB : 0u) + (x.hasR ? L::SB : 0u));
        ++loads[2];
        const size_t at = ((size_t)x.slot * p.H + x.h) * blob_bytes(DKP, DVP);
        if (x.hasS) bulk_load(sm + L::S, t.S + at, L::SB, bars + L_SR);
        if (x.hasR) bulk_load(sm + L::R, t.R + at, L::SB, bars + L_SR);
    };
    const auto prefetch = [&](const Tile &x) {
        const size_t at = ((size_t)x.slot * p.H + x.h) * blob_bytes(DKP, DVP);
#pragma unroll
        for (int b = 0; b < DKP / 64; ++b) {
            tma_prefetch_l2_3d(&tm_q, 64 * b, x.h, (int)x.row0);
            tma_prefetch_l2_3d(&tm_k, 64 * b, x.h, (int)x.row0);
        }
#pragma unroll
        for (int b = 0; b < DVP / 64; ++b) {
            tma_prefetch_l2_3d(&tm_v, 64 * b, x.h, (int)x.row0);
            tma_prefetch_l2_3d(&tm_o, 64 * b, x.h, (int)x.row0);
        }
        if (x.hasS) bulk_prefetch_l2(t.S + at, L::SB);
        if (x.hasR) bulk_prefetch_l2(t.R + at, L::SB);
    };
    Tile cur;
    bool more = s_tile[1] < t.tiles;
    if (more) {
        if (s_tile[1] >= t.split) grid_dependency_wait();
        tile(s_tile[1], cur);
    }
    if (copier && more) {
        load_qk(cur, 0);
        load_o(cur);
        load_vsr(cur);
    }
    __syncwarp();

    const Opnd oQ{sbase + L::Q, false, TILE, 0}, oK{sbase + L::K, false, TILE, 0}, oV{sbase + L::V, false, TILE, 0}, oO{sbase + L::O, false, TILE, 0};
    const auto zero16 = [&](uint32_t off) { *reinterpret_cast<uint4 *>(sm + off) = make_uint4(0, 0, 0, 0); };
    bool bad = false;
    for (int it = 0; more; ++it) {
        const uint32_t ph = it & 1;
        Tile nxt = cur;
        const unsigned ni = s_tile[ph];
        more = ni < t.tiles;
        if (more) {
            if (ni >= t.split) grid_dependency_wait();
            tile(ni, nxt);
        }
        unsigned after = 0;  // the tile after the next: taken here, looked at when it has arrived
        if (tid == 64) after = more ? atomicAdd(t.next, 1u) : t.tiles;
        const int Lc = cur.Lc;
        const bool hasS = cur.hasS, hasR = cur.hasR;
        const float2 *G = reinterpret_cast<const float2 *>(sm + L::G + ph * GATE);
        bool ok = true;
        const auto wait = [&](int b) { ok = ok && mbar_wait_bounded(bars + b, ph, kWaitCycles); };
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
        if (issuer) {
            wait(L_QK);
            if (ok) {
                tc_fence_after();
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
        if (copier && more) prefetch(nxt);  // the next tile on its way into L2
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
        wait(L_QK);  // (the gates came with q and k)
        wait(B_P);
        wait(B_DP);
        ok = __all_sync(0xffffffffu, ok);  // (the warp's lanes exchange sums)
        tc_fence_after();
        const float2 gr = G[r];
        const DecayRow dr(G, r, Lc, p.scale);
        if (dr.none(col)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) wa[e] = wd[e] = 0u;
        } else if (ok) {
            const bool diagonal = grp == quarter;
            float across = 0.f;  // of this row, the pairs with the columns so far
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float a[16], d[16], f[16];
                tmem_ld16(tmem + tlane + T0 + col + 16u * q, a);
                tmem_ld16(tmem + tlane + T1 + col + 16u * q, d);
                dr.get(col + 16 * q, f);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = col + 16 * q + 2 * e;
                    wa[8 * q + e] = pack_bf2(dr.keep(c, a[2 * e], f[2 * e]), dr.keep(c + 1, a[2 * e + 1], f[2 * e + 1]));
                    wd[8 * q + e] = pack_bf2(dr.keep(c, d[2 * e], f[2 * e]), dr.keep(c + 1, d[2 * e + 1], f[2 * e + 1]));
                }
                if (p.dg) {
                    // over the rows: a column's pairs, or (diagonal) those of rows from a token on with columns before it.
                    // (Rows behind the end are zero on both sides of both products.)
                    if (diagonal) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int c = col + 16 * q + e;
                            const float pair = a[e] * f[e] * d[e];
                            a[e] = c <= r ? across : 0.f;
                            across += c < r ? pair : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            a[e] = a[e] * f[e] * d[e];
                            across += a[e];
                        }
                    }
                    const float x = lane_sums(a, lane);
                    if (!(lane & 1)) red[(diagonal ? L::DIAG : L::COLS + (quarter - 1) * C) + col + 16 * q + (lane >> 1)] = x;
                }
            }
            if (p.dg && !diagonal) red[L::ROWS + grp * C + r] = across;
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
        // the state's products scaled per row in TMEM; sums of q . dQ2 and k . dK2 on the way
        const float since = p.scale * hla_decay(gr, g0), until = hla_decay(G[C - 1], gr);
        float reads = 0.f, writes = 0.f;
        const auto dot16 = [&](uint32_t tile, int cl, const float *v) {
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
        const auto load32 = [&](uint32_t T, float (&v)[32]) {
            tmem_ld16(tmem + tlane + T + col, *reinterpret_cast<float(*)[16]>(v));
            tmem_ld16(tmem + tlane + T + col + 16u, *reinterpret_cast<float(*)[16]>(v + 16));
            tmem_wait_ld();
        };
        const auto scale_rows = [&](uint32_t T, float f) {
            float v[32];
            load32(T, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= f;
            tmem_st16(tmem + tlane + T + col, *reinterpret_cast<float(*)[16]>(v));
            tmem_st16(tmem + tlane + T + col + 16u, *reinterpret_cast<float(*)[16]>(v + 16));
            if (T == T2 && p.dg) reads = dot16(L::Q, col, v) + dot16(L::Q, col + 16, v + 16);
            if (T == T3 && p.dg) writes = dot16(L::K, col, v) + dot16(L::K, col + 16, v + 16);
            tmem_wait_st();
        };
        bad = __syncthreads_or(!ok);
        if (bad) break;
        if (issuer) {
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
        if (issuer) {
            tc_fence_after();
            mma_chain<C / 16>(tmem + T2, Opnd{sbase + L::dA, false, TILE, 0}, Opnd{sbase + L::K, true, 0, TILE}, idesc_bf16_f32(128, DKP, 0, 1), hasS);
            mma_chain<C / 16>(tmem + T3, Opnd{sbase + L::dA, true, 0, TILE}, Opnd{sbase + L::Q, true, 0, TILE}, idesc_bf16_f32(128, DKP, 1, 1), hasR);
            mma_commit(bars + B_QK);
        }
        __syncwarp();
        wait(B_KR);
        tc_fence_after();
        if (ok && hasR && col < DVP) scale_rows(T1, until);
        tc_fence_before();
        bad = __syncthreads_or(!ok);
        if (bad) break;
        if (issuer) {
            tc_fence_after();
            mma_chain<C / 16>(tmem + T1, Opnd{sbase + L::A, true, 0, TILE}, Opnd{sbase + L::O, true, 0, TILE}, idesc_bf16_f32(128, DVP, 1, 1), hasR);
            mma_commit(bars + B_V);
        }
        __syncwarp();
        // results: staged and written by tensor stores; rows of a partial chunk directly
        const auto result = [&](uint32_t T, uint32_t stage, void *out, int d) {
            float v[32];
            load32(T, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 w = make_uint4(pack_bf2(v[8 * q], v[8 * q + 1]), pack_bf2(v[8 * q + 2], v[8 * q + 3]),
                                           pack_bf2(v[8 * q + 4], v[8 * q + 5]), pack_bf2(v[8 * q + 6], v[8 * q + 7]));
                const int cl = col + 8 * q;
                if (Lc == C)
                    *reinterpret_cast<uint4 *>(sm + stage + (cl >> 6) * TILE + sw128_offset(r, cl & 63)) = w;
                else if (r < Lc && cl < d)
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + ((size_t)(cur.row0 + r) * p.H + cur.h) * d + cl) = w;
            }
        };
        wait(B_QK);
        tc_fence_after();
        if (ok && col < DKP) {
            result(T2, L::stQ, p.dq, p.dk);
            result(T3, L::stK, p.dk_, p.dk);
        }
        if (p.dg) {
            red[L::READS + grp * C + r] = reads;
            red[L::WRITES + grp * C + r] = writes;
#pragma unroll
            for (int off = 16; off; off >>= 1) thr += __shfl_xor_sync(0xffffffffu, thr, off);
            if (lane == 0) red[L::THR + warp] = thr;
        }
        fence_proxy_async_smem();
        bad = __syncthreads_or(!ok);
        if (bad) break;
        if (copier) {
            if (Lc == C) {
#pragma unroll
                for (int b = 0; b < DKP / 64; ++b) {
                    tma_store_3d(&tm_dq, sm + L::stQ + b * TILE, 64 * b, cur.h, (int)cur.row0);
                    tma_store_3d(&tm_dk, sm + L::stK + b * TILE, 64 * b, cur.h, (int)cur.row0);
                }
                bulk_commit();
            }
            if (more) load_qk(nxt, it + 1);
        }
        __syncwarp();
        if (tid == 64) s_tile[ph ^ 1] = settle(after);  // (read behind the tile's last barrier)
        // dg by one warp, four tokens a lane: from t on, the reads of S, and the pairs with the column blocks before t's;
        // the pairs across t in the diagonal block; before t, the writes that R sees, and the pairs of t's column block with
        // the row blocks behind; and e^{G_C} <S, R>. Exclusive sums are shifted, not subtracted.
        if (p.dg && warp == 2) {
            const int block = lane >> 3;
            const auto four = [&](int at, float (&x)[4]) {
                const float4 y = *reinterpret_cast<const float4 *>(red + at + 4 * lane);
                x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
            };
            float from[4][4] = {}, before[2][4] = {}, dg[4] = {};  // sums over the tokens from t on, and before t
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                four(L::READS + k * C, from[0]);
                four(L::WRITES + k * C, before[0]);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (block > k) four(L::ROWS + k * C, from[1 + k]);
                if (block <= k) four(L::COLS + k * C, before[1]);
            }
            four(L::DIAG, dg);
            float through = 0.f;
            for (int w = 0; w < 16; ++w) through += red[L::THR + w];
            through *= hla_decay(G[C - 1], g0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float *x = from[k];
                x[2] += x[3]; x[1] += x[2]; x[0] += x[1];
                float sum = x[0];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float y = __shfl_down_sync(0xffffffffu, sum, off);
                    if (lane + off < 32) sum += y;
                }
                sum = __shfl_down_sync(0xffffffffu, sum, 1);
                if (k == 0 || block >= k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dg[e] += lane < 31 ? x[e] + sum : x[e];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int first = k ? lane & 24 : 0;  // (columns: of this block)
                const float *x = before[k];
                const float x1 = x[0] + x[1], x2 = x1 + x[2];
                float sum = x2 + x[3];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, sum, off);
                    if (lane - off >= first) sum += y;
                }
                sum = __shfl_up_sync(0xffffffffu, sum, 1);
                if (lane == first) sum = 0.f;
                dg[0] += sum; dg[1] += sum + x[0]; dg[2] += sum + x1; dg[3] += sum + x2;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * lane + e;
                if (i < Lc) st_elem(static_cast<__nv_bfloat16 *>(p.dg), (size_t)(cur.row0 + i) * p.H + cur.h, dg[e] + through);
            }
        }
        wait(B_V);
        tc_fence_after();
        if (copier && ok && more) load_o(nxt);
        __syncwarp();
        if (ok && col < DVP) result(T1, L::stV, p.dv_, p.dv);
        fence_proxy_async_smem();
        tc_fence_before();
        bad = __syncthreads_or(!ok);
        if (bad) break;
        if (copier) {
            if (Lc == C) {
#pragma unroll
                for (int b = 0; b < DVP / 64; ++b) tma_store_3d(&tm_dv, sm + L::stV + b * TILE, 64 * b, cur.h, (int)cur.row0);
                bulk_commit();
            }
            bulk_wait_read_all();  // the staged results are read: their places may be loaded over
            if (more) load_vsr(nxt);
        }
        __syncwarp();
        cur = nxt;
    }
    grid_dependency_wait();  // whatever follows this launch follows the states' too
    if (bad) {  // leave nothing in flight behind: the copies, and whatever products were issued
        if (copier) {
            if (p.dev_status) atomicExch(p.dev_status, (int)KDA_ERR_TIMEOUT);
            bulk_wait_read_all();
            for (int b = 0; b < 3; ++b)
                if (loads[b] > 0) mbar_wait_bounded(bars + L_QK + b, (uint32_t)(loads[b] - 1) & 1u, kWaitCycles);
        }
        if (issuer) {
            mma_commit(bars + B_END);
            mbar_wait_bounded(bars + B_END, 0, kWaitCycles);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ================================================================== host
// 3-D map over a token-major [tokens, H, d] bf16 tensor; box of 64 channels (zeros past d) and 128 tokens.
// `rows` and `cols`: another box, of 32 rows and 32 channels in 64-byte swizzled rows (the outputs' staging).
bool make_tile_map(CUtensorMap *m, const void *base, size_t tokens, int H, int d, int cols = 64, int rows = C) {
    auto enc = tc::get_encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
    cuuint32_t box[3] = {(cuuint32_t)cols, 1, (cuuint32_t)rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
    int sc;
    bool order;
    long long slots, seg_slots;
    size_t order_at, next, gates, blob[2], seg[2], keep[2], bytes;
};
Layout layout(const HlaArgs &a, bool back) {
    Layout l{};
    const int dirs = back ? 2 : 1, dkp = padded(a.dk), dvp = padded(a.dv);
    const bool packed = a.cu_seqlens != nullptr;
    l.sc = hla_segment_chunks(a, C, (long long)a.N * a.H * dirs, device_sm_count());  // one chain's CTA per SM
    l.slots = hla_slots(packed, a.N, a.T, C);
    l.seg_slots = l.sc ? hla_slots(packed, a.N, a.T, l.sc * C) : 0;
    size_t at = 0;
    const auto take = [&](size_t bytes) { const size_t x = at; at += align256(bytes); return x; };
    // more chains than SMs, of different lengths: the longest first
    l.order = packed && !l.sc && seq_order_bytes(a.N) > 0 && (long long)a.N * a.H * dirs > device_sm_count();
    l.order_at = take(l.order ? seq_order_bytes(a.N) : 0);
    l.next = take(back ? sizeof(unsigned) : 0);
    l.gates = take((size_t)l.slots * a.H * GATE);
    for (int d = 0; d < dirs; ++d) {
        l.blob[d] = take(back ? (size_t)l.slots * a.H * blob_bytes(dkp, dvp) : 0);
        l.seg[d] = take((size_t)l.seg_slots * a.H * a.dk * a.dv * 4);
        l.keep[d] = take((size_t)l.seg_slots * a.H * 4);
    }
    l.bytes = at;
    return l;
}

struct Maps {
    CUtensorMap q, k, v, o, dq, dk, dv;
};

template <int DKP, int DVP, int kMode>
cudaError_t chain(const ChainArgs &s, const Maps &m, const Layout &l, int dirs) {
    const auto kern = hla_chain_tc_kernel<DKP, DVP, kMode>;
    constexpr size_t bytes = ChainSmem<DKP, DVP, kMode>::bytes;
    static HlaSmem smem;
    const cudaError_t e = smem.raise(kern, bytes);
    if (e != cudaSuccess) return e;
    kern<<<dim3((unsigned)((l.sc ? l.seg_slots : s.a.N) * s.hn), 1, dirs), kChainThreads, bytes, s.a.stream>>>(m.k, m.v, m.q, m.o, s);
    return cudaGetLastError();
}

template <int DKP, int DVP>
cudaError_t pass_t(const HlaArgs &a, bool back) {
    const size_t tokens = (size_t)a.B * a.T;
    Maps m;
    if (!make_tile_map(&m.q, a.q, tokens, a.H, a.dk) || !make_tile_map(&m.k, a.k, tokens, a.H, a.dk) ||
        !make_tile_map(&m.v, a.v, tokens, a.H, a.dv) ||
        !(back ? make_tile_map(&m.o, a.dO, tokens, a.H, a.dv) : make_tile_map(&m.o, a.o, tokens, a.H, a.dv, 32, 32)))
        return cudaErrorInvalidValue;
    if (back && (!make_tile_map(&m.dq, a.dq, tokens, a.H, a.dk) || !make_tile_map(&m.dk, a.dk_, tokens, a.H, a.dk) ||
                 !make_tile_map(&m.dv, a.dv_, tokens, a.H, a.dv)))
        return cudaErrorInvalidValue;
    const Layout l = layout(a, back);
    const int dirs = back ? 2 : 1;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    ChainArgs s{};
    s.a = a;
    if (back) s.a.ST = nullptr;
    s.seg.sc = l.sc;
    s.hn = a.H;
    s.gates = ws + l.gates;
    for (int d = 0; d < dirs; ++d) {
        s.blob[d] = ws + l.blob[d];
        s.seg.state[d] = reinterpret_cast<float *>(ws + l.seg[d]);
        s.seg.keep[d] = reinterpret_cast<float *>(ws + l.keep[d]);
    }
    cudaError_t e;
    if (l.order) {
        int32_t *order = reinterpret_cast<int32_t *>(ws + l.order_at);
        if ((e = launch_seq_order(a.cu_seqlens, a.N, order, a.stream)) != cudaSuccess) return e;
        s.order = order;
    }
    const unsigned units = (unsigned)(l.slots * a.H);
    if ((e = launch_hla_gates<__nv_bfloat16, C>(a, l.slots, ws + l.gates)) != cudaSuccess) return e;
    if (l.sc) {
        if ((e = chain<DKP, DVP, kEnds>(s, m, l, dirs)) != cudaSuccess) return e;
        if ((e = launch_hla_segment_scan(a, s.seg, l.sc * C, dirs)) != cudaSuccess) return e;
    }
    if (!back) return chain<DKP, DVP, kOut>(s, m, l, 1);
    const auto kern = hla_grad_tc_kernel<DKP, DVP>;
    constexpr size_t bytes = GradTile<DKP, DVP>::bytes;
    static HlaSmem smem;
    if ((e = smem.raise(kern, bytes)) != cudaSuccess) return e;
    // Chains that fill the SMs once or more and then some of them once again leave the others without work meanwhile. Of
    // a dense batch, whose chains are of one length, the heads of that last wave are a launch of their own, and the
    // gradients of the heads before run beside it, if those come to nearly whole waves (96 heads x 8192 tokens, 192 chains
    // on 148 SMs: 658 us against 711, and 650 since the chains are quicker).
    const unsigned sms = (unsigned)device_sm_count();
    const long long chains = (long long)a.N * a.H * dirs;
    int h1 = a.H;
    if (!a.cu_seqlens && !l.sc && chains > sms && chains % sms) {
        const long long per = (long long)a.N * dirs, first = chains / sms * sms / per * per;  // (whole heads)
        const auto idle = [&](long long n) { return (n + sms - 1) / sms * sms - n; };
        if (first > 0 && 2 * idle(first) < idle(chains)) h1 = (int)(first / per);
    }
    s.next = reinterpret_cast<unsigned *>(ws + l.next);
    s.first = units < sms ? units : sms;
    s.hn = h1;
    if ((e = chain<DKP, DVP, kStates>(s, m, l, dirs)) != cudaSuccess) return e;
    if (h1 < a.H) {
        s.next = nullptr;
        s.h0 = h1;
        s.hn = a.H - h1;
        if ((e = chain<DKP, DVP, kStates>(s, m, l, dirs)) != cudaSuccess) return e;
    }
    TileArgs t{};
    t.a = a;
    t.gates = s.gates;
    t.S = s.blob[0];
    t.R = s.blob[1];
    t.tiles = units;
    t.split = (unsigned)(l.slots * h1);
    t.h1 = h1;
    t.next = reinterpret_cast<unsigned *>(ws + l.next);
    // The attribute lets the launch begin once every CTA of the one before has: without a split that would be the launch
    // whose results are read, so there it is left out.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(s.first);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = a.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = h1 < a.H ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, m.q, m.k, m.v, m.o, m.dq, m.dk, m.dv, t);
}

cudaError_t pass(const HlaArgs &a, bool back) {
    const int k = padded(a.dk), v = padded(a.dv);
    if (k == 128) return v == 128 ? pass_t<128, 128>(a, back) : pass_t<128, 64>(a, back);
    return v == 128 ? pass_t<64, 128>(a, back) : pass_t<64, 64>(a, back);
}

}  // namespace

bool hla_tc_supported(const HlaArgs &a) {
    // one tile per (chunk slot, head), counted in 32 bits with what the CTAs take past the last one
    return a.dtype == KDA_DTYPE_BF16 && hla_slots(a.cu_seqlens != nullptr, a.N, a.T, C) <= 0x7fffffffLL / 2 / a.H;
}
size_t hla_tc_workspace(const HlaArgs &a, bool back) { return layout(a, back).bytes; }
cudaError_t launch_hla_forward_tc(const HlaArgs &a) { return pass(a, false); }
cudaError_t launch_hla_backward_tc(const HlaArgs &a) { return pass(a, true); }

}  // namespace kda
