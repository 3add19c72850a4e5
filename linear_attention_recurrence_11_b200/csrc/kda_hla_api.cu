// C ABI of linear attention with one decay per head and of rotary positions: argument validation and
// kernel dispatch (include/kda.h).
#include <stdint.h>

#include "kda_hla.cuh"

namespace {

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool aligned16(const void *p) { return aligned(p, 16); }
size_t dtype_bytes(int t) { return t == KDA_DTYPE_F32 ? 4 : 2; }
bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(int t) { return t == KDA_DTYPE_F32 || t == KDA_DTYPE_BF16; }
bool gate_ok(int g) { return g == KDA_HLA_GATE_TOKEN || g == KDA_HLA_GATE_HEAD; }

// Marks a packed batch in size queries (compared against null, never dereferenced).
const int32_t kPackedMarker = 0;

// Validates the shape arguments shared by the prefill and its backward pass; fills the sizes.
int check_sizes(int B, int T, int H, int dk, int dv, int dtype, bool packed, int num_seqs, int path, kda::HlaArgs *a) {
    if (B <= 0 || T < 0 || H <= 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (packed && (B != 1 || num_seqs <= 0)) return KDA_ERR_INVALID_ARG;
    if (path != KDA_PATH_AUTO && path != KDA_PATH_SIMT && path != KDA_PATH_TC) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    a->B = B; a->T = T; a->H = H; a->dk = dk; a->dv = dv; a->dtype = dtype;
    a->N = packed ? num_seqs : B;
    // one block per (sequence, head) and per (chunk slot, head), in 31-bit grids
    if ((long long)a->N * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if ((long long)B * T > 0x7fffffffLL - 256) return KDA_ERR_UNSUPPORTED;  // tokens are 32-bit coordinates of the copies
    if (kda::hla_slots(packed, a->N, T, 64) > 0x7fffffffLL / H) return KDA_ERR_UNSUPPORTED;
    a->cu_seqlens = packed ? &kPackedMarker : nullptr;
    if (path == KDA_PATH_TC && !kda::hla_tc_supported(*a)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// The tensor cores take every bf16 call that has tokens; a batch without any only hands its states on.
bool use_tc(const kda::HlaArgs &a, int path) { return path != KDA_PATH_SIMT && a.T > 0 && kda::hla_tc_supported(a); }

size_t workspace_of(const kda::HlaArgs &a, bool back, int path) {
    if (use_tc(a, path)) return kda::hla_tc_workspace(a, back);
    return kda::hla_simt_workspace(a, back);
}

}  // namespace

extern "C" {

size_t kda_hla_forward_workspace_size(int B, int T, int H, int dk, int dv, int num_seqs, int dtype, int path) {
    kda::HlaArgs a{};
    if (num_seqs < 0 || check_sizes(B, T, H, dk, dv, dtype, num_seqs > 0, num_seqs, path, &a)) return (size_t)-1;
    return workspace_of(a, false, path);
}

size_t kda_hla_backward_workspace_size(int B, int T, int H, int dk, int dv, int num_seqs, int dtype, int path) {
    kda::HlaArgs a{};
    if (num_seqs < 0 || check_sizes(B, T, H, dk, dv, dtype, num_seqs > 0, num_seqs, path, &a)) return (size_t)-1;
    return workspace_of(a, true, path);
}

int kda_hla_forward(const void *q, const void *k, const void *v, const void *g, const float *S0, void *o, float *S_T,
                    int B, int T, int H, int dk, int dv, float scale, int dtype, int gate, const int32_t *cu_seqlens,
                    int num_seqs, void *workspace, size_t workspace_bytes, int *dev_status, void *stream, int path) {
    kda::HlaArgs a{};
    const int st = check_sizes(B, T, H, dk, dv, dtype, cu_seqlens != nullptr, num_seqs, path, &a);
    if (st) return st;
    if (!gate_ok(gate)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !g || !o)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, g, (const void *)S0, (const void *)o, (const void *)S_T,
                          (const void *)workspace, (const void *)dev_status})
        if (!aligned16(p)) return KDA_ERR_ALIGNMENT;
    if (!aligned(cu_seqlens, sizeof(int32_t))) return KDA_ERR_ALIGNMENT;
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.o = o; a.ST = S_T;
    a.scale = scale; a.gate = gate; a.cu_seqlens = cu_seqlens;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes; a.dev_status = dev_status;
    a.stream = static_cast<cudaStream_t>(stream);
    const size_t need = workspace_of(a, false, path);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    return kda::cuda_status(use_tc(a, path) ? kda::launch_hla_forward_tc(a) : kda::launch_hla_forward_simt(a));
}

int kda_hla_backward(const void *q, const void *k, const void *v, const void *g, const float *S0, const void *dO,
                     const float *dS_T, void *dq, void *dk_out, void *dv_out, void *dg, float *dS0, int B, int T, int H,
                     int dk, int dv, float scale, int dtype, int gate, const int32_t *cu_seqlens, int num_seqs,
                     void *workspace, size_t workspace_bytes, int *dev_status, void *stream, int path) {
    kda::HlaArgs a{};
    const int st = check_sizes(B, T, H, dk, dv, dtype, cu_seqlens != nullptr, num_seqs, path, &a);
    if (st) return st;
    if (!gate_ok(gate)) return KDA_ERR_INVALID_ARG;
    if (gate == KDA_HLA_GATE_HEAD && dg) return KDA_ERR_INVALID_ARG;  // a head's fixed decay has no gradient
    if (T > 0 && (!q || !k || !v || !g || !dO || !dq || !dk_out || !dv_out)) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, g, (const void *)S0, dO, (const void *)dS_T, (const void *)dq, (const void *)dk_out,
                          (const void *)dv_out, (const void *)dg, (const void *)dS0,
                          (const void *)workspace, (const void *)dev_status})
        if (!aligned16(p)) return KDA_ERR_ALIGNMENT;
    if (!aligned(cu_seqlens, sizeof(int32_t))) return KDA_ERR_ALIGNMENT;
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.dO = dO; a.dST = dS_T;
    a.dq = dq; a.dk_ = dk_out; a.dv_ = dv_out; a.dg = dg; a.dS0 = dS0;
    a.scale = scale; a.gate = gate; a.cu_seqlens = cu_seqlens;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes; a.dev_status = dev_status;
    a.stream = static_cast<cudaStream_t>(stream);
    const size_t need = workspace_of(a, true, path);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (cu_seqlens && T > 0) {
        const cudaError_t e = kda::launch_hla_clear_outside(a);
        if (e != cudaSuccess) return kda::cuda_status(e);
    }
    return kda::cuda_status(use_tc(a, path) ? kda::launch_hla_backward_tc(a) : kda::launch_hla_backward_simt(a));
}

int kda_hla_decode_step(const void *q, const void *k, const void *v, const void *g, float *S, void *o, int N, int H,
                        int dk, int dv, float scale, int dtype, int gate, void *stream) {
    if (N <= 0 || H <= 0 || !dtype_ok(dtype) || !gate_ok(gate)) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if ((long long)N * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (!q || !k || !v || !g || !S || !o) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)S, (const void *)o})
        if (!aligned16(p)) return KDA_ERR_ALIGNMENT;
    if (!aligned(g, gate == KDA_HLA_GATE_HEAD ? sizeof(float) : dtype_bytes(dtype))) return KDA_ERR_ALIGNMENT;
    const kda::HlaDecodeArgs a{q, k, v, g, S, o, N, H, dk, dv, dtype, gate, scale, static_cast<cudaStream_t>(stream)};
    return kda::cuda_status(kda::launch_hla_decode(a));
}

int kda_rope(const void *q, const void *k, const void *positions, int positions_64bit, const float *inv_freq, void *q_out,
             void *k_out, int B, int T, int Hq, int Hk, int d, int rot_dim, int interleaved, int inverse, float mscale,
             int dtype, void *stream) {
    if (B <= 0 || T < 0 || Hq <= 0 || Hk < 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (d <= 0 || rot_dim <= 0 || rot_dim > d || (rot_dim & 1)) return KDA_ERR_INVALID_ARG;
    if (d > 1024 || (d & 1)) return KDA_ERR_UNSUPPORTED;
    if (Hq > 32768 || Hk > 32768 || (long long)B * T > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if ((k != nullptr) != (Hk > 0) || (k_out != nullptr) != (Hk > 0)) {
        if (T > 0 || Hk == 0) return KDA_ERR_INVALID_ARG;
    }
    if (T > 0 && (!q || !q_out || !inv_freq)) return KDA_ERR_INVALID_ARG;
    // rows of 16-byte pieces, or of the widest that a row divides into
    const size_t row = d * dtype_bytes(dtype), piece = row % 16 == 0 ? 16 : row % 8 == 0 ? 8 : 4;
    for (const void *p : {q, k, (const void *)q_out, (const void *)k_out})
        if (!aligned(p, piece)) return KDA_ERR_ALIGNMENT;
    if (!aligned(positions, positions_64bit ? sizeof(int64_t) : sizeof(int32_t)) || !aligned(inv_freq, sizeof(float))) return KDA_ERR_ALIGNMENT;
    kda::RopeArgs a{};
    a.q = q; a.k = k; a.positions = positions; a.inv_freq = inv_freq; a.q_out = q_out; a.k_out = k_out;
    a.tokens = (long long)B * T; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot_dim = rot_dim;
    a.pos64 = positions_64bit != 0; a.interleaved = interleaved != 0; a.inverse = inverse != 0;
    a.mscale = mscale; a.dtype = dtype; a.stream = static_cast<cudaStream_t>(stream);
    return kda::cuda_status(kda::launch_rope(a));
}

}  // extern "C"
