"""Linear attention with one decay per head in every form: bf16 storage with fp32 accuracy (path "simt"), and all pairs of
head sizes in both types.

Tolerances, on the 2-norm of the difference over that of the result. fp32 accuracy: 1e-5 as in test_hla_gpu.py; with bf16
storage the results of the activations' type are rounded once more, 2^-8, and the states are not. Tensor cores: as in
test_hla_gpu.py."""
import pytest
import torch

from hla_testutil import backward64, forward64, inputs, rel

pytestmark = pytest.mark.gpu

ROUNDED = 2.0 ** -8 + 1e-5
NAMES = ("o", "S_T", "dq", "dk", "dv", "dg", "dS0")


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


def run(K, x, scale, cu, path):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    B, T, H, dk = x["q"].shape
    N, dv = (0 if cu is None else len(cu) - 1), x["v"].shape[-1]
    ws = [torch.empty(f(B, T, H, dk, dv, N, x["q"].dtype, path), dtype=torch.uint8, device="cuda")
          for f in (K.kda_hla_forward_workspace_size, K.kda_hla_backward_workspace_size)]
    args = [x[n] for n in ("q", "k", "v", "g")]
    out = K.kda_hla_forward(*args, x["S0"], scale=scale, cu_seqlens=c, path=path, workspace=ws[0])
    return out + K.kda_hla_backward(*args, x["do"], x["S0"], x["dS_T"], scale=scale, cu_seqlens=c, path=path, workspace=ws[1])


def check(K, x, scale, path, tol, tol_state, cu=None):
    got = run(K, x, scale, cu, path)
    want = forward64(x, scale, cu) + backward64(x, scale, cu)
    for name, a, b in zip(NAMES, got, want):
        if a is None:
            assert name == "dg" and x["g"].dim() == 1
            continue
        if name == "o" and cu is not None:
            a, b = a[:, cu[0]:cu[-1]], b[:, cu[0]:cu[-1]]
        assert rel(a, b) < (tol_state if name in ("S_T", "dS0") else tol * (4 / 3 if name == "dg" else 1)), (name, rel(a, b))


@pytest.mark.parametrize("B,T,H,dk,dv,gate,s0", [
    (1, 1, 2, 128, 128, "token", True),
    (2, 64, 3, 64, 64, "head", False),
    (1, 65, 2, 128, 64, "token", False),
    (2, 200, 5, 128, 128, "token", True),
    (1, 1500, 2, 128, 128, "token", True),   # few heads: segments
    (1, 1300, 1, 32, 128, "token", False),
])
def test_bf16_in_fp32_accuracy(K, B, T, H, dk, dv, gate, s0):
    check(K, inputs(B, T, H, dk, dv, "bf16", seed=81 + T, gate=gate, s0=s0), dk ** -0.5, "simt", ROUNDED, 1e-5)


@pytest.mark.parametrize("lead,tail", [(0, 0), (5, 70)])
def test_packed_bf16_in_fp32_accuracy(K, lead, tail):
    lens = [1, 130, 0, 64, 200, 1, 900, 63]
    cu = [lead + sum(lens[:i]) for i in range(len(lens) + 1)]
    check(K, inputs(1, cu[-1] + tail, 3, 64, 128, "bf16", seed=82, N=len(lens)), 0.2, "simt", ROUNDED, 1e-5, cu)


@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_pair_of_head_sizes(K, dtype, dk, dv):
    tol, tol_state = (1e-5, 1e-5) if dtype == "f32" else (3 * 2.0 ** -8, 2.0 ** -16 + 1e-5)
    check(K, inputs(2, 333, 3, dk, dv, dtype, seed=83), dk ** -0.5, "auto", tol, tol_state)


@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_pair_of_head_sizes_in_segments(K, dtype, dk, dv):
    """One head and enough tokens that the sequence is cut."""
    tol, tol_state = (1e-5, 1e-5) if dtype == "f32" else (3 * 2.0 ** -8, 2.0 ** -16 + 1e-5)
    check(K, inputs(1, 2100, 1, dk, dv, dtype, seed=84), dk ** -0.5, "auto", tol, tol_state)


def test_decode_follows_both_forms(K):
    """Two prompts' states, from either form, and ten tokens more: the recurrence."""
    x = inputs(2, 110, 3, 128, 64, "bf16", seed=85)
    o64, S64 = forward64(x)
    for path, tol in (("simt", 1e-5), ("tc", 2.0 ** -16 + 1e-5)):
        _, S = K.kda_hla_forward(*(x[n][:, :100].contiguous() for n in ("q", "k", "v", "g")), x["S0"], path=path)
        for t in range(100, 110):
            o = K.kda_hla_decode_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v", "g")), S)
            assert rel(o, o64[:, t]) < 2.0 ** -8 + tol
        assert rel(S, S64) < tol + 1e-6
