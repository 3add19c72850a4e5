"""How accurate linear attention with one decay per head is over many elements, where roundings average: bounds on the 2-norm of
the difference over that of the result that a loss of a bit or two does not pass.

bf16 on the tensor cores. A rounding to bf16 is off by at most 2^-8 of a value, evenly spread, so by at most 2^-8 / sqrt(3) on the
norm. Outputs and gradients take three of them independently (an operand, a state, the result): 2^-8 in all. dg takes four
(both states, their product <S, R> as much again, the result): 2^-8 * 2 / sqrt(3). What is added to a state is the sum of two
bf16 numbers: the second's rounding of the first's remainder, 2^-16 / 3, and the sums in fp32, 2^-20.

fp32. An operand of two TF32 numbers is off by 2^-22 at most (what the second one's cut drops), decays by 2^-22; a result is a
chain of two products, so of four operands and two decays, and sums over 64 tokens and chunks: below 8 x 2^-22 = 2e-6. bf16
storage in fp32 accuracy: 2^-8 / sqrt(3) for the result's rounding and those 2e-6."""
import math

import pytest
import torch

from hla_testutil import backward64, forward64, inputs, rel

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -8
F32 = 8 * 2.0 ** -22
NAMES = ("o", "S_T", "dq", "dk", "dv", "dg", "dS0")


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


def bound(name, dtype, path):
    if dtype == "f32":
        return F32
    if name in ("S_T", "dS0"):
        return F32 if path == "simt" else 2.0 ** -16 / 3 + 2.0 ** -20
    if path == "simt":
        return STEP / math.sqrt(3) + F32
    return STEP * (2 / math.sqrt(3) if name == "dg" else 1)


@pytest.mark.parametrize("dtype,path", [("bf16", "tc"), ("bf16", "simt"), ("f32", "simt")])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32), (32, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_norms(K, dtype, path, dk, dv, packed):
    lens = [700, 1, 900, 65, 334] if packed else None
    cu = [sum(lens[:i]) for i in range(6)] if packed else None
    x = inputs(1 if packed else 2, 2000 if packed else 1000, 6, dk, dv, dtype, seed=91, N=5 if packed else None)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    args, scale = [x[n] for n in ("q", "k", "v", "g")], dk ** -0.5
    got = K.kda_hla_forward(*args, x["S0"], scale=scale, cu_seqlens=c, path=path)
    got += K.kda_hla_backward(*args, x["do"], x["S0"], x["dS_T"], scale=scale, cu_seqlens=c, path=path)
    want = forward64(x, scale, cu) + backward64(x, scale, cu)
    off = {n: rel(a, b) / bound(n, dtype, path) for n, a, b in zip(NAMES, got, want)}
    assert all(y < 1 for y in off.values()), off
