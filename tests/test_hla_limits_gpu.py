"""Linear attention with one decay per head where sizes and gates are at their limits. Tolerances as in test_hla_gpu.py: three
roundings of operands and result in bf16, sums and decays in fp32."""
import pytest
import torch

from hla_testutil import backward64, forward64, inputs, rel

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 3 * 2.0 ** -8}


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growth_within_a_few_tokens(K, dtype):
    """States that grow by 2^80 and shrink again by 2^128 within 29 tokens: each token's outputs and gradients."""
    x = inputs(1, 160, 2, 64, 64, dtype, seed=71, s0=False)
    for at in (0, 96):
        x["g"][:, at:at + 14], x["g"][:, at + 14:at + 29] = 4.0, -5.9375
    o, _ = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"])
    o64, _ = forward64(x)
    got, want = K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"]), backward64(x)
    for t in range(160):
        # a token's row of one head: sums of few terms, which may cancel to a quarter of their size
        for name, a, b in zip(("o", "dq", "dk", "dv"), (o, *got), (o64, *want)):
            assert rel(a[:, t], b[:, t]) < 4 * TOL[dtype], (name, t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_an_overflow(K, dtype):
    """A state that grows past fp32 at token 29 or so: the rows before it are right."""
    x = inputs(1, 40, 2, 64, 64, dtype, seed=72, s0=False)
    x["g"][:] = 3.0
    o, _ = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], scale=0.125)
    o64, _ = forward64(x, 0.125)
    for t in range(27):
        assert rel(o[:, t], o64[:, t]) < 4 * TOL[dtype], t
