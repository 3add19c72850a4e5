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


def test_more_heads_than_a_grids_second_axis(K):
    """More than 65535 x 32 heads: prefill in bf16, backward pass in fp32."""
    H, d = 65535 * 32 + 33, 32
    gen = torch.Generator(device="cuda").manual_seed(73)
    q, k, v, do = (torch.randn(1, 1, H, d, generator=gen, device="cuda") for _ in range(4))
    g = -torch.rand(1, 1, H, generator=gen, device="cuda")
    low = [y.bfloat16() for y in (q, k, v, g)]
    o, _ = K.kda_hla_forward(*low, return_state=False)
    a, b, c = (y.double() for y in low[:3])
    # the score, q k^T, is rounded to bf16 and so is the result
    assert rel(o, (a * b).sum(-1, keepdim=True) * c) < 2 * 2.0 ** -8
    dq, dk, dv, dg, _ = K.kda_hla_backward(q, k, v, g, do, return_dS0=False)
    s, w = (do.double() * v.double()).sum(-1, keepdim=True), (q.double() * k.double()).sum(-1, keepdim=True)
    assert rel(dq, s * k.double()) < 1e-5 and rel(dk, s * q.double()) < 1e-5 and rel(dv, w * do.double()) < 1e-5
    assert (dg == 0).all()


def test_codes_of_refusals(K):
    x = inputs(1, 8, 2, 32, 32, "f32", seed=74)
    args = [x[n] for n in ("q", "k", "v", "g")]

    def code(f, *a, **kw):
        with pytest.raises(K.KdaError) as e:
            f(*a, **kw)
        return e.value.code

    empty = [y[:0] for y in args]
    for path, want in (("tc_single", K.KDA_ERR_INVALID_ARG), ("tc", K.KDA_ERR_UNSUPPORTED)):
        assert code(K.kda_hla_forward, *args, path=path) == want
        assert code(K.kda_hla_backward, *args, x["do"], path=path) == want
    assert code(K.kda_hla_forward, *empty) == K.KDA_ERR_INVALID_ARG
    assert code(K.kda_hla_backward, *empty, x["do"][:0]) == K.KDA_ERR_INVALID_ARG


GUARD = 4096


def guarded(shape, dtype):
    """A tensor between two runs of bytes of 0x5a."""
    n = torch.empty(0, dtype=dtype).element_size()
    for s in shape:
        n *= s
    whole = torch.full((n + 2 * GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
    return whole, whole[GUARD:GUARD + n].view(dtype).view(shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu,clamped", [([0, 50, 1000, 2000], [0, 50, 300, 300]), ([-7, 3, 3, 300], [0, 3, 3, 300]), ([-9, -5, 120, 1 << 30], [0, 0, 120, 300])])
def test_offsets_past_the_tensors(K, dtype, cu, clamped):
    """Offsets below zero or past the tokens count as zero and as the number of tokens, and nothing outside the outputs and
    the workspace is written."""
    x = inputs(1, 300, 2, 64, 64, dtype, seed=75, N=3)
    dt = x["v"].dtype
    c, c2 = (torch.tensor(y, dtype=torch.int32, device="cuda") for y in (cu, clamped))
    keep_o, o = guarded((1, 300, 2, 64), dt)
    keep_s, S = guarded((3, 2, 64, 64), torch.float32)
    keep_w, ws = guarded((K.kda_hla_forward_workspace_size(1, 300, 2, 64, 64, 3, dt),), torch.uint8)
    K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=c, o=o, S_T=S, workspace=ws)
    keep_b, wb = guarded((K.kda_hla_backward_workspace_size(1, 300, 2, 64, 64, 3, dt),), torch.uint8)
    got = K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], cu_seqlens=c, workspace=wb)
    torch.cuda.synchronize()
    for whole in (keep_o, keep_s, keep_w, keep_b):
        assert (whole[:GUARD] == 0x5a).all() and (whole[-GUARD:] == 0x5a).all()
    o2, S2 = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=c2)
    want = K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], cu_seqlens=c2)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
