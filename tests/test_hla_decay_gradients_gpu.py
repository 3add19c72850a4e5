"""The gradient of the log-decays, one head at a time and 32 tokens at a time, so that a head that forgets fast does not
hide behind one that does not.

Tolerances, on the 2-norm of the difference over that of the part compared. Every term is a pair of a write before the token
and a read from it on. bf16: half a step, 2^-8, of the result's own rounding, as much for each of the two states that a
term across chunks is taken with (rounded operands), and as much again for what the sums do to these: 4 x 2^-8. fp32: a term
is good to 2^-20 (the decay's power, 2^-22, and the rounding of the products), and a norm may be a fifth of its terms': 1e-5.
A token with no write before it, and one whose decay is zero in fp32, has a gradient of exactly zero."""
import pytest
import torch

from hla_testutil import backward64, inputs, rel

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 4 * 2.0 ** -8}
RATES = [1.0, 5.0, 10.0, 15.0, 20.0, 60.0]  # (exact in bf16)


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


def gradients(K, x, cu=None, **kw):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], cu_seqlens=c, **kw)


def check_parts(got, want, t0, t1, tol):
    for h in range(got.shape[2]):
        for t in range(t0, t1, 32):
            a, b = got[:, t:min(t + 32, t1), h], want[:, t:min(t + 32, t1), h]
            assert rel(a, b) < tol, (h, t, rel(a, b))


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("bf16", 64, 128), ("bf16", 128, 32), ("f32", 128, 64), ("f32", 32, 32)])
@pytest.mark.parametrize("s0", [False, True])
def test_uniform_decays(K, dtype, dk, dv, s0):
    x = inputs(2, 300, len(RATES), dk, dv, dtype, seed=51, s0=s0)
    x["g"][:] = -torch.tensor(RATES, device="cuda").to(x["g"].dtype)
    got, want = gradients(K, x, scale=0.3)[3], backward64(x, 0.3)[3]
    if not s0:
        assert (got[:, 0] == 0).all()
    check_parts(got, want, 0 if s0 else 1, 300, TOL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_uniform_decays_of_packed_sequences(K, dtype):
    lens = [3, 130, 0, 1, 257, 40]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    x = inputs(1, cu[-1], len(RATES), 64, 64, dtype, seed=52, s0=False)
    x["g"][:] = -torch.tensor(RATES, device="cuda").to(x["g"].dtype)
    got, want = gradients(K, x, cu)[3], backward64(x, 1.0, cu)[3]
    for a, b in zip(cu, cu[1:]):
        assert (got[:, a:a + 1][:, :b - a] == 0).all()
        check_parts(got, want, a + 1, b, TOL[dtype])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_strong_decays_then_weak_ones(K, dtype, d):
    """Head 0: 150 tokens of e^-60, then hardly any decay; head 1 the other way round; head 2: nothing survives a token."""
    x = inputs(1, 300, 3, d, d, dtype, seed=53)
    g = x["g"]
    g[:, :150, 0], g[:, 150:, 0] = -60.0, -0.001
    g[:, :150, 1], g[:, 150:, 1] = -0.001, -60.0
    g[:, :, 2] = -300.0
    got, want = gradients(K, x)[3], backward64(x, 1.0)[3]
    for h in (0, 1):
        for a, b in ((0, 150), (150, 300)):
            assert rel(got[:, a:b, h], want[:, a:b, h]) < TOL[dtype], (h, a)
    assert (got[:, :, 2] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_write_and_one_read(K, dtype):
    """One key that is not zero, at s, and one query, at r: dg is the same number at s + 1 .. r and zero elsewhere,
    whichever blocks of the chunk the two are in."""
    for s, r in ((0, 1), (0, 127), (5, 31), (31, 32), (3, 70), (40, 63), (33, 100), (64, 127), (95, 96), (100, 110), (10, 300), (200, 400)):
        x = inputs(1, 401, 1, 64, 64, dtype, seed=54, s0=False)
        only = torch.zeros(1, 401, 1, 1, device="cuda", dtype=x["q"].dtype)
        only[:, s] = 1
        x["k"] *= only
        x["q"] *= only.roll(r - s, 1)
        x["q"][:, r], x["do"][:, r] = x["k"][:, s], x["v"][:, s]  # (so that nothing within the one term cancels)
        x["g"][:] = -0.015625
        got, want = gradients(K, x)[3][0, :, 0], backward64(x, 1.0)[3][0, :, 0]
        assert (got[:s + 1] == 0).all() and (got[r + 1:] == 0).all(), (s, r)
        assert ((got.double() - want).abs() <= TOL[dtype] * want.abs()).all(), (s, r)
