"""Rotary positions against the rotation in fp64.

Tolerances per element, relative to its pair's length: fp32: the angle (2^-24 of a turn, reduced exactly), sine and cosine
(2^-22) and three roundings: 2^-20. bf16: that and half a step, 2^-8 of the element (2^-8 of its pair's length bounds it)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 2.0 ** -20, "bf16": 2.0 ** -8 + 2.0 ** -20}


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


def rope64(x, inv, pos, interleaved, inverse, mscale):
    rot = 2 * inv.numel()
    a = pos.double()[:, :, None, None] * inv.double()
    c, s = mscale * a.cos(), mscale * a.sin() * (-1 if inverse else 1)
    y = x.double().clone()
    ia, ib = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = p * c - q * s, q * c + p * s
    size = torch.ones_like(y)
    size[..., ia] = size[..., ib] = mscale * (p * p + q * q).sqrt()
    return y, size


def check(out, x, inv, pos, interleaved, inverse, mscale, dtype):
    y, size = rope64(x, inv, pos, interleaved, inverse, mscale)
    rot = 2 * inv.numel()
    assert ((out.double() - y).abs()[..., :rot] <= TOL[dtype] * size[..., :rot]).all()
    assert torch.equal(out[..., rot:], x[..., rot:])


CASES = [  # B, T, Hq, Hk, d, rot, dtype
    (1, 1, 1, 1, 2, 2, "f32"),
    (1, 1, 96, 96, 128, 128, "bf16"),
    (2, 33, 4, 2, 128, 128, "bf16"),
    (2, 33, 4, 2, 128, 64, "bf16"),
    (3, 17, 1, 5, 96, 44, "bf16"),
    (1, 70, 3, 1, 64, 14, "bf16"),
    (1, 70, 3, 1, 66, 66, "f32"),
    (2, 9, 2, 2, 256, 250, "f32"),
    (1, 1025, 8, 1, 64, 64, "f32"),
    (1, 5, 2, 2, 1024, 1024, "bf16"),
    (1, 3, 70, 70, 1024, 1022, "f32"),
    (1, 1, 300, 9, 4, 2, "bf16"),
    (5, 1, 33, 0, 128, 86, "bf16"),
    (1, 4097, 3, 3, 100, 98, "f32"),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot,dtype", CASES)
def test_rope(K, B, T, Hq, Hk, d, rot, dtype, interleaved):
    gen = torch.Generator(device="cuda").manual_seed(31 + T + rot)
    q = torch.randn(B, T, Hq, d, generator=gen, device="cuda").to(DT[dtype])
    k = torch.randn(B, T, Hk, d, generator=gen, device="cuda").to(DT[dtype]) if Hk else None
    inv, _ = K.kda_rope_inv_freq(rot, device="cuda")
    pos = torch.randint(0, 5000, (B, T), generator=gen, device="cuda")
    for inverse in (False, True):
        for p in (pos, pos.int(), None):
            qo, ko = K.kda_rope(q, k, inv, positions=p, interleaved=interleaved, mscale=1.3, inverse=inverse)
            at = torch.arange(T, device="cuda").expand(B, T) if p is None else pos
            check(qo, q, inv, at, interleaved, inverse, 1.3, dtype)
            if Hk:
                check(ko, k, inv, at, interleaved, inverse, 1.3, dtype)


@pytest.mark.parametrize("at", [0, 1 << 20, (1 << 31) - 5, -3, 1 << 40])
def test_far_positions(K, at):
    """The angle is reduced in fp64: 2^-53 of p * inv_freq / 2 pi turns, 1e-5 turns at 2^40 and nothing below 2^32."""
    q = torch.randn(1, 4, 2, 64, generator=torch.Generator(device="cuda").manual_seed(41), device="cuda")
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    pos = at + torch.arange(4, device="cuda").unsqueeze(0)
    out, none = K.kda_rope(q, None, inv, positions=pos)
    assert none is None
    y, size = rope64(q, inv, pos, False, False, 1.0)
    tol = 2.0 ** -20 + 2 * 3.2 * abs(at) * 2.0 ** -52  # both sides' angles, in radians
    assert ((out.double() - y).abs() <= tol * size).all()


@pytest.mark.parametrize("rot", [128, 96, 88, 86, 2])
def test_in_place_and_q_alone(K, rot):
    q = torch.randn(2, 40, 3, 128, generator=torch.Generator(device="cuda").manual_seed(42), device="cuda").bfloat16()
    k = torch.randn(2, 40, 1, 128, generator=torch.Generator(device="cuda").manual_seed(43), device="cuda").bfloat16()
    inv, _ = K.kda_rope_inv_freq(rot, device="cuda")
    for inter in (False, True):
        want = K.kda_rope(q, k, inv, interleaved=inter)
        alone, _ = K.kda_rope(q, None, inv, interleaved=inter)
        assert torch.equal(alone, want[0])
        q2, k2 = q.clone(), k.clone()
        K.kda_rope(q2, k2, inv, interleaved=inter, q_out=q2, k_out=k2)
        assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])


def test_inverse_is_the_gradient(K):
    gen = torch.Generator(device="cuda").manual_seed(44)
    q = torch.randn(1, 30, 2, 64, generator=gen, device="cuda")
    d = torch.randn(1, 30, 2, 64, generator=gen, device="cuda")
    inv, _ = K.kda_rope_inv_freq(48, device="cuda")
    x = q.double().requires_grad_()
    y = rope64(x, inv, torch.arange(30, device="cuda").unsqueeze(0), False, False, 0.8)[0]
    (want,) = torch.autograd.grad((y * d.double()).sum(), x)
    got, _ = K.kda_rope(d, None, inv, mscale=0.8, inverse=True)
    assert (got.double() - want).abs().max() < 2.0 ** -20 * float(d.abs().max()) * 2


def test_captured_and_replayed(K):
    q = torch.randn(1, 12, 2, 64, device="cuda")
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    pos = torch.arange(12, device="cuda", dtype=torch.int32).unsqueeze(0).contiguous()
    K.kda_rope(q, None, inv, positions=pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = K.kda_rope(q, None, inv, positions=pos)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, K.kda_rope(q, None, inv, positions=pos)[0])


def test_layer_with_rotated_keys(K):
    """The operators as a layer uses them: rotate, prefill, then rotate and decode one token at a time; and back. The
    rotation depends on q and k through their distance only, so a shift of all positions changes no output."""
    from hla_testutil import forward64, inputs, rel
    x = inputs(2, 150, 3, 128, 128, "bf16", seed=45)
    inv, m = K.kda_rope_inv_freq(64, device="cuda")
    outs = []
    for shift in (0, 100000):
        pos = (shift + torch.arange(150, device="cuda", dtype=torch.int32)).expand(2, 150).contiguous()
        q, k = K.kda_rope(x["q"], x["k"], inv, positions=pos, mscale=m)
        o, S = K.kda_hla_forward(*(y[:, :140].contiguous() for y in (q, k, x["v"], x["g"])), None, scale=0.1)
        parts = [o]
        for t in range(140, 150):
            qt, kt = K.kda_rope(x["q"][:, t:t + 1].contiguous(), x["k"][:, t:t + 1].contiguous(), inv, positions=pos[:, t:t + 1].contiguous(), mscale=m)
            parts.append(K.kda_hla_decode_step(qt[:, 0], kt[:, 0], x["v"][:, t].contiguous(), x["g"][:, t].contiguous(), S, scale=0.1).unsqueeze(1))
        outs.append(torch.cat(parts, 1))
        y = dict(x, q=q, k=k, S0=None)
        assert rel(outs[-1], forward64(y, 0.1)[0]) < 3 * 2.0 ** -8
        dq, dk, dv, dg, _ = K.kda_hla_backward(q, k, x["v"], x["g"], x["do"], scale=0.1)
        gq, gk = K.kda_rope(dq, dk, inv, positions=pos, mscale=m, inverse=True)
        assert torch.isfinite(gq).all() and torch.isfinite(gk).all()
    # each run's operands and outputs are rounded on their own: q, k, scores, states and outputs on both sides
    assert rel(outs[0], outs[1]) < 2 * 5 * 2.0 ** -8


def test_frequencies(K):
    base, m = K.kda_rope_inv_freq(64)
    assert m == 1.0 and base.dtype == torch.float32 and float(base[0]) == 1.0
    lin, _ = K.kda_rope_inv_freq(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin * 4, base, rtol=1e-6)
    ntk, _ = K.kda_rope_inv_freq(64, scaling="base", factor=4.0)
    assert float(ntk[0]) == 1.0 and abs(float(base[-1] / ntk[-1]) - 4.0) < 1e-5
    ramp, m = K.kda_rope_inv_freq(64, scaling="ramp", factor=8.0, original_length=4096)
    assert abs(m - 1.2079441541679836) < 1e-12
    assert torch.equal(ramp[:8], base[:8]) and torch.allclose(ramp[-4:] * 8, base[-4:], rtol=1e-6)
    assert ((ramp[1:] <= ramp[:-1])).all()
    short, _ = K.kda_rope_inv_freq(64, scaling="ramp", factor=8.0, original_length=6)  # no pair turns even once
    assert torch.allclose(short * 8, base, rtol=1e-6)
    for bad in (dict(rot_dim=7), dict(rot_dim=8, scaling="no"), dict(rot_dim=8, scaling="ramp", factor=2.0), dict(rot_dim=8, factor=0.5)):
        with pytest.raises(ValueError):
            K.kda_rope_inv_freq(**bad)


def test_refusals(K):
    q = torch.randn(1, 4, 2, 64, device="cuda")
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    with pytest.raises(ValueError):
        K.kda_rope(q, q.bfloat16(), inv)
    with pytest.raises(ValueError):
        K.kda_rope(q, q[:, :2].contiguous(), inv)
    with pytest.raises(ValueError):
        K.kda_rope(q, None, inv.double())
    with pytest.raises(ValueError):
        K.kda_rope(q, None, inv, positions=torch.zeros(1, 4, device="cuda"))
    with pytest.raises(ValueError):
        K.kda_rope(q, None, inv, positions=torch.zeros(1, 3, device="cuda", dtype=torch.int32))
    with pytest.raises(K.KdaError):  # more rotated channels than the head has
        K.kda_rope(q, None, torch.ones(33, device="cuda"))
