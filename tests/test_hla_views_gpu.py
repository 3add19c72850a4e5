"""Views into longer tensors as arguments that are read by element: a token's gates, positions and frequencies from the middle
of an array, offsets of some of the sequences. Their addresses are those of an element, not of 16 bytes; the results are those
of a copy, to the bit."""
import pytest
import torch

from hla_testutil import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


def same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_a_single_requests_positions(K, dtype):
    q = torch.randn(1, 9, 3, 64, device="cuda").bfloat16()
    k = torch.randn(1, 9, 1, 64, device="cuda").bfloat16()
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    pos = torch.arange(1000, 1009, device="cuda", dtype=dtype).unsqueeze(0)
    want = K.kda_rope(q, k, inv, positions=pos)
    for t in range(9):
        view = pos[:, t:t + 1]
        assert view.is_contiguous()
        got = K.kda_rope(q[:, t:t + 1], k[:, t:t + 1], inv, positions=view)
        assert same(got, [x[:, t:t + 1] for x in want]), t


def test_frequencies_from_an_array_of_them(K):
    q = torch.randn(1, 5, 2, 32, device="cuda")
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    for a in (1, 2, 3, 5):
        assert same(K.kda_rope(q, None, inv[a:a + 16]), K.kda_rope(q, None, inv[a:a + 16].clone()))


@pytest.mark.parametrize("d,rot,dtype", [(100, 98, torch.bfloat16), (66, 44, torch.bfloat16), (66, 64, torch.float32), (6, 6, torch.float32)])
def test_a_single_token_of_odd_rows(K, d, rot, dtype):
    """Rows that are no multiple of 16 bytes: every token's begin where a row may."""
    q = torch.randn(1, 7, 1, d, device="cuda").to(dtype)
    inv, _ = K.kda_rope_inv_freq(rot, device="cuda")
    for inter in (False, True):
        want, _ = K.kda_rope(q, None, inv, interleaved=inter)
        for t in range(7):
            pos = torch.full((1, 1), t, device="cuda")
            x = q.clone()
            got, _ = K.kda_rope(x[:, t:t + 1], None, inv, positions=pos, interleaved=inter, q_out=x[:, t:t + 1])
            assert torch.equal(got, want[:, t:t + 1])
            assert torch.equal(x[:, :t], q[:, :t]) and torch.equal(x[:, t + 1:], q[:, t + 1:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_a_single_requests_gates(K, dtype, gate):
    """B = 1 and a number of heads whose gates do not fill 16 bytes: every token's step."""
    x = inputs(1, 9, 3, 64, 64, dtype, seed=61, gate=gate)
    S, S2 = x["S0"].clone(), x["S0"].clone()
    wide = torch.cat([x["g"], x["g"]]) if gate == "head" else None
    for t in range(9):
        tok = [x[n][:, t] for n in ("q", "k", "v")]
        g = wide[t % 3:t % 3 + 3] if gate == "head" else x["g"][:, t]
        assert g.is_contiguous()
        o = K.kda_hla_decode_step(*tok, g, S)
        o2 = K.kda_hla_decode_step(*tok, g.clone(), S2)
        assert torch.equal(o, o2) and torch.equal(S, S2), t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_rest_of_a_prompt(K, dtype):
    x = inputs(1, 150, 3, 64, 64, dtype, seed=62)
    side = torch.cuda.Stream()
    for cut in (1, 3, 8, 13):
        q, k, v, g, do = (x[n][:, cut:] for n in ("q", "k", "v", "g", "do"))
        assert g.is_contiguous()
        torch.cuda.synchronize()
        for s in (None, side):
            got = K.kda_hla_forward(q, k, v, g, x["S0"], stream=s) + K.kda_hla_backward(q, k, v, g, do, x["S0"], x["dS_T"], stream=s)
            torch.cuda.synchronize()
            g2 = g.clone()
            want = K.kda_hla_forward(q, k, v, g2, x["S0"]) + K.kda_hla_backward(q, k, v, g2, do, x["S0"], x["dS_T"])
            assert same(got, want), cut


def test_decays_per_head_from_an_array_of_them(K):
    x = inputs(1, 70, 3, 32, 32, "bf16", seed=63, gate="head")
    wide = torch.cat([x["g"], x["g"]])
    for a in (1, 2, 3):
        g = wide[a:a + 3]
        assert same(K.kda_hla_forward(x["q"], x["k"], x["v"], g), K.kda_hla_forward(x["q"], x["k"], x["v"], g.clone()))
        got, want = (K.kda_hla_backward(x["q"], x["k"], x["v"], y, x["do"]) for y in (g, g.clone()))
        assert same(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_offsets_of_some_sequences(K, dtype):
    x = inputs(1, 260, 2, 64, 64, dtype, seed=64, s0=False)
    cu = torch.tensor([0, 5, 70, 70, 201, 260], dtype=torch.int32, device="cuda")
    for a in (1, 2, 3):
        c = cu[a:a + 3]
        t0, t1 = int(c[0]), int(c[-1])
        o, S = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=c)
        o2, S2 = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=c.clone())
        assert torch.equal(o[:, t0:t1], o2[:, t0:t1]) and torch.equal(S, S2)
        got, want = (K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=y) for y in (c, c.clone()))
        assert same(got, want)


def test_a_step_on_views_captured(K):
    """The step of a single request with views of its gates and positions, in a graph."""
    x = inputs(1, 9, 3, 64, 64, "bf16", seed=65)
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    pos = torch.arange(9, device="cuda", dtype=torch.int32).unsqueeze(0)
    S, t = x["S0"].clone(), 5

    def step():
        q, k = K.kda_rope(x["q"][:, t:t + 1], x["k"][:, t:t + 1], inv, positions=pos[:, t:t + 1])
        return K.kda_hla_decode_step(q[:, 0], k[:, 0], x["v"][:, t], x["g"][:, t], S)

    want = step()
    S.copy_(x["S0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_what_is_still_refused(K):
    """Tensors that the kernels read 16 bytes at a time."""
    x = inputs(1, 4, 2, 32, 32, "f32", seed=66)
    odd = torch.empty(x["q"].numel() + 1, device="cuda")[1:].view(x["q"].shape)  # (4 bytes past a boundary)
    with pytest.raises(K.KdaError):
        K.kda_hla_forward(odd, x["k"], x["v"], x["g"])
    with pytest.raises(K.KdaError):
        K.kda_rope(odd, None, K.kda_rope_inv_freq(32, device="cuda")[0])
