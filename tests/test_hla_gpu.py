"""Linear attention with one decay per head against the recurrence in fp64, token by token (its gradients by
automatic differentiation of that).

Tolerances, on the 2-norm of the difference over that of the result. fp32: sums of at most a few hundred terms, each
rounded to 2^-24 of the running sum, and decays good to 2^-22: below 32 x 2^-24 = 2e-6 x a factor 5 for norms reduced by
cancellation. bf16 outputs: half a step, 2^-8, of the result's own rounding, and as much for each of the two operands that
the tensor cores take rounded (scores and states): 3 x 2^-8. States and their gradients stay fp32 outputs with bf16 inputs:
a scaled operand is the sum of two bf16 numbers, off by at most 2^-16, and the sums as in fp32: 2^-16 + 1e-5."""
import pytest
import torch

from hla_testutil import backward64, forward64, inputs, rel

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 3 * 2.0 ** -8}
TOL_STATE = {"f32": 1e-5, "bf16": 2.0 ** -16 + 1e-5}


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


def cu_of(lens, lead=0):
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def run_forward(K, x, cu=None, **kw):
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, S = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=c, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    return o, S


def run_backward(K, x, cu=None, **kw):
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], cu_seqlens=c, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    return out


def check_forward(K, x, dtype, scale, cu=None, **kw):
    o, S = run_forward(K, x, cu, scale=scale, **kw)
    o64, S64 = forward64(x, scale, cu)
    t0, t1 = (0, o.shape[1]) if cu is None else (cu[0], cu[-1])
    assert rel(o[:, t0:t1], o64[:, t0:t1]) < TOL[dtype]
    assert rel(S, S64) < TOL_STATE[dtype]
    return o, S


def check_backward(K, x, dtype, scale, cu=None, **kw):
    got = run_backward(K, x, cu, scale=scale, **kw)
    want = backward64(x, scale, cu)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        if name == "dg" and x["g"].dim() == 1:
            assert a is None
            continue
        # four roundings for the gradients: the outputs', scores' and states', and dg's two operands
        tol = TOL_STATE[dtype] if name == "dS0" else TOL[dtype] * (4 / 3 if name == "dg" else 1)
        assert rel(a, b) < tol, (name, rel(a, b))
    return got


SHAPES = [  # B, T, H, dk, dv, dtype, gate, S0
    (1, 1, 1, 128, 128, "bf16", "token", False),
    (2, 1, 3, 128, 128, "bf16", "token", True),
    (1, 63, 2, 128, 128, "bf16", "token", True),
    (1, 64, 2, 128, 128, "bf16", "head", False),
    (1, 65, 1, 128, 128, "bf16", "token", True),
    (2, 127, 2, 128, 128, "bf16", "token", True),
    (1, 128, 2, 128, 128, "bf16", "token", True),
    (1, 129, 2, 128, 128, "bf16", "head", True),
    (3, 300, 5, 128, 128, "bf16", "token", False),
    (1, 513, 3, 128, 128, "bf16", "token", True),
    (2, 1290, 9, 128, 128, "bf16", "token", True),   # more chunks than SMs, partial ones among them
    (3, 1030, 7, 64, 128, "bf16", "token", False),
    (1, 2700, 9, 128, 64, "bf16", "head", True),
    (1, 1, 2, 32, 64, "f32", "token", True),
    (2, 97, 3, 64, 32, "f32", "head", True),
    (1, 200, 2, 128, 128, "f32", "token", False),
    (1, 130, 2, 128, 64, "f32", "token", True),
    (1, 161, 3, 64, 128, "bf16", "token", True),
    (2, 70, 2, 64, 64, "bf16", "token", True),
    (1, 90, 2, 32, 32, "bf16", "token", True),
    (1, 150, 80, 64, 64, "bf16", "token", True),     # more chains in the backward pass than SMs, and not twice as many
    (2, 129, 43, 128, 64, "bf16", "token", False),
    (80, 5, 2, 32, 32, "bf16", "token", True),       # (whole heads of which do not come to whole waves)
]


@pytest.mark.parametrize("B,T,H,dk,dv,dtype,gate,s0", SHAPES)
def test_forward(K, B, T, H, dk, dv, dtype, gate, s0):
    x = inputs(B, T, H, dk, dv, dtype, seed=100 + T, gate=gate, s0=s0)
    check_forward(K, x, dtype, dk ** -0.5)


@pytest.mark.parametrize("B,T,H,dk,dv,dtype,gate,s0", SHAPES)
def test_backward(K, B, T, H, dk, dv, dtype, gate, s0):
    x = inputs(B, T, H, dk, dv, dtype, seed=200 + T, gate=gate, s0=s0)
    check_backward(K, x, dtype, dk ** -0.5)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 64)])
@pytest.mark.parametrize("lead,tail", [(0, 0), (5, 70)])
def test_packed(K, dtype, d, lead, tail):
    """Empty and one-token sequences, cuts inside tiles, rows of no sequence in front and behind: those rows' outputs
    stay as they were, and their gradients are zero; whatever stands there reaches nothing."""
    lens = [1, 130, 0, 64, 200, 1, 1, 63, 129]
    cu = cu_of(lens, lead)
    T = cu[-1] + tail
    x = inputs(1, T, 3, d, d, dtype, seed=7, N=len(lens))
    for n in ("q", "k", "v", "do"):
        x[n][:, :lead] = float("nan")
        x[n][:, cu[-1]:] = float("nan")
    o = torch.full((1, T, 3, d), 7.0, dtype=x["v"].dtype, device="cuda")
    o, S = check_forward(K, x, dtype, 0.2, cu, o=o)
    assert (o[:, :lead] == 7).all() and (o[:, cu[-1]:] == 7).all()
    assert torch.equal(S[2], x["S0"][2])  # the empty sequence's state passes through
    clean = {n: (y if y is None or n not in ("q", "k", "v", "do") else torch.nan_to_num(y)) for n, y in x.items()}
    got = run_backward(K, x, cu, scale=0.2)
    want = backward64(clean, 0.2, cu)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        tol = TOL_STATE[dtype] if name == "dS0" else TOL[dtype] * (4 / 3 if name == "dg" else 1)
        assert rel(a, b) < tol, (name, rel(a, b))
        if name != "dS0":
            assert (a[:, :lead] == 0).all() and (a[:, cu[-1]:] == 0).all()
    assert torch.equal(got[4][2], x["dS_T"][2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_of_nans_stays_alone(K, dtype):
    """Sequences that share a tile with one that holds NaN and infinities keep their results, to the bit."""
    lens = [70, 200, 1, 59]
    cu = cu_of(lens)
    x = inputs(1, cu[-1], 2, 64, 64, dtype, seed=27, N=len(lens))
    want = run_forward(K, x, cu) + run_backward(K, x, cu)
    for i, n in enumerate(("q", "k", "v", "do", "g")):
        x[n][:, cu[1] + 20 * i:cu[2] - 3] = float("nan") if i % 2 else float("inf") if n != "g" else float("nan")
    got = run_forward(K, x, cu) + run_backward(K, x, cu)
    for a, b in zip(want, got):
        for n in (0, 2, 3):
            part = (lambda y: y[n]) if a.dtype == torch.float32 and a.shape[0] == len(lens) else (lambda y: y[:, cu[n]:cu[n + 1]])
            assert torch.equal(part(a), part(b))


@pytest.mark.parametrize("dtype,T", [("bf16", 300), ("f32", 300), ("bf16", 5000)])
def test_states_updated_in_place(K, dtype, T):
    """S_T may be S0 itself."""
    x = inputs(1, T, 2, 64, 64, dtype, seed=28)
    o, S = run_forward(K, x)
    o2, S2 = run_forward(K, x, S_T=x["S0"])
    assert S2 is x["S0"] and torch.equal(S2, S) and torch.equal(o2, o)


def test_packed_more_chains_than_sms(K):
    """Many short and a few long sequences: chains in order of length, chunks of all of them in one grid."""
    lens = [5, 1, 0, 260, 128, 3, 7, 129, 0, 1, 64, 2, 90, 700, 1, 33, 256, 1, 1, 11]
    x = inputs(1, sum(lens), 9, 128, 128, "bf16", seed=8, N=len(lens))
    check_forward(K, x, "bf16", 0.5, cu_of(lens))
    check_backward(K, x, "bf16", 0.5, cu_of(lens))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_decays_at_their_limits(K, dtype, d):
    """No decay at all, a reset (-infinity), decays that underflow fp32, and weak ones after strong ones in one chunk."""
    x = inputs(1, 300, 4, d, d, dtype, seed=9)
    g = x["g"]
    g[:, :, 0] = 0.0
    g[:, 40::70, 1] = float("-inf")
    g[:, :, 2] = -300.0
    g[:, :150, 3] = -60.0
    g[:, 150:, 3] = -0.001
    o, S = check_forward(K, x, dtype, 1.0)
    for h in range(4):  # per head, so that none hides behind another
        o64, S64 = forward64({n: (y if y is None else y[:, h:h + 1] if n in ("S0", "dS_T") else y[:, :, h:h + 1]) for n, y in x.items()}, 1.0)
        assert rel(o[:, :, h:h + 1], o64) < TOL[dtype]
        assert rel(S[:, h:h + 1], S64) < TOL_STATE[dtype]
    got = run_backward(K, x, scale=1.0)
    want = backward64(x, 1.0)
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        for h in range(4):
            assert rel(a[:, :, h], b[:, :, h]) < TOL[dtype], (name, h)
    for h in (0, 1):  # (heads 2 and 3 scale nothing that fp32 could hold)
        assert rel(got[3][:, :, h], want[3][:, :, h]) < TOL[dtype] * 4 / 3, h
    assert torch.isfinite(got[3]).all()
    for h in range(4):  # head 2's, e^-300 times something, is zero in fp32
        assert rel(got[4][:, h], want[4][:, h].float()) < TOL_STATE[dtype], h


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_long_without_decay(K, dtype, d):
    """A long sequence that forgets nothing: the state's sums run over every token."""
    x = inputs(1, 4100, 1, d, d, dtype, seed=10, rate=0.0)
    check_forward(K, x, dtype, 1.0)
    check_backward(K, x, dtype, 1.0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_prompt_in_two_parts_then_tokens(K, dtype, d):
    """A prompt split at an odd place through its state, then decode steps: the whole sequence's outputs."""
    T, cut, steps, scale = 230, 101, 6, 0.3
    x = inputs(2, T + steps, 3, d, d, dtype, seed=11)
    o64, S64 = forward64(x, scale)
    part = lambda a, b: [x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")]  # noqa: E731
    o1, S = K.kda_hla_forward(*part(0, cut), x["S0"], scale=scale)
    o2, S = K.kda_hla_forward(*part(cut, T), S, scale=scale)
    outs = [o1, o2]
    for t in range(T, T + steps):
        q, k, v, g = (y[:, 0].contiguous() for y in part(t, t + 1))
        outs.append(K.kda_hla_decode_step(q, k, v, g, S, scale=scale).unsqueeze(1))
    assert rel(torch.cat(outs, 1), o64) < TOL[dtype]
    assert rel(S, S64) < TOL_STATE[dtype] * 2  # through two prefills


@pytest.mark.parametrize("N,H,dk,dv,dtype,gate", [(1, 1, 128, 128, "bf16", "token"), (1, 32, 128, 128, "bf16", "head"),
                                                  (7, 3, 32, 64, "f32", "token"), (5, 2, 64, 32, "bf16", "token"),
                                                  (300, 9, 128, 128, "bf16", "token"), (2, 2, 128, 32, "f32", "head")])
def test_decode(K, N, H, dk, dv, dtype, gate):
    x = inputs(N, 1, H, dk, dv, dtype, seed=12, gate=gate)
    o64, S64 = forward64(x, 0.25)
    S = x["S0"].clone()
    g = x["g"] if gate == "head" else x["g"][:, 0].contiguous()
    o = K.kda_hla_decode_step(*(x[n][:, 0].contiguous() for n in ("q", "k", "v")), g, S, scale=0.25)
    # one product sum in fp32, rounded once
    assert rel(o, o64[:, 0]) < (1e-6 if dtype == "f32" else 2.0 ** -8)
    assert rel(S, S64) < 1e-6


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_gradients_by_differences(K, dtype, d):
    """The gradients along random directions against central differences of the definition in fp64."""
    x = inputs(1, 140, 2, d, d, dtype, seed=13)
    got = run_backward(K, x, scale=0.5)

    def loss(y):
        o, S = forward64(y, 0.5)
        return float((o * x["do"].double()).sum() + (S * x["dS_T"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(14)
    for name, grad in zip(("q", "k", "v", "g", "S0"), got):
        u = torch.randn(x[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        base = {n: (None if y is None else y.double()) for n, y in x.items()}
        up, down = dict(base), dict(base)
        up[name], down[name] = base[name] + h * u, base[name] - h * u
        diff = (loss(up) - loss(down)) / (2 * h)
        dot = float((grad.double() * u).sum())
        # a sum over independent directions: the gradient's normwise error times its norm, at four standard deviations
        assert abs(dot - diff) < 4 * TOL[dtype] * 4 / 3 * float(torch.linalg.vector_norm(grad.double())), name


def test_two_calls_give_the_same_bits(K):
    x = inputs(2, 400, 4, 128, 128, "bf16", seed=15)
    a, b = run_forward(K, x), run_forward(K, x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = run_backward(K, x), run_backward(K, x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_same_bits_over_long_chains_with_partial_ends(K):
    """Hundreds of chunks per chain, whose last one ends inside its tile: nothing may depend on when a copy arrives."""
    x = inputs(1, 20024, 96, 128, 128, "bf16", seed=26)
    first = run_forward(K, x) + run_backward(K, x)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, run_forward(K, x) + run_backward(K, x)))
    tail = {n: (y if y is None or n in ("S0", "dS_T") else y[:, -24:].contiguous()) for n, y in x.items()}
    tail["S0"] = K.kda_hla_forward(*(x[n][:, :-24].contiguous() for n in ("q", "k", "v", "g")), x["S0"])[1]
    o64, S64 = forward64(tail)
    assert rel(first[0][:, -24:], o64) < TOL["bf16"] and rel(first[1], S64) < 2 * TOL_STATE["bf16"]
    for name, a, b in zip(("dq", "dk", "dv", "dg"), first[2:6], backward64(tail)):
        assert rel(a[:, -24:], b) < TOL["bf16"] * 4 / 3, name


def test_two_streams_at_once(K):
    """Calls on two streams, each with its own workspace, none waiting for the other."""
    xs = [inputs(1, 700, 6, 128, 128, "bf16", seed=16 + i) for i in range(2)]
    want = [run_forward(K, x) + run_backward(K, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], stream=s)
               + K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_and_replayed(K):
    """Prefill, backward pass and a decode step captured in one graph, replayed on other inputs in the same places."""
    x, y = inputs(2, 190, 3, 128, 128, "bf16", seed=18), inputs(2, 190, 3, 128, 128, "bf16", seed=19)
    tok = [x[n][:, 0].contiguous() for n in ("q", "k", "v", "g")]
    S = x["S0"].clone()
    args = (x["q"], x["k"], x["v"], x["g"])

    def step():
        f = K.kda_hla_forward(*args, x["S0"])
        b = K.kda_hla_backward(*args, x["do"], x["S0"], x["dS_T"])
        return (*f, *b, K.kda_hla_decode_step(*tok, S))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in ("q", "k", "v", "g", "do", "S0", "dS_T"):
        x[n].copy_(y[n])
    S.copy_(y["S0"])
    for t, n in zip(tok, ("q", "k", "v", "g")):
        t.copy_(y[n][:, 0])
    graph.replay()
    torch.cuda.synchronize()
    got = [z.clone() for z in out]
    S2 = y["S0"].clone()
    want = (*run_forward(K, y), *run_backward(K, y), K.kda_hla_decode_step(*(y[n][:, 0].contiguous() for n in ("q", "k", "v", "g")), S2))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(S, S2)


def test_backward_of_many_heads_captured_and_on_two_streams(K):
    """More chains than SMs: the last heads' chains and the first heads' gradients run side by side, in a graph and beside
    another stream's as on their own."""
    xs = [inputs(1, 700, 90, 64, 64, "bf16", seed=40 + i) for i in range(2)]
    want = [run_backward(K, x) for x in xs]

    def call(x, **kw):
        return K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], **kw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(xs[0])
    for i in (0, 1, 0):
        for n in ("q", "k", "v", "g", "do", "S0", "dS_T"):
            xs[0][n].copy_(inputs(1, 700, 90, 64, 64, "bf16", seed=40 + i)[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [call(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_no_tokens(K):
    x = inputs(2, 0, 3, 128, 128, "bf16", seed=20)
    o, S = run_forward(K, x)
    assert o.numel() == 0 and torch.equal(S, x["S0"])
    out = run_backward(K, x)
    assert torch.equal(out[4], x["dS_T"])
    c = torch.zeros(4, dtype=torch.int32, device="cuda")  # three empty sequences in front of tokens of none
    x = inputs(1, 9, 2, 64, 64, "f32", seed=21, N=3)
    o, S = K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], None, cu_seqlens=c)
    assert (S == 0).all()


def test_offsets_past_the_tensors_are_clamped(K):
    """Offsets that reach past the tokens, or fall, never lead outside the tensors."""
    x = inputs(1, 100, 2, 128, 128, "bf16", seed=22, N=3)
    for cu in ([0, 50, 1000, 2000], [0, 80, 40, 100], [-7, 3, 3, 100]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        K.kda_hla_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=c)
        K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS_T"], cu_seqlens=c)
        torch.cuda.synchronize()


def test_more_elements_than_32_bits_count(K):
    """Tensors and states of more than 2^31 elements: the last tokens, and the last requests, against calls on them alone."""
    T, H, d, tail = 175000, 96, 128, 300
    assert T * H * d > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(25)
    q, k, v, do = (torch.randn(1, T, H, d, generator=gen, device="cuda", dtype=torch.bfloat16) * 0.1 for _ in range(4))
    g = -torch.rand(1, T, H, generator=gen, device="cuda").bfloat16() * 0.1
    end = lambda x: x[:, T - tail:].contiguous()  # noqa: E731
    _, S0 = K.kda_hla_forward(*(x[:, :T - tail] for x in (q, k, v, g)))
    o, S = K.kda_hla_forward(q, k, v, g)
    o2, S2 = K.kda_hla_forward(end(q), end(k), end(v), end(g), S0)
    assert rel(end(o), o2) < 3 * 2.0 ** -8 and rel(S, S2) < 4 * TOL_STATE["bf16"]
    del o
    whole = K.kda_hla_backward(q, k, v, g, do)
    part = K.kda_hla_backward(*(end(x) for x in (q, k, v, g, do)), S0)
    for a, b in zip(whole[:4], part[:4]):  # (chunks end elsewhere: other roundings on both sides)
        assert rel(end(a), b) < 2 * TOL["bf16"]
    del whole
    inv, _ = K.kda_rope_inv_freq(64, device="cuda")
    at = torch.arange(T, device="cuda", dtype=torch.int32).unsqueeze(0)
    a, _ = K.kda_rope(q, None, inv, positions=at)
    b, _ = K.kda_rope(end(q), None, inv, positions=at[:, T - tail:].contiguous())
    assert torch.equal(end(a), b)
    del q, k, v, do, a
    N = 1400
    assert N * H * d * d > 2 ** 31
    S = torch.randn(N, H, d, d, generator=gen, device="cuda")
    x = [torch.randn(N, H, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    g = -torch.rand(N, H, generator=gen, device="cuda").bfloat16()
    S2 = S[-2:].clone()
    o = K.kda_hla_decode_step(*x, g, S)
    o2 = K.kda_hla_decode_step(*(y[-2:].contiguous() for y in x), g[-2:].contiguous(), S2)
    assert torch.equal(o[-2:], o2) and torch.equal(S[-2:], S2)


def test_python_refusals(K):
    x = inputs(1, 64, 2, 64, 64, "f32", seed=23)
    call = lambda **kw: K.kda_hla_forward(**{**dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], S0=x["S0"]), **kw})  # noqa: E731
    with pytest.raises(ValueError):
        call(q=x["q"].bfloat16())
    with pytest.raises(ValueError):
        call(g=x["g"].double())
    with pytest.raises(ValueError):
        call(q=x["q"].transpose(1, 2))
    with pytest.raises(ValueError):
        call(S0=x["S0"][:, :1])
    with pytest.raises(ValueError):
        call(v=x["v"].cpu())
    with pytest.raises(ValueError):
        call(g=x["g"][0, 0].double())
    with pytest.raises(K.KdaError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        K.kda_hla_backward(x["q"], x["k"], x["v"], x["g"], x["do"][:, :5])
    y = inputs(1, 64, 2, 96, 64, "f32", seed=24)
    with pytest.raises(K.KdaError):
        K.kda_hla_forward(y["q"], y["k"], y["v"], y["g"])
