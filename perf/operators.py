"""Cases for the linear-attention operators with one decay per head, and for rotary positions.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t            (per sequence and head)

  forward   a prompt: all o_t and the state after the last token, from a state S0 or none; dense or packed batches
  backward  the gradients of q, k, v, g and S0 from those of the outputs and of the last state
  decode    one token for each of N requests, the states updated in place
  rope      the positions' rotation of q and k ahead of them, or (inverse) of their gradients

States are fp32 [N, H, dv, dk]. The log-decay g is [B, T, H] in the activations' type (gate "token"), or fp32 [H],
one number per head (gate "head", which has no gradient). `run` computes the operators in elementary torch
operations, or, where `own` is set, by the calls a program makes of the framework.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HEAD_DIMS = (32, 64, 128)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the layer's prefill: 96 heads of 128 channels over one prompt of 8192 tokens
        _attn("fwd_h96_t8192_bf16", "forward", "bf16", B=1, T=8192, H=96, dk=128, dv=128),
        # serving: prompts of very different lengths packed in one batch, some of them continued (a state S0);
        # an empty one, single tokens and lengths that end inside a tile among them
        _attn("fwd_packed_bf16", "forward", "bf16", T=0, H=32, dk=128, dv=128, s0=True,
              lens="1,4099,700,0,64,2500,129,1,317,1024,77,6001"),
        # one long prompt with few heads, whose decays are fixed numbers
        _attn("fwd_long_h8_t65536_bf16", "forward", "bf16", B=1, T=65536, H=8, dk=128, dv=128, gate="head"),
        # the smallest prompt, in fp32, where latency counts
        _attn("fwd_small_t256_d32_f32", "forward", "f32", B=1, T=256, H=1, dk=32, dv=32),
        # a training step's backward pass: two sequences of 2048 tokens with a few heads, through the states
        _attn("bwd_b2_h4_t2048_bf16", "backward", "bf16", B=2, T=2048, H=4, dk=128, dv=128, s0=True),
        # the layer's backward pass over one long sequence
        _attn("bwd_h96_t8192_bf16", "backward", "bf16", B=1, T=8192, H=96, dk=128, dv=128),
        # training in fp32: packed sequences of odd lengths, other head sizes
        _attn("bwd_packed_f32", "backward", "f32", T=0, H=16, dk=64, dv=128, s0=True, lens="333,1,1200,65,500"),
        # one step of a full serving batch
        _attn("dec_n256_h96_bf16", "decode", "bf16", B=256, T=1, H=96, dk=128, dv=128, s0=True),
        # one step of a single request
        _attn("dec_n1_h32_bf16", "decode", "bf16", B=1, T=1, H=32, dk=128, dv=128, s0=True),
        # the prompt's q and k rotated, half layout, all channels
        _rope("rope_h96_t8192_bf16", "bf16", B=1, T=8192, H=96, d=128, rot=128),
        # a serving batch's single tokens, far positions, interleaved pairs in half of the head
        _rope("rope_n256_far_bf16", "bf16", B=256, T=1, H=32, d=128, rot=64, interleaved=True, far=1 << 20),
        # the gradients rotated back, fp32
        _rope("rope_back_f32", "f32", B=2, T=2047, H=16, d=64, rot=64, inverse=True, mscale=1.25),
    ]


def _attn(name, op, dtype, *, T, H, dk, dv, B=1, gate="token", s0=False, lens=""):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "T": sum(map(int, lens.split(","))) if lens else T, "H": H,
            "dk": dk, "dv": dv, "gate": gate, "s0": s0, "lens": lens}


def _rope(name, dtype, *, B, T, H, d, rot, interleaved=False, inverse=False, far=0, mscale=1.0):
    return {"name": name, "op": "rope", "dtype": dtype, "B": B, "T": T, "H": H, "d": d, "rot": rot,
            "interleaved": interleaved, "inverse": inverse, "far": far, "mscale": mscale}


def draw(rng):
    """One more case: lengths from one token to 65536, 1 to 96 heads, at most the listed prefill's token rows."""
    spread = lambda lo, hi: min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))  # noqa: E731
    op = rng.choice(("forward", "forward", "backward", "backward", "decode", "rope"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    H = spread(1, 96)
    if op == "rope":
        d = rng.choice((32, 64, 96, 128, 256))
        rows = spread(1, 786432 * 128 // d // H)
        B = rng.choice((1, 1, 2, 3, 8)) if rows >= 8 else 1
        c = _rope("", dtype, B=B, T=max(1, rows // B), H=H, d=d, rot=2 * rng.randrange(1, d // 2 + 1),
                  interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, far=rng.choice((0, 0, 1 << 17, 1 << 20)),
                  mscale=rng.choice((1.0, 1.0, 0.75, 1.3)))
        c.pop("name")
        return c
    dk, dv = rng.choice(HEAD_DIMS), rng.choice(HEAD_DIMS)
    if rng.random() < 0.5:
        dk = dv = 128
    gate = rng.choice(("token", "token", "head"))
    if op == "decode":
        c = _attn("", op, dtype, B=spread(1, 256), T=1, H=H, dk=dk, dv=dv, gate=gate, s0=True)
    else:
        tokens = spread(1, min(65536, 786432 // H) // (2 if dtype == "f32" else 1))
        B, lens = rng.choice((1, 1, 2, 3, 5)) if tokens >= 8 else 1, ""
        if tokens >= 8 and rng.random() < 0.4:  # packed: cuts anywhere, so that empty and one-token sequences come up
            cuts = sorted([0, tokens] + [rng.randrange(tokens + 1) for _ in range(rng.randrange(1, 12))] + [tokens // 2] * rng.randrange(2))
            B, lens = 1, ",".join(str(b - a) for a, b in zip(cuts, cuts[1:]))
        c = _attn("", op, dtype, B=B, T=max(1, tokens // B), H=H, dk=dk, dv=dv, gate=gate, s0=rng.random() < 0.5, lens=lens)
    c.pop("name")
    return c


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) % (1 << 62))
    dt = TYPES[case["dtype"]]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    B, T, H = case["B"], case["T"], case["H"]
    if case["op"] == "rope":
        d, half = case["d"], case["rot"] // 2
        at = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T)
        if case["far"]:  # every sequence somewhere in a long context
            at = at + torch.randint(0, case["far"], (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        inv = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float32, device="cuda")
        return {"case": case, "q": randn(B, T, H, d).to(dt), "k": randn(B, T, H, d).to(dt), "positions": at.contiguous(), "inv_freq": inv}
    dk, dv = case["dk"], case["dv"]
    lens = [int(x) for x in case["lens"].split(",")] if case["lens"] else None
    N = len(lens) if lens else B
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)  # noqa: E731
    # heads that remember from about two tokens to about five hundred, as models with such decays spread theirs
    rate = torch.exp2(-(1.0 + 8.0 * torch.arange(H, device="cuda") / max(1, H - 1)))
    if case["gate"] == "head":
        g = -rate
    else:
        g = (-2.0 * rate * torch.sigmoid(randn(B, T, H))).to(dt)
    s = {"case": case, "lens": lens, "scale": dk ** -0.5, "q": unit(randn(B, T, H, dk)).to(dt), "k": unit(randn(B, T, H, dk)).to(dt),
         "v": randn(B, T, H, dv).to(dt), "g": g, "cu": None, "S0": None}
    if lens:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda")
    if case["s0"]:
        s["S0"] = 0.1 * randn(N, H, dv, dk)
    if case["op"] == "backward":
        s["do"] = randn(B, T, H, dv).to(dt)
        s["dS_T"] = 0.1 * randn(N, H, dv, dk) if case["s0"] else None
    if case["op"] == "decode":
        for x in "qkv":
            s[x] = s[x][:, 0].contiguous()
        s["g"] = s["g"] if case["gate"] == "head" else s["g"][:, 0].contiguous()
    return s


# ------------------------------------------------------------------- runs
def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "rope":
        return _plain_rope(state, c)
    if c["op"] == "decode":
        return _plain_decode(state)
    back = c["op"] == "backward"
    xs = [state[x] for x in ("q", "k", "v")] + ([state["do"]] if back else [])
    g = state["g"].expand(xs[0].shape[:3])
    if state["lens"]:
        *xs, g = _padded(xs + [g.unsqueeze(-1)], state["lens"], state["cu"])
        g = g.squeeze(-1)
    f = _plain_backward if back else _plain_forward
    extra = (state["S0"], state["dS_T"], state["scale"]) if back else (state["S0"], state["scale"])
    out = list(f(*xs, g, *extra))
    if state["lens"]:
        n = 4 if back else 1
        out[:n] = [_packed(x, state["lens"], state["cu"]) for x in out[:n]]
    if back and c["gate"] == "head":
        out[3] = None
    dt = TYPES[c["dtype"]]
    n = 4 if back else 1
    return tuple(x if x is None else x.to(dt) for x in out[:n]) + tuple(out[n:])


def _own(state, c):
    from linear_attention_recurrence_11_b200 import kda
    if c["op"] == "rope":
        return kda.kda_rope(state["q"], state["k"], state["inv_freq"], positions=state["positions"],
                            interleaved=c["interleaved"], mscale=c["mscale"], inverse=c["inverse"])
    q, k, v, g = (state[x] for x in ("q", "k", "v", "g"))
    if c["op"] == "decode":
        return kda.kda_hla_decode_step(q, k, v, g, state["S0"], scale=state["scale"]), state["S0"]
    if c["op"] == "forward":
        return kda.kda_hla_forward(q, k, v, g, state["S0"], scale=state["scale"], cu_seqlens=state["cu"])
    return kda.kda_hla_backward(q, k, v, g, state["do"], state["S0"], state["dS_T"], scale=state["scale"], cu_seqlens=state["cu"])


# ------------------------------------------------------------- plain forms
def _places(lens, cu):
    """For [N, longest] places of a padded batch: the packed token of each, and whether there is one."""
    at = torch.arange(max(max(lens), 1), device=cu.device)
    n = (cu[1:] - cu[:-1]).unsqueeze(1)
    return (cu[:-1].unsqueeze(1) + at).clamp(max=int(sum(lens)) - 1).long(), at < n


def _padded(xs, lens, cu):
    idx, there = _places(lens, cu)
    return [x[0][idx] * there[..., None, None] for x in xs]


def _packed(x, lens, cu):
    _, there = _places(lens, cu)
    return x[there].unsqueeze(0)


def _chunked(g, *xs):
    """g [B, T, H] and xs [B, T, H, d] as [B, H, n, C, ...]: fp32, padded with zeros, which change nothing."""
    T = g.shape[1]
    C = 64 if T <= 16384 else 256
    pad = -T % C
    lay = lambda x: torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad)).unflatten(1, (-1, C)).permute(0, 3, 1, 2, 4)  # noqa: E731
    return lay(g.unsqueeze(-1)).squeeze(-1), [lay(x) for x in xs]


def _flat(x, T):
    return x.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :T]


def _decays(g):
    """Of [B, H, n, C] log-decays, all sums in fp64: D (row r, column s <= r) within a chunk, from a chunk's start to
    each token, from each token to the chunk's end, and between the chunks' borders: E [n + 1, n + 1], row >= column."""
    G = g.double().cumsum(-1)
    C, n = g.shape[-1], g.shape[-2]
    low = torch.ones(C, C, dtype=torch.bool, device=g.device).tril()
    D = torch.where(low, G.unsqueeze(-1) - G.unsqueeze(-2), -math.inf).exp().float()
    border = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))
    low = torch.ones(n + 1, n + 1, dtype=torch.bool, device=g.device).tril()
    E = torch.where(low, border.unsqueeze(-1) - border.unsqueeze(-2), -math.inf).exp().float()
    return D, G.exp().float().unsqueeze(-1), (G[..., -1:] - G).exp().float().unsqueeze(-1), E


def _states(E, k, v, into, S0):
    """The states [B, H, n + 1, dk, dv] at the chunks' borders, from each chunk's own sum of k v^T."""
    own_sums = (k * into).transpose(-1, -2) @ v
    S = (E[..., 1:] @ own_sums.flatten(-2)) if S0 is None else (E @ torch.cat([S0.mT.unsqueeze(2), own_sums], 2).flatten(-2))
    return S.unflatten(-1, own_sums.shape[-2:])


def _plain_forward(q, k, v, g, S0, scale):
    T = q.shape[1]
    g, (q, k, v) = _chunked(g, q, k, v)
    D, since, until, E = _decays(g)
    S = _states(E, k, v, until, S0)
    o = ((q @ k.mT) * D) @ v + since * (q @ S[:, :, :-1])
    return _flat(scale * o, T), S[:, :, -1].mT.contiguous()


def _plain_backward(q, k, v, do, g, S0, dS_T, scale):
    T = q.shape[1]
    g, (q, k, v, do) = _chunked(g, q, k, v, do)
    do = scale * do
    D, since, until, E = _decays(g)
    S = _states(E, k, v, until, S0)
    # the states' gradients at the borders: the same sums, from the last token to the first
    sums = (q * since).mT @ do
    back = E.mT
    dS = (back[..., :-1] @ sums.flatten(-2)) if dS_T is None else (back @ torch.cat([sums, dS_T.mT.unsqueeze(2)], 2).flatten(-2))
    dS = dS.unflatten(-1, sums.shape[-2:])
    A, dA = (q @ k.mT) * D, (do @ v.mT) * D
    S0c, dS1 = S[:, :, :-1], dS[:, :, 1:]
    from_before, from_after = since * (do @ S0c.mT), until * (v @ dS1.mT)
    dq = dA @ k + from_before
    dk = dA.mT @ q + from_after
    dv = A.mT @ do + until * (k @ dS1)
    # g_t scales whatever a token from t on reads of one before t: pairs within the chunk, the chunk's later tokens
    # with the state before it, its earlier ones with the gradient behind it, and what passes through it as a whole
    C = g.shape[-1]
    low = torch.ones(C, C, dtype=torch.bool, device=g.device).tril()
    before = torch.nn.functional.pad(((q @ k.mT) * dA).double().cumsum(-1)[..., :-1], (1, 0))
    within = torch.where(low, before, 0.0).sum(-2)
    read = (q * from_before).double().sum(-1).flip(-1).cumsum(-1).flip(-1)
    written = torch.nn.functional.pad((k * from_after).double().sum(-1).cumsum(-1)[..., :-1], (1, 0))
    through = since[..., -1, 0] * (S0c.double() * dS1.double()).sum((-1, -2))
    dg = within + read + written + through.unsqueeze(-1)
    return (*(_flat(x, T) for x in (dq, dk, dv)), _flat(dg.unsqueeze(-1), T).squeeze(-1), dS[:, :, 0].mT.contiguous())


def _plain_decode(s):
    q, k, v, S = s["q"].float(), s["k"].float(), s["v"].float(), s["S0"]
    S.mul_(s["g"].float().exp()[..., None, None].expand(*q.shape[:2], 1, 1)).add_(v.unsqueeze(-1) * k.unsqueeze(-2))
    return (s["scale"] * (S * q.unsqueeze(-2)).sum(-1)).to(s["q"].dtype), S


def _plain_rope(s, c):
    a = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    cos, sin = (c["mscale"] * a.cos()).float(), (c["mscale"] * (-a.sin() if c["inverse"] else a.sin())).float()
    return tuple(_rotated(s[x].float(), cos, sin, c).to(s[x].dtype) for x in ("q", "k"))


def _rotated(x, cos, sin, c):
    r, h = c["rot"], c["rot"] // 2
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :h], x[..., h:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1), x[..., r:]], -1)


# ------------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    rows = case["B"] * case["T"] * case["H"]
    if case["op"] == "rope":
        return {"bytes": rows * case["d"] * es * 4 + case["B"] * case["T"] * 4, "flops": rows * case["rot"] * 6}
    dk, dv = case["dk"], case["dv"]
    N = len(case["lens"].split(",")) if case["lens"] else case["B"]
    state = 4 * N * case["H"] * dk * dv
    gate = rows * es if case["gate"] == "token" else case["H"] * 4
    if case["op"] == "decode":
        return {"bytes": rows * (2 * dk + 2 * dv) * es + gate + 2 * state, "flops": 5 * rows * dk * dv}
    if case["op"] == "forward":
        return {"bytes": rows * (2 * dk + 2 * dv) * es + gate + state * (2 if case["s0"] else 1), "flops": 5 * rows * dk * dv}
    return {"bytes": rows * (4 * dk + 3 * dv) * es + gate * (2 if case["gate"] == "token" else 1) + state * (3 if case["s0"] else 1),
            "flops": 14 * rows * dk * dv}


# --------------------------------------------------- the definition in fp64
def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda x: None if x is None else x.double()  # noqa: E731
    if case["op"] == "rope":
        turn = torch.polar(torch.full((), float(case["mscale"]), dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, :, None, None] * s["inv_freq"].double())
        turn = turn.conj() if case["inverse"] else turn
        out = []
        for x in (s["q"].double(), s["k"].double()):
            y, r = x.clone(), case["rot"]
            ev, od = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., ev].contiguous(), x[..., od].contiguous()) * turn
            y[..., ev], y[..., od] = z.real, z.imag
            out.append(y)
        return tuple(out)
    q, k, v, g, S0 = (f64(s[x]) for x in ("q", "k", "v", "g", "S0"))
    scale, H, dk, dv = s["scale"], case["H"], case["dk"], case["dv"]
    if case["op"] == "decode":
        S = S0 * g.exp()[..., None, None] + torch.einsum("nhj,nhi->nhji", v, k)
        return scale * torch.einsum("nhji,nhi->nhj", S, q), S
    g = g.expand(q.shape[:3])
    lens = s["lens"] or [case["T"]] * case["B"]
    N, T = len(lens), max(max(lens), 1)
    if T * N * H * dk * dv > 2e11:  # some seconds
        return None
    # token by token over all sequences side by side; one that has ended takes a token that changes nothing
    spans = [(0, sum(lens[:i])) for i in range(N)] if s["lens"] else [(i, 0) for i in range(N)]

    def side_by_side(x):
        y = torch.zeros(N, T, *x.shape[2:], dtype=torch.float64, device="cuda")
        for i, (b, t0) in enumerate(spans):
            y[i, :lens[i]] = x[b, t0:t0 + lens[i]]
        return y

    def back_in_place(y, like):
        x = torch.zeros(like.shape[:2] + y.shape[2:], dtype=torch.float64, device="cuda")
        for i, (b, t0) in enumerate(spans):
            x[b, t0:t0 + lens[i]] = y[i, :lens[i]]
        return x

    Q, K, V, G = (side_by_side(x) for x in (q, k, v, g))
    keep = G.exp()[..., None, None]
    S = torch.zeros(N, H, dv, dk, dtype=torch.float64, device="cuda") if S0 is None else S0.clone()
    if case["op"] == "forward":
        O = torch.empty_like(V)
        for t in range(T):
            S.mul_(keep[:, t]).add_(V[:, t].unsqueeze(-1) * K[:, t].unsqueeze(-2))
            O[:, t] = (S @ Q[:, t].unsqueeze(-1)).squeeze(-1)
        return back_in_place(scale * O, v), S
    dO = scale * side_by_side(s["do"].double())
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    for t in range(T):
        S.mul_(keep[:, t]).add_(V[:, t].unsqueeze(-1) * K[:, t].unsqueeze(-2))
        dQ[:, t] = (S.mT @ dO[:, t].unsqueeze(-1)).squeeze(-1)
    R = torch.zeros_like(S) if s["dS_T"] is None else s["dS_T"].double()
    last = (S * R).sum((-1, -2))
    for t in reversed(range(T)):
        R = R + dO[:, t].unsqueeze(-1) * Q[:, t].unsqueeze(-2)
        dK[:, t] = (R.mT @ V[:, t].unsqueeze(-1)).squeeze(-1)
        dV[:, t] = (R @ K[:, t].unsqueeze(-1)).squeeze(-1)
        R = R * keep[:, t]
    dG = ((Q * dQ).sum(-1) - (K * dK).sum(-1)).flip(1).cumsum(1).flip(1) + last.unsqueeze(1)
    if S0 is None:
        dG[:, 0] = 0.0  # there is no state that the first token's decay could scale
    return (back_in_place(dQ, q), back_in_place(dK, k), back_in_place(dV, v), back_in_place(dG, g) if case["gate"] == "token" else None, R)
