"""Linear attention with one decay per head, token by token in fp64 (the definition), and seeded inputs."""
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, T, H, dk, dv, dtype, *, seed, gate="token", s0=True, N=None, rate=None, device="cuda"):
    """q, k, v, g, do, S0, dS_T. Decay rates from 2^-1 to 2^-9 per token over the heads, unless `rate` is given."""
    gen = torch.Generator(device=device).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
    dt = DT[dtype]
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)  # noqa: E731
    r = torch.exp2(-(1.0 + 8.0 * torch.arange(H, device=device) / max(1, H - 1))) if rate is None else torch.full((H,), rate, device=device)
    g = -r if gate == "head" else (-2.0 * r * torch.sigmoid(randn(B, T, H))).to(dt)
    N = B if N is None else N
    return dict(q=unit(randn(B, T, H, dk)).to(dt), k=unit(randn(B, T, H, dk)).to(dt), v=randn(B, T, H, dv).to(dt), g=g,
                do=randn(B, T, H, dv).to(dt), S0=0.3 * randn(N, H, dv, dk) if s0 else None,
                dS_T=0.3 * randn(N, H, dv, dk) if s0 else None)


def _spans(x, cu):
    B, T = x["q"].shape[:2]
    return [(b, 0, T) for b in range(B)] if cu is None else [(0, a, b) for a, b in zip(cu, cu[1:])]


def _seq(x, b, t0, t1):
    g = x["g"] if x["g"].dim() == 3 else x["g"].expand(x["q"].shape[:3])
    return [x[n][b, t0:t1].double() for n in ("q", "k", "v")] + [g[b, t0:t1].double()]


def forward64(x, scale=1.0, cu=None):
    """o [B, T, H, dv] (zero outside the sequences) and S_T, in fp64."""
    H, dk, dv = x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]
    o = torch.zeros(x["v"].shape, dtype=torch.float64, device=x["v"].device)
    out = []
    for n, (b, t0, t1) in enumerate(_spans(x, cu)):
        q, k, v, g = _seq(x, b, t0, t1)
        S = torch.zeros(H, dv, dk, dtype=torch.float64, device=o.device) if x["S0"] is None else x["S0"][n].double()
        for t in range(t1 - t0):
            S = S * g[t].exp()[:, None, None] + v[t, :, :, None] * k[t, :, None, :]
            o[b, t0 + t] = scale * (S * q[t, :, None, :]).sum(-1)
        out.append(S)
    return o, torch.stack(out)


def backward64(x, scale=1.0, cu=None):
    """dq, dk, dv, dg [B, T, H], dS0 in fp64, by automatic differentiation of the definition."""
    H, dk, dv = x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]
    full = [torch.zeros(x[n].shape, dtype=torch.float64, device=x["q"].device) for n in ("q", "k", "v")]
    dg = torch.zeros(x["q"].shape[:3], dtype=torch.float64, device=x["q"].device)
    dS0 = []
    for n, (b, t0, t1) in enumerate(_spans(x, cu)):
        with torch.enable_grad():
            q, k, v, g = (y.detach().clone().requires_grad_() for y in _seq(x, b, t0, t1))
            S0 = torch.zeros(H, dv, dk, dtype=torch.float64, device=q.device) if x["S0"] is None else x["S0"][n].double()
            S0.requires_grad_()
            S, loss = S0, torch.zeros((), dtype=torch.float64, device=q.device)
            do = x["do"][b, t0:t1].double()
            for t in range(t1 - t0):
                S = S * g[t].exp()[:, None, None] + v[t, :, :, None] * k[t, :, None, :]
                loss = loss + (do[t] * scale * (S * q[t, :, None, :]).sum(-1)).sum()
            if x["dS_T"] is not None:
                loss = loss + (S * x["dS_T"][n].double()).sum()
            loss = loss + 0.0 * (S0.sum() + g.sum() + q.sum() + k.sum() + v.sum())
            grads = torch.autograd.grad(loss, [q, k, v, g, S0])
        for y, z in zip(full, grads[:3]):
            y[b, t0:t1] = z
        dg[b, t0:t1] = torch.where(torch.isnan(grads[3]), 0.0, grads[3])
        dS0.append(grads[4])
    return (*full, dg, torch.stack(dS0))


def rel(a, b):
    """2-norm of the difference over that of the reference."""
    a, b = a.double(), b.double()
    n = float(torch.linalg.vector_norm(b))
    d = float(torch.linalg.vector_norm(a - b))
    return d / n if n else d
