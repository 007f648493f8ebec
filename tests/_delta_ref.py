"""The gated delta rule and the root-mean-square norm in 64 bits, on the host,
written from their definitions; gradients by torch's differentiation of them."""
from __future__ import annotations

import torch


def delta_inputs(b, t, h, g, p, n, dtype, seed, decay=True):
    """Seeded inputs with unit keys and queries, stored in the io dtype."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    def unit(v):
        return (v / v.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(dtype)

    x = {"q": unit(normal(b, t, g, n)), "k": unit(normal(b, t, g, n) + 0.3 * normal(g, n)), "v": normal(b, t, h, p).to(dtype),
         "g": (-torch.rand(b, t, h, generator=gen, dtype=torch.float64) * 0.5).float() if decay else None,
         "beta": torch.rand(b, t, h, generator=gen, dtype=torch.float64).float(),
         "h0": normal(b, h, n, p).float(), "dy": normal(b, t, h, p).to(dtype), "dh": normal(b, h, n, p).float()}
    return x


def delta(q, k, v, g, beta, scale, h0=None, lengths=None):
    """y [b][t][h][p] (zero behind a sequence's end) and the final state, float64."""
    b, t, h, p = v.shape
    rep = h // q.shape[2]
    q, k = q.double().repeat_interleave(rep, 2), k.double().repeat_interleave(rep, 2)
    v, beta = v.double(), beta.double()
    a = torch.exp(g.double()) if g is not None else torch.ones_like(beta)
    s = torch.zeros(b, h, q.shape[3], p, dtype=torch.float64) if h0 is None else h0.double()
    ends = torch.full((b,), t) if lengths is None else lengths.clamp(0, t)
    ys = []
    for i in range(t):
        old = a[:, i, :, None, None] * s
        u = beta[:, i, :, None] * (v[:, i] - torch.einsum("bhnp,bhn->bhp", old, k[:, i]))
        new = old + torch.einsum("bhn,bhp->bhnp", k[:, i], u)
        live = (i < ends)[:, None, None]
        s = torch.where(live[..., None], new, s)
        ys.append(torch.where(live, scale * torch.einsum("bhnp,bhn->bhp", new, q[:, i]), 0.0))
    return (torch.stack(ys, 1) if ys else v.clone()), s


def delta_grads(x, scale, lengths=None, init=True, d_final=True):
    """Gradients of <dy, y> + <dh, final state> as a dict of float64 tensors."""
    names = [n for n in ("q", "k", "v", "g", "beta") if x[n] is not None] + (["h0"] if init else [])
    leaf = {n: x[n].double().requires_grad_() for n in names}
    y, s = delta(leaf["q"], leaf["k"], leaf["v"], leaf.get("g"), leaf["beta"], scale, leaf.get("h0"), lengths)
    ends = torch.full((y.shape[0],), y.shape[1]) if lengths is None else lengths.clamp(0, y.shape[1])
    live = (torch.arange(y.shape[1])[None] < ends[:, None])[..., None, None]
    j = torch.where(live, x["dy"].double() * y, 0.0).sum() + ((x["dh"].double() * s).sum() if d_final else 0.0)
    return dict(zip(names, torch.autograd.grad(j, list(leaf.values()), allow_unused=True)))


def norm(x, eps, residual=None, weight=None):
    """(sum, y) of the norm, float64."""
    s = x.double() + (residual.double() if residual is not None else 0.0)
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return s, y * weight.double() if weight is not None else y


def norm_grads(s, dy, eps, weight=None, d_sum=None):
    leaf = s.double().requires_grad_()
    w = weight.double().requires_grad_() if weight is not None else None
    _, y = norm(leaf, eps, weight=w)
    d = torch.autograd.grad((y * dy.double()).sum(), [leaf] + ([w] if w is not None else []))
    return d[0] + (d_sum.double() if d_sum is not None else 0.0), (d[1] if w is not None else None)


def rel(got, want):
    """Relative 2-norm of the difference; a wrong non-finite value counts as infinite."""
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    if not bool(torch.isfinite(got).all()):
        return float("inf")
    d, n = (got - want).norm().item(), want.norm().item()
    return d / n if n > 0 else d
