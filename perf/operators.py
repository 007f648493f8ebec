"""Measured cases of the gated delta rule (prefill, one token, gradient) and of the
root-mean-square norm (with the residual's addition, and its gradient).

``run`` computes a case in its plain form, elementary torch operations in 32 bits;
with ``own`` it calls the library (``m3_delta_fwd``, ``m3_delta_step``,
``m3_delta_bwd``, ``m3_rms_norm_fwd``, ``m3_rms_norm_bwd``).  ``exact`` gives the
same outputs from the definitions, token by token in 64 bits.

Layouts: q, k [batch][seqlen][groups][dstate], v, y [batch][seqlen][heads][headdim],
g (log decay), beta [batch][seqlen][heads], state [batch][heads][dstate][headdim].
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _delta(name, op, batch, seqlen, nheads, ngroups, headdim=64, dstate=128, dtype="bf16", ragged=False, init=False):
    return dict(name=name, op=op, batch=batch, seqlen=seqlen, nheads=nheads, ngroups=ngroups, headdim=headdim,
                dstate=dstate, dtype=dtype, ragged=ragged, init=init)


def _norm(name, op, rows, width, dtype="bf16", residual=True, out="io", block=0, weight=True):
    return dict(name=name, op=op, rows=rows, width=width, dtype=dtype, residual=residual, out=out, block=block,
                weight=weight)


def listed():
    return [
        # the prompt pass of a 1.5B-scale layer: a batch of full prompts, a state kept for decoding
        _delta("prefill_layer", "prefill", 8, 4096, 32, 32),
        # one long document, few sequences: the chain over chunks is what takes the time
        _delta("prefill_long", "prefill", 1, 32768, 32, 32),
        # a padded batch that resumes from carried states, keys shared by a group of 8 heads
        _delta("prefill_resumed_ragged", "prefill", 4, 1531, 8, 1, ragged=True, init=True),
        # a small float32 model, odd head sizes
        _delta("prefill_f32_odd", "prefill", 3, 333, 4, 2, 40, 48, "f32", init=True),
        # decoding for 256 sequences: the states' traffic
        _delta("step_b256", "step", 256, 1, 32, 32),
        # decoding for one sequence: latency
        _delta("step_b1", "step", 1, 1, 8, 1),
        # a training step's gradient: a layer with grouped keys, and one with keys of every head
        _delta("gradient_grouped", "gradient", 4, 2048, 8, 1),
        _delta("gradient_layer", "gradient", 2, 4096, 32, 32),
        # the residual stream into a layer whose projections take 8-bit activations
        _norm("norm_e4m3", "norm", 32768, 2048, out="e4m3", block=128),
        # the same place when one token of a small batch is decoded
        _norm("norm_decode", "norm", 16, 2048),
        # the gradient of the residual stream's norm
        _norm("norm_gradient", "norm_gradient", 16384, 2048),
        # the gradient of the norm of keys and queries: many short float32 rows
        _norm("norm_gradient_keys_f32", "norm_gradient", 40001, 128, "f32", residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "gradient", "norm", "norm_gradient"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_gradient"):
        width = rng.choice([_log(rng, 64, 8192), 128, 2048, 4096])
        rows = _log(rng, 1, 60_000_000 // width)
        out = rng.choice(["io", "e4m3"]) if op == "norm" else "io"
        return dict(op=op, rows=rows, width=width, dtype=dtype, residual=rng.random() < 0.7, out=out,
                    block=rng.choice([0, 128]) if out == "e4m3" else 0, weight=rng.random() < 0.8)
    nheads = rng.choice([1, 4, 8, 12, 32])
    ngroups = rng.choice([g for g in (1, 2, 4, nheads) if nheads % g == 0])
    dstate, headdim = rng.choice([(128, 64), (128, 64), (128, 64), (128, 128), (64, 64), (48, 40)])
    if dtype == "f32":
        most = 40_000
    else:
        most = 600_000 if (dstate, headdim) == (128, 64) else 60_000
    if op == "gradient":
        most //= 6
    if op == "step":
        return dict(op=op, batch=_log(rng, 1, 256), seqlen=1, nheads=nheads, ngroups=ngroups, headdim=headdim,
                    dstate=dstate, dtype=dtype, ragged=False, init=True)
    seqlen = _log(rng, 1, 8192 if op == "prefill" else 2048)
    batch = max(1, min(16, _log(rng, 1, 16), most // (seqlen * nheads) if most >= seqlen * nheads else 1))
    return dict(op=op, batch=batch, seqlen=seqlen, nheads=nheads, ngroups=ngroups, headdim=headdim, dstate=dstate,
                dtype=dtype, ragged=rng.random() < 0.4, init=op == "prefill" and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --
def _inputs(case, seed):
    """The tensors that the operator reads, made from the seed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    io = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_gradient"):
        rows, width = case["rows"], case["width"]
        x = {"x": normal(rows, width).to(io)}
        if case["residual"]:
            x["r"] = (normal(rows, width) * 2.0).to(io)
        if case["weight"]:
            x["w"] = 1.0 + 0.2 * normal(width)
        if case["op"] == "norm_gradient":
            x["dy"] = normal(rows, width).to(io)
        return x
    b, t, h, g, p, n = (case[k] for k in ("batch", "seqlen", "nheads", "ngroups", "headdim", "dstate"))
    shared = normal(g, n)      # keys of a trained layer are not quite independent of one another

    def unit(v):
        return (v / v.square().sum(-1, keepdim=True).sqrt()).to(io)

    x = {"q": unit(normal(b, t, g, n)), "k": unit(normal(b, t, g, n) + 0.3 * shared), "v": normal(b, t, h, p).to(io)}
    a = -torch.exp(torch.rand(h, device="cuda", generator=gen) * 3.0 - 2.0)
    x["g"] = torch.log1p(torch.exp(normal(b, t, h) - (1.0 if t > 8192 else 0.0))) * a
    x["beta"] = torch.sigmoid(normal(b, t, h))
    if case["init"] or case["op"] == "step":
        x["h0"] = normal(b, h, n, p)
    if case["ragged"]:
        some = torch.randint(0, t + 1, (b,), device="cuda", generator=gen)
        some[0] = t            # one of the batch fills it
        x["lengths"] = some.to(torch.int32)
    if case["op"] == "gradient":
        x["dy"] = normal(b, t, h, p).to(io)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    s = {"case": case, "x": x}
    io = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]
        s["sum"] = torch.empty_like(x["x"]) if case["residual"] else None
        s["y"] = torch.empty_like(x["x"]) if case["out"] == "io" else None
        if case["out"] == "e4m3":
            s["y8"] = torch.empty(rows, width, device="cuda", dtype=torch.float8_e4m3fn)
            s["scale"] = torch.empty(rows, -(-width // case["block"]) if case["block"] else 1, device="cuda")
    elif case["op"] == "norm_gradient":
        s["dx"] = torch.empty_like(x["x"])
        s["dw"] = torch.empty(case["width"], device="cuda") if case["weight"] else None
    elif case["op"] == "prefill":
        s["y"] = torch.zeros_like(x["v"])          # rows behind a sequence's end stay as they are
        s["h"] = torch.empty(case["batch"], case["nheads"], case["dstate"], case["headdim"], device="cuda")
    elif case["op"] == "step":
        s["y"] = torch.empty_like(x["v"])
        s["h"] = torch.empty_like(x["h0"])
    else:
        s["d"] = {k: torch.empty_like(x[k]) for k in ("q", "k", "v")}
        for k in ("g", "beta"):
            s["d"][k] = torch.empty(x[k].shape, device="cuda", dtype=io)
    return s


# ------------------------------------------------------------- plain forms --
def _plain_delta(q, k, v, g, beta, scale, lengths, h0):
    """The chunked form: inside a chunk the triangular system of the delta rule, across chunks the state."""
    b, t, h, p = v.shape
    n, rep = q.shape[3], h // q.shape[2]
    g, beta, seen = g.float(), beta.float(), None
    if lengths is not None:
        seen = (torch.arange(t, device=v.device) < lengths[:, None])[..., None]
        g, beta = g * seen, beta * seen
    pad = -t % CHUNK
    nc = (t + pad) // CHUNK

    def chunks(x):             # [b][t][heads][...] -> [b][heads][chunk][CHUNK][...]
        x = torch.cat([x, x.new_zeros(b, pad, *x.shape[2:])], 1) if pad else x
        return x.reshape(b, nc, CHUNK, *x.shape[2:]).movedim(3, 1)

    qc, kc, vc, gc, bc = (chunks(x.float()) for x in (q, k, v, g, beta))
    kk, qk = kc @ kc.mT, qc @ kc.mT
    qc, kc, kk, qk = (x.repeat_interleave(rep, 1) for x in (qc, kc, kk, qk))
    cum = gc.double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=v.device, dtype=torch.bool).tril()
    gam = torch.where(low, torch.exp((cum[..., :, None] - cum[..., None, :]).float().clamp(max=0.0)), 0.0)
    x = -torch.tril(bc[..., None] * kk * gam, -1)
    eye = torch.eye(CHUNK, device=v.device)
    inv = eye + x              # (I - x)^-1 = (I + x)(I + x^2)(I + x^4)...
    for _ in range(int(math.log2(CHUNK)) - 1):
        x = x @ x
        inv = inv + x @ inv
    since, until = torch.exp(cum.float())[..., None], torch.exp((cum[..., -1:] - cum).float())[..., None]
    u, w = inv @ (bc[..., None] * vc), inv @ (bc[..., None] * since * kc)
    att, qd, kd, whole = qk * gam * scale, qc * since * scale, (kc * until).mT, torch.exp(cum[..., -1].float())
    s = h0.float() if h0 is not None else torch.zeros(b, h, n, p, device=v.device)
    ys = []
    for c in range(nc):
        new = u[:, :, c] - w[:, :, c] @ s
        ys.append(qd[:, :, c] @ s + att[:, :, c] @ new)
        s = whole[:, :, c, None, None] * s + kd[:, :, c] @ new
    y = torch.stack(ys, 2).movedim(1, 3).reshape(b, nc * CHUNK, h, p)[:, :t]
    return (y if seen is None else y * seen[..., None]), s


def _plain_step(x, scale):
    rep = x["v"].shape[2] // x["q"].shape[2]
    q, k = (x[n][:, 0].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    s = x["h0"] * torch.exp(x["g"][:, 0])[..., None, None]
    u = x["beta"][:, 0, :, None] * (x["v"][:, 0].float() - (s * k[..., None]).sum(2))
    s = s + k[..., None] * u[:, :, None]
    return (scale * (s * q[..., None]).sum(2))[:, None], s


def _plain_norm(case, x):
    s = x["x"].float() + x["r"].float() if case["residual"] else x["x"].float()
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    return s, y * x["w"] if case["weight"] else y


def _plain_e4m3(case, y):
    rows, width = y.shape
    block = case["block"] or width
    blocks = -(-width // block)
    z = torch.cat([y, y.new_zeros(rows, blocks * block - width)], 1) if blocks * block > width else y
    z = z.reshape(rows, blocks, block)
    scale = z.abs().amax(-1).clamp(min=1e-30) / 448.0
    return (z / scale[..., None]).reshape(rows, -1)[:, :width].to(torch.float8_e4m3fn), scale


def _plain_norm_gradient(case, x):
    # the norm's input is the stored sum, so the gradient of the sum is the residual stream's plus the norm's
    s = x["x"].float()
    dy = x["dy"].float()
    rs = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    hat = s * rs
    wdy = dy * x["w"] if case["weight"] else dy
    dx = rs * (wdy - hat * (wdy * hat).mean(-1, keepdim=True))
    if case["residual"]:
        dx = dx + x["r"].float()
    return dx, (dy * hat).sum(0)


EPS = 1e-5


def _scale(case):
    return case["dstate"] ** -0.5


def run(state):
    if own:
        return _run_own(state)
    case, x, io = state["case"], state["x"], DTYPES[state["case"]["dtype"]]
    if case["op"] == "norm":
        s, y = _plain_norm(case, x)
        out = {"sum": s.to(io)} if case["residual"] else {}
        if case["out"] == "io":
            return {**out, "y": y.to(io)}
        y8, scale = _plain_e4m3(case, y)
        return {**out, "y8": y8, "scale": scale}
    if case["op"] == "norm_gradient":
        dx, dw = _plain_norm_gradient(case, x)
        return {"dx": dx.to(io), **({"dw": dw} if case["weight"] else {})}
    if case["op"] == "step":
        y, h = _plain_step(x, _scale(case))
        return {"y": y.to(io), "h": h}
    if case["op"] == "prefill":
        y, h = _plain_delta(x["q"], x["k"], x["v"], x["g"], x["beta"], _scale(case), x.get("lengths"), x.get("h0"))
        return {"y": y.to(io), "h": h}
    with torch.enable_grad():
        leaf = {k: x[k].float().requires_grad_() for k in ("q", "k", "v", "g", "beta")}
        y, _ = _plain_delta(*leaf.values(), _scale(case), x.get("lengths"), None)
        d = torch.autograd.grad(y, list(leaf.values()), x["dy"].float())
    return {"d" + k: v.to(io) for k, v in zip(leaf, d)}


def _run_own(state):
    import selective_state_space_m3_b200 as m3

    case, x = state["case"], state["x"]
    io = m3.M3_BF16 if case["dtype"] == "bf16" else m3.M3_F32
    if case["op"] == "norm":
        m3.m3_rms_norm_fwd(x["x"], EPS, residual=x.get("r"), weight=x.get("w"), sum=state["sum"], y=state["y"],
                           y8=state.get("y8"), scale=state.get("scale"), scale_block=case["block"])
        return {k: state[k] for k in ("sum", "y", "y8", "scale") if state.get(k) is not None}
    if case["op"] == "norm_gradient":
        if "ws" not in state:
            size = m3.m3_rms_norm_bwd_workspace_size(case["rows"], case["width"], io)
            state["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        m3.m3_rms_norm_bwd(x["x"], x["dy"], EPS, state["dx"], state["ws"], weight=x.get("w"), d_sum=x.get("r"),
                           dweight=state["dw"])
        return {k: state[k] for k in ("dx", "dw") if state[k] is not None}
    if "dims" not in state:
        state["dims"] = m3.Dims(case["batch"], case["seqlen"], case["nheads"], case["ngroups"], case["headdim"],
                                case["dstate"], 1, CHUNK, io)
    dims = state["dims"]
    if case["op"] == "step":
        # a decoding program updates its state in place; here every pass starts from the same one
        m3.m3_delta_step(dims, x["h0"], x["q"], x["k"], x["v"], x["g"], x["beta"], state["y"], scale=_scale(case),
                         h_out=state["h"])
        return {"y": state["y"], "h": state["h"]}
    if case["op"] == "prefill":
        if "ws" not in state:
            state["ws"] = _workspace(m3.m3_delta_workspace_size(dims))
        m3.m3_delta_fwd(dims, x["q"], x["k"], x["v"], x["g"], x["beta"], state["y"], state["ws"], scale=_scale(case),
                        lengths=x.get("lengths"), init_h=x.get("h0"), final_h=state["h"])
        return {"y": state["y"], "h": state["h"]}
    if "ws" not in state:
        state["ws"] = _workspace(m3.m3_delta_bwd_workspace_size(dims))
    d = state["d"]
    m3.m3_delta_bwd(dims, x["q"], x["k"], x["v"], x["g"], x["beta"], x["dy"],
                    {"dq": d["q"], "dk": d["k"], "dv": d["v"], "dg": d["g"], "dbeta": d["beta"]}, state["ws"],
                    scale=_scale(case), lengths=x.get("lengths"))
    return {"d" + k: d[k] for k in ("q", "k", "v", "g", "beta")}


def _workspace(size):
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    ws[:256].zero_()           # the status word
    return ws


# ------------------------------------------------------------------- sizes --
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        cells = case["rows"] * case["width"]
        read, written = cells * e * (2 if case["residual"] else 1), cells * e if case["residual"] else 0
        if case["out"] == "io":
            written += cells * e
        else:
            written += cells + 4 * case["rows"] * (-(-case["width"] // case["block"]) if case["block"] else 1)
        return {"bytes": read + written + 4 * case["width"] * case["weight"], "flops": 5 * cells}
    if case["op"] == "norm_gradient":
        cells = case["rows"] * case["width"]
        return {"bytes": cells * e * (4 if case["residual"] else 3) + 8 * case["width"] * case["weight"],
                "flops": 10 * cells}
    b, t, h, g, p, n = (case[k] for k in ("batch", "seqlen", "nheads", "ngroups", "headdim", "dstate"))
    tok, state = b * t, 4 * b * h * n * p
    read = tok * (2 * g * n + h * p) * e + 8 * tok * h
    step = 6 * n * p           # S^T k, the outer product and S^T q of one token
    if case["op"] == "step":
        return {"bytes": read + tok * h * p * e + 2 * state, "flops": tok * h * step}
    if case["op"] == "prefill":
        return {"bytes": read + tok * h * p * e + state * (2 if case["init"] else 1), "flops": tok * h * step}
    return {"bytes": read + tok * h * p * e + tok * (2 * g * n + h * p + 2 * h) * e, "flops": tok * h * 3 * step}


# ---------------------------------------------------------- the definition --
def exact(case, seed):
    x = {k: v if v.dtype == torch.int32 else v.double() for k, v in _inputs(case, seed).items()}
    if case["op"] == "norm":
        return _exact_norm(case, x)
    if case["op"] == "norm_gradient":
        return _exact_norm_gradient(case, x)
    b, t, h, p, n = (case[k] for k in ("batch", "seqlen", "nheads", "headdim", "dstate"))
    head = torch.arange(h, device="cuda") // (h // case["ngroups"])
    scale = 1.0 / math.sqrt(n)
    s = x["h0"].clone() if "h0" in x else torch.zeros(b, h, n, p, device="cuda", dtype=torch.float64)
    live = None
    if "lengths" in x:
        live = torch.arange(t, device="cuda")[None] < x["lengths"][:, None]
    y = torch.zeros(b, t, h, p, device="cuda", dtype=torch.float64)
    back = case["op"] == "gradient"
    states = [s] if back else None
    for i in range(t):
        k, q = x["k"][:, i][:, head], x["q"][:, i][:, head]
        old = s * x["g"][:, i].exp()[..., None, None]
        u = x["beta"][:, i, :, None] * (x["v"][:, i] - torch.einsum("bhnp,bhn->bhp", old, k))
        new = old + torch.einsum("bhn,bhp->bhnp", k, u)
        out = scale * torch.einsum("bhnp,bhn->bhp", new, q)
        if live is not None:
            m = live[:, i, None, None]
            new, out = torch.where(m[..., None], new, s), torch.where(m, out, 0.0)
        s = new
        y[:, i] = out
        if back:
            states.append(s)
    if not back:
        return {"y": y, "h": s}
    d = {k: torch.zeros_like(x[k]) for k in ("q", "k", "v", "g", "beta")}
    ds = torch.zeros_like(s)
    for i in reversed(range(t)):
        k, q, v, beta = x["k"][:, i][:, head], x["q"][:, i][:, head], x["v"][:, i], x["beta"][:, i, :, None]
        a, before, after = x["g"][:, i].exp()[..., None, None], states[i], states[i + 1]
        do = scale * x["dy"][:, i]
        if live is not None:
            do = do * live[:, i, None, None]
        here = ds + torch.einsum("bhn,bhp->bhnp", q, do)
        miss = v - torch.einsum("bhnp,bhn->bhp", a * before, k)
        du = torch.einsum("bhnp,bhn->bhp", here, k)
        dmiss = beta * du
        parts = {"q": torch.einsum("bhnp,bhp->bhn", after, do),
                 "k": torch.einsum("bhnp,bhp->bhn", here, beta * miss) - torch.einsum("bhnp,bhp->bhn", a * before, dmiss),
                 "v": dmiss, "beta": (du * miss).sum(-1)}
        into = here - torch.einsum("bhn,bhp->bhnp", k, dmiss)      # the gradient of the decayed state
        parts["g"] = (into * a * before).sum((-1, -2))
        prior = a * into
        if live is not None:
            m = live[:, i, None, None]
            parts = {n_: w * (m if w.dim() == 3 else m[..., 0]) for n_, w in parts.items()}
            prior = torch.where(m[..., None], prior, ds)
        ds = prior
        for n_ in ("v", "g", "beta"):
            d[n_][:, i] = parts[n_]
        for n_ in ("q", "k"):
            d[n_][:, i] = parts[n_].reshape(b, case["ngroups"], -1, n).sum(2)
        states.pop()
    return {"d" + k: v for k, v in d.items()}


def _exact_norm(case, x):
    s = x["x"] + x["r"] if case["residual"] else x["x"]
    y = s / torch.sqrt((s * s).sum(-1, keepdim=True) / case["width"] + EPS)
    if case["weight"]:
        y = y * x["w"]
    out = {"sum": s} if case["residual"] else {}
    if case["out"] == "io":
        return {**out, "y": y}
    step = case["block"] or case["width"]
    scale = torch.stack([c.abs().amax(-1).clamp(min=1e-30) / 448.0 for c in y.split(step, 1)], 1)
    wide = scale.repeat_interleave(step, 1)[:, :case["width"]]
    return {**out, "y8": (y / wide).to(torch.float8_e4m3fn).double(), "scale": scale}


def _exact_norm_gradient(case, x):
    s, dy, width = x["x"], x["dy"], case["width"]
    ms = (s * s).sum(-1, keepdim=True) / width + EPS
    up = dy * x["w"] if case["weight"] else dy
    # d/ds of s ms^(-1/2): ms^(-1/2) up - s ms^(-3/2) (up . s) / width
    dx = up / ms.sqrt() - s * (up * s).sum(-1, keepdim=True) / (width * ms * ms.sqrt())
    if case["residual"]:
        dx = dx + x["r"]
    return {"dx": dx, **({"dw": (dy * s / ms.sqrt()).sum(0)} if case["weight"] else {})}
