"""Cases of the gated delta scan (forward, backward) and of the norms around it, with their plain forms.

A case is a call as a program makes it: a prompt (or several, packed) brought into the recurrent states,
a training step's gradients of the same, and the norms before and after the recurrence at the sizes of
decoding and of training.  ``own`` selects the library's kernels; otherwise the plain torch forms run.
"""
import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # continuing many requests by a few tokens each (checking drafted tokens): latency counts
        _scan("scan gdn few tokens", "scan", "gdn", "bfloat16", 32, 16, 128, 128, 64, 250, 1),
        # one user's short prompt
        _scan("scan gdn one prompt", "scan", "gdn", "bfloat16", 32, 32, 128, 128, 1, 777, 0),
        # a prefill batch of ragged prompts, q and k heads shared by two value heads
        _scan("scan gdn prefill", "scan", "gdn", "bfloat16", 32, 16, 128, 128, 7, 12301, 1),
        # a prefill batch with a gate per key row
        _scan("scan kda prefill", "scan", "kda", "bfloat16", 32, 32, 128, 128, 5, 6150, 1),
        # the wide state, float32 as the decode step takes it
        _scan("scan kda wide float32", "scan", "kda", "float32", 32, 32, 128, 256, 3, 1900, 1),
        # a training step's gradients, ragged documents
        _scan("scan bwd gdn", "scan_bwd", "gdn", "bfloat16", 32, 16, 128, 128, 4, 8190, 0),
        _scan("scan bwd kda", "scan_bwd", "kda", "bfloat16", 32, 32, 128, 128, 3, 3001, 0),
        # the small state shape in float32 (gradient checks, calibration)
        _scan("scan bwd small float32", "scan_bwd", "gdn", "float32", 8, 8, 64, 64, 2, 515, 1),
        # one decoded token of each request: residual add and norm before the block
        _norm("norm in decode", "norm_in", "bfloat16", "bfloat16", 64, 1, 4096, True, "rms"),
        # unit-norm q rows of a training batch, gradients
        _norm("norm in bwd heads", "norm_in_bwd", "bfloat16", "bfloat16", 8192, 32, 128, False, "l2"),
        # the readout's gated norm while decoding: float32 readout, bfloat16 gate
        _norm("norm out decode", "norm_out", "float32", "bfloat16", 256, 32, 128, False, "rms"),
        # the gated norm's gradients over a training batch
        _norm("norm out bwd", "norm_out_bwd", "bfloat16", "bfloat16", 8192, 32, 128, False, "rms"),
    ]


def _scan(name, op, form, dtype, heads, heads_k, dk, dv, n_seq, tokens, states):
    c = {"op": op, "form": form, "dtype": dtype, "heads": heads, "heads_k": heads_k, "dk": dk, "dv": dv,
         "n_seq": n_seq, "tokens": tokens, "states": states}
    return dict(c, name=name) if name else c


def _norm(name, op, dtype, dtype_out, outer, inner, d, residual, kind):
    c = {"op": op, "dtype": dtype, "dtype_out": dtype_out, "outer": outer, "inner": inner, "d": d,
         "residual": residual, "kind": kind}
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "norm_in", "norm_in_bwd", "norm_out", "norm_out_bwd"])
    if op.startswith("scan"):
        form = rng.choice(["gdn", "kda"])
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (128, 256)])
        heads = rng.choice([4, 8, 16, 32])
        heads_k = heads // rng.choice([1, 1, 2])
        n_seq = _log(rng, 1, 64)
        most = (12000 if form == "gdn" else 6000) if op == "scan" else (8000 if form == "gdn" else 3000)
        most = most * 128 // dv if dtype != "float32" else most * 128 // dv // 2
        tokens = max(n_seq, _log(rng, 40, most))
        return _scan(None, op, form, dtype, heads, heads_k, dk, dv, n_seq, tokens, rng.choice([0, 1]))
    dtype = rng.choice(["bfloat16", "float16", "float32"])
    dtype_out = rng.choice([dtype, "bfloat16", "float32"])
    d = rng.choice([16, 64, 128, 256, _log(rng, 20, 8192), 8 * _log(rng, 64, 1024)])
    rows = _log(rng, 1, min(262144, 33554432 // d))
    inner = rng.choice([1, 4, 32]) if d <= 256 else 1
    residual = rng.choice([True, False])
    kind = rng.choice(["rms", "l2"]) if op.startswith("norm_in") else "rms"
    return _norm(None, op, dtype, dtype_out, max(1, rows // inner), inner, d, residual, kind)


def _lengths(c):
    """Ragged lengths that sum to the case's tokens, each at least one (the same for every seed)."""
    r = random.Random(c["tokens"] * 1009 + c["n_seq"])
    n, total = c["n_seq"], c["tokens"]
    w = [r.uniform(0.5, 2.0) for _ in range(n)]
    lens = [1 + int((total - n) * x / sum(w)) for x in w]
    lens[r.randrange(n)] += total - sum(lens)
    return lens


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return _prepare_scan(case, rn) if case["op"].startswith("scan") else _prepare_norm(case, rn)


def _prepare_scan(c, rn):
    dt = DTYPES[c["dtype"]]
    T, H, Hk, dk, dv, n = (c[x] for x in ("tokens", "heads", "heads_k", "dk", "dv", "n_seq"))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    s = {"case": c, "lens": _lengths(c), "q": unit(rn(T, Hk, dk)).to(dt), "k": unit(rn(T, Hk, dk)).to(dt), "v": rn(T, H, dv).to(dt)}
    # gates as the workloads draw them, with a spread from token to token
    if c["form"] == "gdn":
        s["gate"] = torch.sigmoid(4.0 + rn(H) + 0.5 * rn(T, H))
    else:
        s["gate"] = torch.sigmoid(3.0 + 1.5 * rn(H, dk) + 0.5 * rn(T, H, dk))
    s["beta"] = torch.sigmoid(rn(T, H))
    s["s0"] = rn(n, H, dk, dv) * 0.3 if c["states"] else None
    at = [0]
    for x in s["lens"]:
        at.append(at[-1] + x)
    s["seq_start"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    if c["op"] == "scan":
        s["y"], s["s1"] = torch.empty_like(s["v"]), torch.empty(n, H, dk, dv, device="cuda")
    else:
        s["dy"] = rn(T, H, dv).to(dt)
        s["ds1"] = rn(n, H, dk, dv) * 0.3 if c["states"] else None
        for x in ("q", "k", "v", "gate", "beta"):
            s["d" + x] = torch.empty_like(s[x])
        s["ds0"] = torch.empty(n, H, dk, dv, device="cuda")
    if own:
        import quantized_delta_rule_02_amd as sq
        s["form"] = sq.SQ_FORM_GDN if c["form"] == "gdn" else sq.SQ_FORM_KDA
        nbytes = sq.sq_delta_scan_bytes(s["form"], dt, H, Hk, dk, dv, n, T, backward=c["op"] == "scan_bwd")
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_norm(c, rn):
    dt, do = DTYPES[c["dtype"]], DTYPES[c["dtype_out"]]
    shape = (c["outer"], c["inner"], c["d"])
    d = c["d"]
    s = {"case": c, "kind": c["kind"], "eps": 1e-6, "weight": 1.0 + 0.1 * rn(d), "res_scale": 0.7}
    s["chan_scale"] = 1.0 + 0.1 * rn(d) if c["residual"] else None
    out = torch.empty(shape, dtype=do, device="cuda")
    if c["op"] == "norm_in":
        s["x"] = rn(*shape).to(dt)
        s["r"] = rn(*shape).to(dt) if c["residual"] else None
        s["h"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["n"] = out
    elif c["op"] == "norm_in_bwd":
        s["h"], s["dn"] = rn(*shape).to(dt), rn(*shape).to(do)
        s["r"] = rn(*shape).to(dt) if c["residual"] else None
        s["dh"] = rn(*shape).to(dt) if c["residual"] else None
        s["dr"] = torch.empty_like(s["h"]) if c["residual"] else None
        s["dx"] = torch.empty_like(s["h"])
    else:
        s["y"], s["z"] = rn(*shape).to(dt), rn(*shape).to(do)
        if c["op"] == "norm_out":
            s["x"] = rn(*shape).to(do) if c["residual"] else None
            s["o"] = out
        else:
            s["do"], s["dy"], s["dz"] = rn(*shape).to(do), torch.empty_like(s["y"]), torch.empty_like(s["z"])
    if c["op"].endswith("bwd"):
        s["dweight"] = torch.empty(d, device="cuda")
        s["dchan_scale"] = torch.empty(d, device="cuda") if c["residual"] else None
        if own:
            import quantized_delta_rule_02_amd as sq
            s["workspace"] = torch.empty(sq.sq_norm_bytes(c["outer"] * c["inner"], d), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import quantized_delta_rule_02_amd as sq
    op = s["case"]["op"]
    if op == "scan":
        sq.sq_delta_scan(s["form"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["y"], seq_start=s["seq_start"],
                         s0=s["s0"], s1=s["s1"], workspace=s["workspace"])
        return {"y": s["y"], "s1": s["s1"]}
    if op == "scan_bwd":
        sq.sq_delta_scan_bwd(s["form"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["dy"], s["dq"], s["dk"], s["dv"],
                             s["dgate"], s["dbeta"], seq_start=s["seq_start"], s0=s["s0"], ds1=s["ds1"], ds0=s["ds0"],
                             workspace=s["workspace"])
        return {x: s[x] for x in ("dq", "dk", "dv", "dgate", "dbeta", "ds0")}
    kind = sq.SQ_NORM_RMS if s["kind"] == "rms" else sq.SQ_NORM_L2
    if op == "norm_in":
        sq.sq_norm_in(s["x"], s["n"], weight=s["weight"], r=s["r"], h=s["h"], chan_scale=s["chan_scale"],
                      res_scale=s["res_scale"], kind=kind, eps=s["eps"])
        return {"n": s["n"], "h": s["h"]}
    if op == "norm_in_bwd":
        sq.sq_norm_in_bwd(s["h"], s["dn"], s["dx"], weight=s["weight"], r=s["r"], dh=s["dh"], dr=s["dr"],
                          chan_scale=s["chan_scale"], res_scale=s["res_scale"], dweight=s["dweight"],
                          dchan_scale=s["dchan_scale"], kind=kind, eps=s["eps"], workspace=s["workspace"])
        return {x: s[x] for x in ("dx", "dr", "dweight", "dchan_scale")}
    if op == "norm_out":
        sq.sq_norm_out(s["y"], s["o"], weight=s["weight"], z=s["z"], act=sq.SQ_ACT_SILU, x=s["x"],
                       chan_scale=s["chan_scale"], res_scale=s["res_scale"], eps=s["eps"])
        return {"o": s["o"]}
    sq.sq_norm_out_bwd(s["y"], s["do"], s["dy"], weight=s["weight"], z=s["z"], dz=s["dz"], act=sq.SQ_ACT_SILU,
                       chan_scale=s["chan_scale"], res_scale=s["res_scale"], dweight=s["dweight"],
                       dchan_scale=s["dchan_scale"], eps=s["eps"], workspace=s["workspace"])
    return {x: s[x] for x in ("dy", "dz", "dweight", "dchan_scale")}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "scan":
        y, s1 = _plain_scan(s, s["q"].float(), s["k"].float(), s["v"].float(), s["gate"], s["beta"], s["s0"])
        return {"y": y.to(s["v"].dtype), "s1": s1}
    if op == "scan_bwd":
        names = ("q", "k", "v", "gate", "beta", "s0")
        s0 = s["s0"] if s["s0"] is not None else torch.zeros_like(s["ds0"])
        leaf = [t.float().detach().requires_grad_() for t in (s["q"], s["k"], s["v"], s["gate"], s["beta"], s0)]
        y, s1 = _plain_scan(s, *leaf)
        outs, grads = [y], [s["dy"].float()]
        if s["ds1"] is not None:
            outs, grads = outs + [s1], grads + [s["ds1"]]
        got = torch.autograd.grad(outs, leaf, grads)
        return {"d" + x: t if x == "s0" else t.to(s[x].dtype) for x, t in zip(names, got)}
    return _plain_norm(s, torch.float32)


def _plain_scan(s, q, k, v, gate, beta, s0):
    """The recurrence in chunks: within a chunk the updates u = beta e solve (I + A beta) e = V - (gamma K) S.

    The chunks follow one another (a loop: each starts from the last one's state); all sequences and heads
    go through a chunk together.  Decays are exponentials of differences of cumulative logarithms, in 64 bits.
    """
    c = s["case"]
    gdn = c["form"] == "gdn"
    H, Hk, dk, dv, n = (c[x] for x in ("heads", "heads_k", "dk", "dv", "n_seq"))
    C = 32 if gdn else 16
    lens = torch.tensor(s["lens"], device=q.device)
    nc = (max(s["lens"]) + C - 1) // C
    t = torch.arange(nc * C, device=q.device)
    live = t[None] < lens[:, None]
    at = (s["seq_start"][:-1, None].long() + t[None]).clamp(max=q.shape[0] - 1)

    def chunks(x, fill):     # [T, H', ...] -> [n, nc, H', C, ...], rows past a sequence's end hold `fill`
        x = torch.where(live.view(n, nc * C, *[1] * (x.dim() - 1)), x[at], torch.as_tensor(fill, dtype=x.dtype, device=x.device))
        return x.unflatten(1, (nc, C)).transpose(2, 3)

    rep = lambda x: x.repeat_interleave(H // Hk, dim=2)  # noqa: E731
    q, k = rep(chunks(q, 0.0)), rep(chunks(k, 0.0))
    v, beta = chunks(v, 0.0), chunks(beta, 0.0)[..., None]
    L = chunks(gate, 1.0).double().log().cumsum(3)                  # [n, nc, H, C(, dk)]
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    if gdn:
        decay = (L[..., :, None] - L[..., None, :]).masked_fill(~low, -math.inf).exp().float()
        A, P = (k @ k.transpose(-1, -2)) * decay, (q @ k.transpose(-1, -2)) * decay
        L = L[..., None]
    else:
        decay = (L[..., :, None, :] - L[..., None, :, :]).masked_fill(~low[..., None], -math.inf).exp().float()
        A, P = ((x[..., :, None, :] * k[..., None, :, :] * decay).sum(-1) for x in (k, q))
        del decay
    gamma, rest = L.exp().float(), (L[..., -1:, :] - L).exp().float()
    N = (A * beta.transpose(-1, -2)).tril(-1)
    inv = torch.eye(C, device=q.device) - N                        # (I + N)^-1 = (I - N)(I + N^2)(I + N^4)...
    power = 2
    while power < C:
        N = N @ N
        inv = inv + inv @ N
        power *= 2
    Kg, Qg, Kr = k * gamma, q * gamma, (k * rest).transpose(-1, -2)
    last = gamma[..., -1, :, None]                                  # [n, nc, H, 1 or dk, 1]
    S = s0 if s0 is not None else torch.zeros(n, H, dk, dv, device=q.device)
    ys = []
    for i in range(nc):
        u = beta[:, i] * (inv[:, i] @ (v[:, i] - Kg[:, i] @ S))
        ys.append(Qg[:, i] @ S + P[:, i] @ u)
        S = last[:, i] * S + Kr[:, i] @ u
    y = torch.stack(ys, 1).transpose(2, 3).reshape(n, nc * C, H, dv)
    return y[live], S


def _plain_norm(s, ft):
    """Both norms and their gradients (the usual derivative of x / sqrt(mean x^2 + eps)), in `ft`."""
    op, eps, d = s["case"]["op"], s["eps"], s["case"]["d"]
    f = lambda x: None if x is None else x.to(ft)  # noqa: E731
    w, cs, rs = f(s["weight"]), f(s["chan_scale"]), s["res_scale"]
    scale = rs * cs if cs is not None else torch.full((d,), rs, dtype=ft, device=w.device)
    div = d if s["kind"] == "rms" else 1

    def inverse(x):
        return 1.0 / (x.square().sum(-1, keepdim=True) / div + eps).sqrt()

    def back(x, dhat):       # gradient of x * inverse(x)
        i = inverse(x)
        return i * (dhat - x * i * i * (dhat * x).sum(-1, keepdim=True) / div)

    to = (lambda x, like: x.to(like.dtype)) if ft == torch.float32 else (lambda x, like: x)
    if op == "norm_in":
        h = f(s["x"]) + scale * f(s["r"]) if s["r"] is not None else f(s["x"])
        return {"n": to(h * inverse(h) * w, s["n"]), "h": to(h, s["x"]) if s["r"] is not None else None}
    if op == "norm_in_bwd":
        h, dn = f(s["h"]), f(s["dn"])
        dx = back(h, dn * w)
        dw = (dn * h * inverse(h)).double().sum((0, 1)).to(ft)
        if s["r"] is None:
            return {"dx": to(dx, s["dx"]), "dr": None, "dweight": dw, "dchan_scale": None}
        dx = dx + f(s["dh"])
        dcs = (rs * dx * f(s["r"])).double().sum((0, 1)).to(ft)
        return {"dx": to(dx, s["dx"]), "dr": to(scale * dx, s["dr"]), "dweight": dw, "dchan_scale": dcs}
    y, z = f(s["y"]), f(s["z"])
    sig = 1.0 / (1.0 + (-z).exp())
    yh = y * inverse(y)
    if op == "norm_out":
        o = scale * w * yh * z * sig
        return {"o": to(o + f(s["x"]) if s["x"] is not None else o, s["o"])}
    do = f(s["do"])
    dact = do * scale * w * yh
    dcs = (rs * do * w * yh * z * sig).double().sum((0, 1)).to(ft) if cs is not None else None
    return {"dy": to(back(y, do * scale * w * z * sig), s["dy"]), "dz": to(dact * sig * (1 + z * (1 - sig)), s["dz"]),
            "dweight": (do * scale * yh * z * sig).double().sum((0, 1)).to(ft), "dchan_scale": dcs}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_scan(s) if case["op"].startswith("scan") else _exact_norm(s)


def _exact_scan(s):
    """Token by token, one sequence after another, from the recurrence and its derivative."""
    c = s["case"]
    grp = c["heads"] // c["heads_k"]
    dbl = lambda x: x.double()  # noqa: E731
    q, k = dbl(s["q"]).repeat_interleave(grp, 1), dbl(s["k"]).repeat_interleave(grp, 1)
    v, beta = dbl(s["v"]), dbl(s["beta"])[..., None]
    a = dbl(s["gate"]).unsqueeze(-1)
    a = a.unsqueeze(-1) if a.dim() == 3 else a                     # [T, H, dk or 1, 1]
    H, dk, dv, n = c["heads"], c["dk"], c["dv"], c["n_seq"]
    bwd = c["op"] == "scan_bwd"
    y = torch.zeros_like(v)
    S1 = torch.zeros(n, H, dk, dv, dtype=torch.float64, device=v.device)
    dq, dk_, dv_, da, db = (torch.zeros_like(x) for x in (q, k, v, a, beta))
    ds0 = torch.zeros_like(S1)
    col, row = (lambda x: x[:, :, None]), (lambda x: x[:, None, :])
    t0 = 0
    for b, ln in enumerate(s["lens"]):
        S = dbl(s["s0"][b]) if s["s0"] is not None else torch.zeros_like(S1[0])
        kept = []
        for t in range(t0, t0 + ln):
            if bwd:
                kept.append(S)
            S = a[t] * S
            e = v[t] - (col(k[t]) * S).sum(1)
            S = S + col(k[t]) * row(beta[t] * e)
            if not bwd:
                y[t] = (col(q[t]) * S).sum(1)
        S1[b] = S
        if bwd:
            dy = dbl(s["dy"][t0:t0 + ln])
            G = dbl(s["ds1"][b]) if s["ds1"] is not None else torch.zeros_like(S)
            for i in range(ln - 1, -1, -1):
                t, before = t0 + i, kept.pop()
                Sd = a[t] * before
                e = v[t] - (col(k[t]) * Sd).sum(1)
                u = beta[t] * e
                G = G + col(q[t]) * row(dy[i])
                dq[t] = ((Sd + col(k[t]) * row(u)) * row(dy[i])).sum(2)
                du = (col(k[t]) * G).sum(1)
                dv_[t] = beta[t] * du
                db[t] = (du * e).sum(1, keepdim=True)
                dk_[t] = (G * row(u) - Sd * row(dv_[t])).sum(2)
                G = G - col(k[t]) * row(dv_[t])
                full = (G * before).sum(2, keepdim=True)
                da[t] = full if a.shape[2] > 1 else full.sum(1, keepdim=True)
                G = a[t] * G
            ds0[b] = G
        t0 += ln
    if not bwd:
        return {"y": y, "s1": S1}
    pair = lambda x: x.unflatten(1, (c["heads_k"], grp)).sum(2)  # noqa: E731
    return {"dq": pair(dq), "dk": pair(dk_), "dv": dv_, "dgate": da.reshape(s["gate"].shape),
            "dbeta": db.reshape(s["beta"].shape), "ds0": ds0}


def _exact_norm(s):
    """The definitions in 64 bits; the gradients by differentiating them."""
    op = s["case"]["op"]
    got = {n: x.double().requires_grad_() for n, x in s.items() if isinstance(x, torch.Tensor) and x.is_floating_point()}
    w, cs = got["weight"], got.get("chan_scale")
    scale = s["res_scale"] * cs if cs is not None else s["res_scale"]

    def hat(x):
        sq = (x * x).mean(-1, keepdim=True) if s["kind"] == "rms" else (x * x).sum(-1, keepdim=True)
        return x / torch.sqrt(sq + s["eps"])

    grad = lambda o, names, do: dict(zip(names, torch.autograd.grad(o, [got[n] for n in names], do)))  # noqa: E731
    if op == "norm_in":
        with torch.no_grad():
            h = got["x"] + scale * got["r"] if s["r"] is not None else got["x"]
            return {"n": hat(h) * w, "h": h if s["r"] is not None else None}
    if op == "norm_in_bwd":
        g = grad(hat(got["h"]) * w, ["h", "weight"], got["dn"].detach())
        if s["r"] is None:
            return {"dx": g["h"], "dr": None, "dweight": g["weight"], "dchan_scale": None}
        dx = (g["h"] + got["dh"]).detach()
        more = grad(scale * got["r"], ["r", "chan_scale"], dx)
        return {"dx": dx, "dr": more["r"], "dweight": g["weight"], "dchan_scale": more["chan_scale"]}
    block = scale * (hat(got["y"]) * w * torch.nn.functional.silu(got["z"]))
    if op == "norm_out":
        return {"o": (block + got["x"] if s["x"] is not None else block).detach()}
    g = grad(block, ["y", "z", "weight"] + (["chan_scale"] if cs is not None else []), got["do"].detach())
    return {"dy": g["y"], "dz": g["z"], "dweight": g["weight"], "dchan_scale": g.get("chan_scale")}


# ---------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"].startswith("scan"):
        b = torch.finfo(DTYPES[c["dtype"]]).bits // 8
        T, H, Hk, dk, dv = (c[x] for x in ("tokens", "heads", "heads_k", "dk", "dv"))
        qk, vv, state = 2 * T * Hk * dk * b, T * H * dv * b, 4 * c["n_seq"] * H * dk * dv
        gates = 4 * T * H * (1 + (dk if c["form"] == "kda" else 1))
        if c["op"] == "scan":    # q k v gate beta and the states in, y and the states out
            return {"bytes": qk + 2 * vv + gates + state * (1 + c["states"]), "flops": 6 * T * H * dk * dv}
        return {"bytes": 2 * qk + 3 * vv + 2 * gates + state * (1 + 2 * c["states"]), "flops": 18 * T * H * dk * dv}
    bi, bo = (torch.finfo(DTYPES[c[x]]).bits // 8 for x in ("dtype", "dtype_out"))
    n, r = c["outer"] * c["inner"] * c["d"], c["residual"]
    per = {"norm_in": bi + bo + 2 * bi * r, "norm_in_bwd": 2 * bi + bo + 3 * bi * r,
           "norm_out": bi + 2 * bo + bo * r, "norm_out_bwd": 2 * bi + 3 * bo}[c["op"]]
    return {"bytes": n * per + 4 * c["d"], "flops": 10 * n}
