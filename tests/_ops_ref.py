"""Float64 references of the gated delta scan and its gradients, token by token (CPU, plain torch)."""
import torch


def rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def scan_inputs(form, H, Hk, dk, dv, lens, seed, dtype, gate="usual"):
    """Inputs on the CPU; q, k, v, dy hold values of `dtype`.  `gate`: how strong the decay is."""
    T, n = sum(lens), len(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(rnd(T, Hk, dk, seed=seed)), "k": unit(rnd(T, Hk, dk, seed=seed + 1)), "v": rnd(T, H, dv, seed=seed + 2),
         "dy": rnd(T, H, dv, seed=seed + 3)}
    x = {n_: t.to(dtype) for n_, t in x.items()}
    gs = (T, H, dk) if form == 1 else (T, H)
    g = rnd(*gs, seed=seed + 4)
    if gate == "usual":
        a = torch.sigmoid(3.0 + 1.5 * g)
    elif gate == "one":
        a = torch.ones(gs, dtype=torch.float64)
    elif gate == "strong":                      # from 1 down to 1e-12, so that products of a chunk leave float32's range
        a = 10.0 ** (-6.0 * g.abs()).clamp(min=-12.0)
    elif gate == "resets":                      # mostly weak decay, now and then everything is forgotten
        a = torch.where(g > 1.2, torch.full(gs, 1e-9, dtype=torch.float64), torch.sigmoid(4.0 + g))
    x["gate"] = a.float()
    x["beta"] = torch.sigmoid(rnd(T, H, seed=seed + 5)).float()
    x["s0"] = (0.3 * rnd(n, H, dk, dv, seed=seed + 6)).float()
    x["ds1"] = (0.3 * rnd(n, H, dk, dv, seed=seed + 7)).float()
    return x


def _wide(x, grp):
    f = {n: t.double() for n, t in x.items()}
    f["q"], f["k"] = f["q"].repeat_interleave(grp, 1), f["k"].repeat_interleave(grp, 1)
    f["beta"] = f["beta"][..., None]
    f["gate"] = f["gate"].reshape(*f["gate"].shape[:2], -1, 1)
    return f


def scan_ref(x, lens, s0=True):
    """y [T, H, dv] and the final states, float64."""
    H, dv = x["v"].shape[1:]
    f = _wide(x, H // x["q"].shape[1])
    y, S1, t0 = torch.zeros_like(f["v"]), torch.zeros_like(f["s0"]), 0
    for b, n in enumerate(lens):
        S = f["s0"][b].clone() if s0 else torch.zeros_like(f["s0"][b])
        for t in range(t0, t0 + n):
            S = f["gate"][t] * S
            u = f["beta"][t] * (f["v"][t] - (f["k"][t][..., None] * S).sum(1))
            S = S + f["k"][t][..., None] * u[:, None]
            y[t] = (f["q"][t][..., None] * S).sum(1)
        S1[b] = S
        t0 += n
    return y, S1


def scan_grad_ref(x, lens, s0=True, ds1=True):
    """Gradients by differentiating scan_ref."""
    names = ("q", "k", "v", "gate", "beta", "s0")
    leaf = {n: x[n].double().requires_grad_() for n in names}
    y, S1 = scan_ref_diff(leaf, lens, s0)
    loss = (y * x["dy"].double()).sum()
    if ds1:
        loss = loss + (S1 * x["ds1"].double()).sum()
    got = torch.autograd.grad(loss, [leaf[n] for n in names], allow_unused=True)
    return {"d" + n: torch.zeros_like(leaf[n]) if g is None else g for n, g in zip(names, got)}


def scan_ref_diff(x, lens, s0=True):
    H = x["v"].shape[1]
    f = _wide(x, H // x["q"].shape[1])
    ys, Ss, t0 = [], [], 0
    for b, n in enumerate(lens):
        S = f["s0"][b] if s0 else torch.zeros_like(f["s0"][b])
        for t in range(t0, t0 + n):
            S = f["gate"][t] * S
            u = f["beta"][t] * (f["v"][t] - (f["k"][t][..., None] * S).sum(1))
            S = S + f["k"][t][..., None] * u[:, None]
            ys.append((f["q"][t][..., None] * S).sum(1))
        Ss.append(S)
        t0 += n
    return torch.stack(ys) if ys else torch.zeros(0, *x["v"].shape[1:], dtype=torch.float64), torch.stack(Ss)
