"""Float64 references of the causal convolution, the selective scan (with gradients) and the quantised rows (CPU, plain torch).

`size=True` runs the same sums over magnitudes: what a result's terms amount to before any of them cancel, which is what a float32
rounding error goes by.
"""
import torch

from _ops_ref import rnd


def starts(lens, lead=0):
    at = [lead]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32)


# ---------------------------------------------------------------- convolution

def conv_inputs(C, W, lens, seed, dtype, extra=0):
    T, n = sum(lens) + extra, len(lens)
    x = {"x": rnd(T, C, seed=seed), "dy": rnd(T, C, seed=seed + 1), "s0": rnd(n, W - 1, C, seed=seed + 2), "ds1": rnd(n, W - 1, C, seed=seed + 3)}
    x = {k: v.to(dtype) for k, v in x.items()}
    x["weight"], x["bias"] = (rnd(C, W, seed=seed + 4) / W ** 0.5).float(), (0.3 * rnd(C, seed=seed + 5)).float()
    return x


def conv_ref(x, lens, lead=0, silu=True, s0=True, bias=True, grads=False, ds1=True, size=False):
    """y and s1 (or dx, dweight, dbias and ds0), float64; rows outside the sequences are zero."""
    f = {k: v.double().abs() if size else v.double() for k, v in x.items()}
    T, C = f["x"].shape
    W = f["weight"].shape[1]
    b = f["bias"] if bias else torch.zeros(C, dtype=torch.float64)
    out = {"y": torch.zeros(T, C, dtype=torch.float64), "s1": torch.zeros_like(f["s0"]), "dx": torch.zeros(T, C, dtype=torch.float64),
           "dweight": torch.zeros(C, W, dtype=torch.float64), "dbias": torch.zeros(C, dtype=torch.float64), "ds0": torch.zeros_like(f["s0"])}
    t0 = lead
    for i, n in enumerate(lens):
        first = f["s0"][i] if s0 else torch.zeros_like(f["s0"][i])
        seen = torch.cat([first, f["x"][t0:t0 + n]])
        p = b + sum(seen[j:j + n] * f["weight"][:, j] for j in range(W))
        real = p
        if size and silu:          # the activation's derivative goes by the value itself
            g = {k: v.double() for k, v in x.items()}
            gs = torch.cat([g["s0"][i] if s0 else torch.zeros_like(g["s0"][i]), g["x"][t0:t0 + n]])
            real = (g["bias"] if bias else 0.0) + sum(gs[j:j + n] * g["weight"][:, j] for j in range(W))
        sg = real.sigmoid()
        out["y"][t0:t0 + n] = p * (sg if silu and not size else 1.0)
        out["s1"][i] = seen[n:]
        dp = f["dy"][t0:t0 + n]
        if silu:
            act = sg * (1 + real * (1 - sg))
            # of a magnitude: the derivative's own terms, and what an error of p changes in it (its second derivative is below 1)
            dp = dp * (act.abs() + sg * (1 + real.abs()) + p if size else act)
        ds = torch.zeros_like(seen)
        if ds1:
            ds[n:] += f["ds1"][i]
        for j in range(W):
            ds[j:j + n] += dp * f["weight"][:, j]
            out["dweight"][:, j] += (dp * seen[j:j + n]).sum(0)
        out["dbias"] += dp.sum(0)
        out["dx"][t0:t0 + n] = ds[W - 1:]
        out["ds0"][i] = ds[:W - 1]
        t0 += n
    return {k: out[k] for k in (("dx", "dweight", "dbias", "ds0") if grads else ("y", "s1"))}


# ---------------------------------------------------------------- selective scan

def ssm_inputs(C, N, G, lens, seed, dtype, extra=0, steps="usual"):
    T, n = sum(lens) + extra, len(lens)
    x = {"u": rnd(T, C, seed=seed), "dt": 0.5 * rnd(T, C, seed=seed + 1), "b": rnd(T, G, N, seed=seed + 2), "c": rnd(T, G, N, seed=seed + 3),
         "z": 2.0 * rnd(T, C, seed=seed + 4), "dy": rnd(T, C, seed=seed + 5)}
    if steps == "spread":                       # steps from 1e-6 to 20: decays that forget everything beside ones that forget nothing
        x["dt"] = 6.0 * rnd(T, C, seed=seed + 1)
    x = {k: v.to(dtype) for k, v in x.items()}
    x["a"] = -((1.0 + torch.arange(N).double()) * (1.0 + 0.1 * rnd(C, N, seed=seed + 6)).clamp(0.5, 2.0)).float()
    x["dt_bias"] = (rnd(C, seed=seed + 7) - 3.0).float()
    x["d"] = (1.0 + 0.3 * rnd(C, seed=seed + 8)).float()
    x["s0"], x["ds1"] = (0.5 * rnd(n, C, N, seed=seed + 9)).float(), (0.5 * rnd(n, C, N, seed=seed + 10)).float()
    return x


def ssm_ref(x, lens, lead=0, z=True, d=True, bias=True, softplus=True, s0=True, ds1=True, grads=False, size=False, rate=1.0):
    """y and s1 (or all gradients), float64, token by token; rows outside the sequences are zero.  `rate`: of the decays' exponents."""
    mag = (lambda t: t.abs()) if size else (lambda t: t)
    f = {k: v.double() for k, v in x.items()}
    T, C = f["u"].shape
    G, N = f["b"].shape[1:]
    a = f["a"]
    raw = f["dt"] + (f["dt_bias"] if bias else 0.0)
    delta = torch.where(raw > 40, raw, torch.log1p(raw.clamp(max=40).exp())) if softplus else raw
    slope = raw.sigmoid() if softplus else torch.ones_like(raw)
    decay = lambda t: (delta[t][:, None] * (rate * a)).exp()  # noqa: E731
    u, dt = mag(f["u"]), mag(delta)
    D = mag(f["d"]) if d else torch.zeros(C, dtype=torch.float64)
    b, c = (mag(f[k]).repeat_interleave(C // G, 1) for k in ("b", "c"))
    sg = f["z"].sigmoid()
    gate = mag(f["z"] * sg) if z else torch.ones_like(u)
    dgate = sg * (1 + f["z"] * (1 - sg))
    dgate = sg * (1 + f["z"].abs() * (1 - sg)) if size else dgate
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    p, s1, kept = zero(T, C), zero(len(lens), C, N), []
    dp = mag(f["dy"]) * gate
    out = {"du": zero(T, C), "ddt": zero(T, C), "da": zero(C, N), "db": zero(T, G, N), "dc": zero(T, G, N), "dd": zero(C), "ddt_bias": zero(C),
           "ds0": zero(len(lens), C, N)}
    t0 = lead
    for i, n in enumerate(lens):
        h = mag(f["s0"][i]) if s0 else zero(C, N)
        kept = [h]
        for t in range(t0, t0 + n):
            h = decay(t) * h + (dt[t] * u[t])[:, None] * b[t]
            p[t] = (h * c[t]).sum(1) + D * u[t]
            kept.append(h)
        s1[i] = h
        if grads:
            g = mag(f["ds1"][i]) if ds1 else zero(C, N)
            for t in range(t0 + n - 1, t0 - 1, -1):
                h, before, e = kept.pop(), kept[-1], decay(t)
                g = g + dp[t][:, None] * c[t]
                out["dc"][t] = (dp[t][:, None] * h).view(G, C // G, N).sum(1)
                out["db"][t] = (g * (dt[t] * u[t])[:, None]).view(G, C // G, N).sum(1)
                gb = (g * b[t]).sum(1)
                out["du"][t] = dt[t] * gb + D * dp[t]
                out["ddt"][t] = ((mag(a) * g * e * before).sum(1) + u[t] * gb) * slope[t]
                out["da"] += g * e * before * dt[t][:, None]
                g = g * e
            out["ds0"][i] = g
            out["dd"] += (dp[t0:t0 + n] * u[t0:t0 + n]).sum(0)
            out["ddt_bias"] += out["ddt"][t0:t0 + n].sum(0)
        t0 += n
    if not grads:
        return {"y": p * gate, "s1": s1}
    out["dz"] = mag(f["dy"]) * p * dgate
    out["dz"][:lead] = 0
    out["dz"][t0:] = 0
    return out


# ---------------------------------------------------------------- quantised rows

TOP = {0: 127, 1: 7, 2: 448}


def e4m3_values():
    """The non-negative finite values in order: 0, 2^-9 .. 7 x 2^-9, then 1.xxx x 2^(e - 7)."""
    return [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8) if (e, m) != (15, 7)]


def cache_ref(x, group, fmt):
    """Scales (float32) and codes as the numbers they stand for, by a search of the format's list in exact rational arithmetic."""
    from bisect import bisect_left
    from fractions import Fraction
    values = [Fraction(v) for v in (e4m3_values() if fmt == 2 else range(TOP[fmt] + 1))]
    x = x.float()
    R, d = x.shape
    amax = x.unflatten(1, (-1, group)).abs().amax(-1)
    scales = (amax.double() / TOP[fmt]).float()             # a double's rounding to float32 of a quotient of float32 numbers is exact
    codes = torch.zeros(R, d, dtype=torch.float64)
    for r in range(R):
        for j in range(d):
            s = Fraction(float(scales[r, j // group]))
            if s == 0:
                continue
            q = abs(Fraction(float(x[r, j]))) / s
            i = min(bisect_left(values, q), len(values) - 1)
            best = min((max(i - 1, 0), i), key=lambda i: (abs(values[i] - q), i % 2))
            codes[r, j] = float(values[best]) * (-1.0 if x[r, j] < 0 else 1.0)
    return scales, codes
