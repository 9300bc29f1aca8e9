"""The references of the convolution and the selective scan against differentiation and differences (CPU)."""
import pytest
import torch

import _mix_ref as ref


def _leaves(x, names):
    return {k: v.double().requires_grad_(k in names) for k, v in x.items()}


@pytest.mark.parametrize("silu", (True, False))
def test_conv_gradients(silu):
    lens, W = [0, 1, 9, 3], 4
    x = ref.conv_inputs(3, W, lens, 1, torch.float64)
    names = ("x", "weight", "bias", "s0")
    f = _leaves(x, names)

    def loss(f):
        ys, t0, total = [], 0, 0.0
        for i, n in enumerate(lens):
            seen = torch.cat([f["s0"][i], f["x"][t0:t0 + n]])
            p = f["bias"] + sum(seen[j:j + n] * f["weight"][:, j] for j in range(W))
            y = torch.nn.functional.silu(p) if silu else p
            total = total + (y * x["dy"][t0:t0 + n].double()).sum() + (seen[n:] * x["ds1"][i].double()).sum()
            ys.append(y)
            t0 += n
        return total, torch.cat(ys)

    total, y = loss(f)
    got = ref.conv_ref(x, lens, silu=silu, grads=True)
    for k, g in zip(names, torch.autograd.grad(total, [f[k] for k in names])):
        torch.testing.assert_close(got["d" + k], g, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(ref.conv_ref(x, lens, silu=silu)["y"], y.detach(), rtol=1e-12, atol=1e-12)
    # against a difference along a random direction: 1e-6 steps, errors of their square and of 1e-16 / 1e-6
    eps, way = 1e-6, {k: ref.rnd(*x[k].shape, seed=70 + i) for i, k in enumerate(names)}
    at = lambda s: loss({k: v.double() + (s * way[k] if k in way else 0) for k, v in x.items()})[0]  # noqa: E731
    diff = (at(eps) - at(-eps)) / (2 * eps)
    assert abs(diff - sum((got["d" + k] * way[k]).sum() for k in names)) < 1e-7 * (1 + abs(diff))


@pytest.mark.parametrize("softplus,z", ((True, True), (False, True), (True, False)))
def test_ssm_gradients(softplus, z):
    lens, C, N, G = [4, 0, 7], 4, 8, 2
    x = ref.ssm_inputs(C, N, G, lens, 3, torch.float64)
    if not softplus:
        x["dt"] = x["dt"].abs() * 0.1
        x["dt_bias"] = x["dt_bias"].abs() * 0.01
    names = ["u", "dt", "a", "b", "c", "d", "dt_bias", "s0"] + (["z"] if z else [])

    def loss(f):
        total, t0 = 0.0, 0
        for i, n in enumerate(lens):
            h = f["s0"][i]
            for t in range(t0, t0 + n):
                delta = f["dt"][t] + f["dt_bias"]
                delta = torch.nn.functional.softplus(delta) if softplus else delta
                B, Cm = (f[k][t].repeat_interleave(C // G, 0) for k in ("b", "c"))
                h = (delta[:, None] * f["a"]).exp() * h + (delta * f["u"][t])[:, None] * B
                y = (h * Cm).sum(1) + f["d"] * f["u"][t]
                y = y * torch.nn.functional.silu(f["z"][t]) if z else y
                total = total + (y * x["dy"][t].double()).sum()
            total = total + (h * x["ds1"][i].double()).sum()
            t0 += n
        return total

    f = _leaves(x, names)
    got = ref.ssm_ref(x, lens, z=z, softplus=softplus, grads=True)
    key = lambda k: {"dt_bias": "ddt_bias"}.get(k, "d" + k)  # noqa: E731
    for k, g in zip(names, torch.autograd.grad(loss(f), [f[k] for k in names])):
        torch.testing.assert_close(got[key(k)], g, rtol=1e-10, atol=1e-12)
    eps, way = 1e-6, {k: ref.rnd(*x[k].shape, seed=90 + i) for i, k in enumerate(names)}
    at = lambda s: loss({k: v.double() + (s * way[k] if k in way else 0) for k, v in x.items()})  # noqa: E731
    diff = (at(eps) - at(-eps)) / (2 * eps)
    assert abs(diff - sum((got[key(k)] * way[k]).sum() for k in names)) < 1e-6 * (1 + abs(diff))


def test_e4m3_list_is_torchs():
    mine = torch.tensor(ref.e4m3_values(), dtype=torch.float64)
    theirs = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(mine, theirs)


def test_run_slots_are_distinct():
    """Run c of sequence b has the slot (start_b >> log) + b + c: distinct, in order, below (n_tokens >> log) + n_seq; every
    sequence has at least one, empty ones too."""
    import random
    r = random.Random(9)
    for _ in range(300):
        log = r.choice([4, 5, 6, 9])
        R = 1 << log
        lens = [r.choice([0, 0, 1, R - 1, R, R + 1, r.randrange(4 * R)]) for _ in range(r.randrange(1, 12))]
        at, seen = r.randrange(2 * R), []
        for b, n in enumerate(lens):
            seen += [(at >> log) + b + c for c in range(max(1, (n + R - 1) // R))]
            at += n
        assert seen == sorted(set(seen)) and seen[-1] < ((at + r.randrange(3)) >> log) + len(lens)
