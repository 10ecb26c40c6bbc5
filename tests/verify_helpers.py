"""Shared helpers of the verify-round operators' GPU tests: inputs, host views, error bounds."""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda"
# Half a step of each type, relative to the value: the most one rounding changes it.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def host(t):
    """A tensor's values as float64 (or integers) on the host."""
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def random_parents(rng, rows, total):
    """A random tree per request (packed), -1 behind the last row."""
    out = np.full(total, -1, np.int32)
    t = 0
    for r in rows:
        for i in range(r):
            if t < total:
                out[t] = rng.integers(-1, i) if i else -1
            t += 1
    return out


def close(got, ref, tol, what):
    """Elementwise |got - ref| <= tol; a NaN or infinity must be the same on both sides."""
    got, ref, tol = np.asarray(got, np.float64), np.asarray(ref, np.float64), np.broadcast_to(tol, np.shape(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    inf = ~fine & ~np.isnan(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities"
    d = np.abs(got[fine] - ref[fine])
    bad = d > tol[fine]
    if bad.any():
        i = int(np.argmax(d - tol[fine]))
        at = tuple(int(k[i]) for k in np.nonzero(fine))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, worst at {at}: {got[at]!r} for {ref[at]!r}, "
                             f"bound {float(tol[at]):.3g}")
