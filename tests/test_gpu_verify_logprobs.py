"""token_logprobs against the float64 oracle (needs an MI355X).

Bounds. z = ln 2 (M + log2 l): l sums n positive terms in float32, at most n / 256 + 64 of them one after
another in a lane and joins of a few dozen more, each term off by |t| 2^-24 + 2^-22 relative (t the exponent,
terms with large |t| being as much smaller); with M up to 1.45 max|x| rounded to 2^-24 of itself,
|error of z| <= 2^-24 (n / 64 + 128 + 4 max|x|).  The entropy's second sum has the same relative error.
"""
import numpy as np
import pytest
import torch

import verify_router_gemv_amd as v
from oracle import verify_oracle
from verify_helpers import DEV, close, gen, host, normal, say

pytestmark = pytest.mark.gpu
BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32


def check(x, tokens, top, what=""):
    T, V = x.shape
    say(f"case logprobs {what} T={T} V={V} top={top} {x.dtype}")
    r = v.token_logprobs(x, tokens, top)
    torch.cuda.synchronize()
    hx = host(x)
    ht = host(tokens) if tokens is not None else np.zeros((T, 0), np.int64)
    lp, h, ids, tlp = verify_oracle.token_logprobs(hx, ht, top)
    big = np.abs(np.where(np.isfinite(hx), hx, 0)).max(initial=0)
    tol = 2.0 ** -24 * (V / 64 + 128 + 4 * big)
    assert np.array_equal(host(r.top_ids), ids), f"{what}: ids"
    close(host(r.logprobs), lp, tol, f"{what} logprobs")
    close(host(r.top_logprobs), tlp, tol, f"{what} top_logprobs")
    close(host(r.entropy), h, tol * (2 + h), f"{what} entropy")


def rows(T, V, dtype, seed=0, pad=0, scale=3.0):
    g = gen(seed)
    x = normal(g, T, V + pad, dtype=dtype, scale=scale)
    return x[:, pad // 2:pad // 2 + V], g


@pytest.mark.parametrize("dtype", [BF, FH, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 63, 64, 65, 1000, 1023, 1024, 1031, 4096, 9999])
def test_vocabularies(dtype, V):
    for pad in (0, 2, 6):    # rows that start at any multiple of the element's size
        x, g = rows(3, V, dtype, V, pad)
        tokens = torch.randint(-1, V + 1, (3, 4), generator=g, device=DEV).int()
        check(x, tokens, min(V, 5), f"pad {pad}")


@pytest.mark.parametrize("top", [0, 1, 2, 15, 16])
@pytest.mark.parametrize("T,V", [(1, 50001), (2, 131072), (40, 20011), (300, 3001), (1100, 1500)])
def test_alternatives(top, T, V):
    x, g = rows(T, V, BF if V % 2 else F32, T + top)
    check(x, torch.randint(0, V, (T, 1), generator=g, device=DEV), top)


def test_token_types_and_counts():
    x, g = rows(9, 2000, F32)
    for N, dt in ((0, torch.int32), (1, torch.int64), (65, torch.int32), (200, torch.int64)):
        check(x, torch.randint(-5, 2005, (9, N), generator=g, device=DEV).to(dt), 3, f"{N} tokens {dt}")
    check(x, None, 2, "no tokens")
    check(x[:, :1], None, 1, "one logit")
    far = torch.tensor([[1 << 40, -(1 << 40), 1 << 32]] * 9, device=DEV)   # no token, not token 0 again
    check(x, far, 0, "ids past 32 bits")


def test_ties_go_to_the_lowest_id():
    for V, T in ((500, 3), (70000, 2), (5000, 600)):
        x = torch.zeros(T, V, dtype=BF, device=DEV)
        check(x, torch.zeros(T, 1, dtype=torch.int32, device=DEV), 16, "all equal")
        x[:, ::7] = 2
        x[:, V - 3:] = 5
        check(x, torch.zeros(T, 1, dtype=torch.int32, device=DEV), 16, "groups")
        x = (torch.arange(V, device=DEV) // 3).float().expand(T, V).contiguous()     # rising: the last are the best
        check(x, torch.full((T, 1), V - 1, dtype=torch.int32, device=DEV), 16, "rising")


def test_masked_logits():
    lo = float("-inf")
    for V, T in ((300, 4), (40000, 2), (2500, 1030)):
        x, g = rows(T, V, F32, 9)
        x = x.clone()
        x[0] = lo                                   # nothing left
        x[1, :] = lo
        x[1, V - 2] = 3.0                           # one left
        if T > 2:
            x[2, 5:] = lo                           # fewer than the alternatives asked for
            x[3, torch.rand(V, generator=g, device=DEV) < 0.9] = lo
        check(x, torch.randint(0, V, (T, 3), generator=g, device=DEV).int(), 8, "masked")
        x, _ = rows(T, V, BF, 10)
        x = x.clone()
        x[:, ::2] = torch.finfo(BF).min             # masked with the type's lowest value
        check(x, torch.randint(0, V, (T, 3), generator=g, device=DEV).int(), 8, "lowest value")


def test_nan_and_infinity():
    x, g = rows(4, 30000, F32, 11)
    x = x.clone()
    x[1, 100] = float("nan")
    x[2, 29999] = float("inf")
    tokens = torch.tensor([[5, 100, -1]] * 4, device=DEV)
    r = v.token_logprobs(x, tokens, 3)
    lp, h = host(r.logprobs), host(r.entropy)
    assert np.isnan(lp[1:3, :2]).all() and np.isnan(h[1:3]).all()
    assert (lp[:, 2] == -np.inf).all() and np.isfinite(lp[[0, 3]][:, :2]).all()
    assert 100 not in host(r.top_ids)[1] and host(r.top_ids)[2, 0] == 29999
    x[:] = float("nan")
    x[:, 7] = 1.0
    r = v.token_logprobs(x, None, 3)
    assert host(r.top_ids).tolist() == [[7, -1, -1]] * 4


def test_peaked_and_large_logits():
    x, g = rows(5, 10000, F32, 12, scale=0.5)
    x = x.clone()
    x[:, 77] = 60.0
    check(x, torch.full((5, 1), 77, dtype=torch.int32, device=DEV), 4, "peaked")
    check(x * 1000, torch.full((5, 1), 78, dtype=torch.int32, device=DEV), 4, "large")
    check(x + 30000, torch.full((5, 1), 78, dtype=torch.int32, device=DEV), 4, "shifted")


def test_row_distances():
    g = gen(13)
    big = normal(g, 6, 5000, dtype=BF)
    check(big[:, 17:1300], None, 4, "columns of a wider matrix")
    check(big[::2, :777], None, 4, "every other row")
    one = normal(g, 1, 600, dtype=FH)
    check(one.expand(4, 600).contiguous(), None, 2, "repeated")
    with pytest.raises(v.MoeRoundError):
        v.token_logprobs(one.expand(4, 600))
    with pytest.raises(ValueError, match="contiguous"):
        v.token_logprobs(big.t())


def test_refusals_and_empty():
    x, _ = rows(3, 10, F32)
    for kw in (dict(top=17), dict(top=11), dict(top=-1), dict(tokens=torch.zeros(2, 1, dtype=torch.int32, device=DEV)),
               dict(tokens=torch.zeros(3, 2, dtype=torch.int32, device=DEV).t().contiguous().t())):
        with pytest.raises(ValueError):
            v.token_logprobs(x, **kw)
    with pytest.raises(TypeError):
        v.token_logprobs(x, torch.zeros(3, 1, device=DEV))
    r = v.token_logprobs(x[:0], torch.zeros(0, 2, dtype=torch.int64, device=DEV), 3)
    assert r.logprobs.shape == (0, 2) and r.top_ids.shape == (0, 3) and r.entropy.shape == (0,)


def test_captured_and_on_other_streams():
    x, g = rows(3, 60001, BF, 14)
    x = x.clone()
    tokens = torch.randint(0, 60001, (3, 2), generator=g, device=DEV)
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        v.token_logprobs(x, tokens, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        r = v.token_logprobs(x, tokens, 4)
    for i in range(4):
        x.copy_(normal(gen(20 + i), 3, 60001, dtype=BF, scale=2.0))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            eager = v.token_logprobs(x, tokens, 4)
        torch.cuda.synchronize()
        for a, b in zip(r, eager):
            assert torch.equal(a, b)
