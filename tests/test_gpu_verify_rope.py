"""qk_norm_rope against the float64 oracle (needs an MI355X).

Bound: one rounding to the cache's type, HALF relative, on top of the float32 arithmetic: the norm sums at
most 256 squares (relative error under 2^-19 in any order), and a rotation adds two products of a value and
a sine or cosine good to 2^-21 of 1; so |error| <= HALF |y| + 2^-18 (|a| + |b|) with a, b the pair.  Below
2^-14 float16 has a fixed step of 2^-24, so its rounding is off by up to 2^-25 there whatever the value.
"""
import numpy as np
import pytest
import torch

import verify_router_gemv_amd as v
from oracle import verify_oracle
from verify_helpers import DEV, HALF, close, gen, host, i32, normal, say

pytestmark = pytest.mark.gpu


def pair_size(y, half, interleaved):
    """|a| + |b| of the pair an element is rotated with (|y| itself outside the rotated part)."""
    s = np.abs(y)
    out = s.copy()
    r = 2 * half
    if interleaved:
        out[..., 0:r:2] = out[..., 1:r:2] = s[..., 0:r:2] + s[..., 1:r:2]
    else:
        out[..., :half] = out[..., half:r] = s[..., :half] + s[..., half:r]
    return out


def check(T, heads, kv, D, rot, dtype, cache, P=16, interleaved=False, norm=(True, True), nhd=False, far=1 << 18, seed=0,
          skip=(), eps=1e-6, scale=1.0, in_place=False):
    say(f"case rope T={T} heads={heads}/{kv} D={D} rot={rot} {dtype}->{cache} P={P}")
    g = gen(seed)
    pages = -(-T // P) + 2
    qkv = normal(g, T, (heads + 2 * kv) * D + 8, dtype=dtype, scale=scale)[:, 8:].view(T, heads + 2 * kv, D) \
        if dtype != torch.float32 else normal(g, T, (heads + 2 * kv) * D + 4, scale=scale)[:, 4:].view(T, heads + 2 * kv, D)
    q, k, val = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    positions = torch.randint(0, far, (T,), generator=g, device=DEV).int()
    slots = torch.randperm(pages * P, generator=g, device=DEV)[:T].int()
    for t, s in skip:
        slots[t] = s
    inv_freq = (1e6 ** (-torch.arange(0, rot, 2, device=DEV).double() / max(rot, 1))).float()
    w = [1 + 0.3 * normal(g, D) if n else None for n in norm]
    shape = (pages, P, kv, D) if nhd else (pages, kv, P, D)
    caches = [normal(g, *shape, dtype=cache) for _ in range(2)]
    kc, vc = [c.permute(0, 2, 1, 3) if nhd else c for c in caches]
    before = [host(kc).copy(), host(vc).copy()]
    q_in = host(q).copy()
    out = q if in_place else normal(g, T, heads, D, dtype=cache)
    out_before = host(out).copy()
    got = v.qk_norm_rope(q, k, val, positions, slots, inv_freq, kc, vc, out, q_weight=w[0], k_weight=w[1], eps=eps,
                         interleaved=interleaved)
    assert got is out
    torch.cuda.synchronize()
    pos, freq, half = host(positions), host(inv_freq), rot // 2
    ref = [verify_oracle.norm_rope(x, None if ww is None else host(ww), pos, freq, eps, interleaved)
           for x, ww in ((q_in, w[0]), (host(k), w[1]))]
    u = HALF[cache]
    tol = [u * np.abs(y) + 2.0 ** -18 * pair_size(y, half, interleaved) + 2.0 ** -24 for y in ref]
    live = (host(slots) >= 0) & (host(slots) < pages * P)
    want, bound = np.where(live[:, None, None], ref[0], out_before), np.where(live[:, None, None], tol[0], 0)
    close(host(out), want, bound, "q_out")
    page, place = host(slots)[live] // P, host(slots)[live] % P
    for name, c, old, new, b in (("k_cache", kc, before[0], ref[1], tol[1]), ("v_cache", vc, before[1], host(val), None)):
        want, bound = old.copy(), np.zeros_like(old)
        want[page, :, place] = new[live]
        bound[page, :, place] = u * np.abs(new[live]) + 2.0 ** -25 if b is None else b[live]
        close(host(c), want, bound, name)


BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (F32, BF), (F32, FH)])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (256, 256), (256, 64), (256, 112), (128, 0)])
def test_types_and_heads(dtype, cache, D, rot):
    check(5, 6, 3, D, rot, dtype, cache, interleaved=False)
    check(3, 4, 1, D, rot, dtype, cache, interleaved=True)


@pytest.mark.parametrize("T", [1, 2, 63, 511, 512, 600])
def test_rows(T):
    check(T, 5, 1, 128, 128, BF, BF, seed=T)
    check(T, 33, 7, 64, 32, F32, FH, nhd=True, P=32, interleaved=True, seed=T)


@pytest.mark.parametrize("heads,kv", [(1, 1), (16, 16), (40, 8), (71, 71)])
def test_head_counts(heads, kv):
    check(4, heads, kv, 128, 64, BF, BF)
    check(513, heads, kv, 64, 64, BF, BF)


@pytest.mark.parametrize("norm", [(True, False), (False, True), (False, False)])
def test_without_norms(norm):
    check(4, 4, 2, 128, 128, BF, BF, norm=norm)


def test_pages_of_other_sizes():
    for P in (1, 7, 48, 1024):
        check(20, 4, 2, 64, 64, FH, FH, P=P)


def test_far_positions():
    check(40, 2, 1, 128, 128, F32, BF, far=(1 << 31) - 1)


def test_rows_without_a_slot_are_skipped():
    check(9, 4, 2, 128, 64, BF, BF, skip=((0, -1), (4, -5), (7, 1 << 30), (8, (1 << 31) - 1)))
    check(600, 4, 2, 64, 64, F32, BF, skip=((0, -1), (599, 16 * 40)))


def test_in_place_queries():
    check(7, 8, 2, 128, 128, BF, BF, in_place=True)
    check(520, 36, 4, 256, 64, FH, FH, in_place=True)


def test_extreme_values():
    check(3, 4, 2, 128, 128, F32, BF, scale=1e-12)      # the mean square is far below eps
    check(3, 4, 2, 128, 128, F32, BF, scale=1e15)
    check(3, 4, 2, 128, 128, BF, BF, scale=1e-12, eps=0.0)


def test_zero_rows_of_input_and_nan_stay_in_their_head():
    g = gen(3)
    q, k, val = normal(g, 4, 3, 128, dtype=BF), normal(g, 4, 2, 128, dtype=BF), normal(g, 4, 2, 128, dtype=BF)
    q[1, 1] = 0
    q[2, 0, 5] = float("nan")
    q[3, 2, 7] = float("inf")
    val[0, 1, 3] = float("-inf")
    kc, vc = normal(g, 2, 2, 16, 128, dtype=BF), normal(g, 2, 2, 16, 128, dtype=BF)
    w = torch.ones(128, device=DEV)
    out = v.qk_norm_rope(q, k, val, i32([0, 1, 2, 3]), i32([3, 17, 2, 30]), w[:64].contiguous(), kc, vc, q_weight=w, k_weight=w)
    assert (out[1, 1] == 0).all()
    nan = torch.isnan(out.float()).any(-1)
    assert nan.tolist() == [[False] * 3, [False] * 3, [True, False, False], [False, False, True]]
    assert vc[0, 1, 3, 3] == float("-inf") and torch.isfinite(kc.float()).all()


def test_refusals():
    g = gen(4)
    q, k = normal(g, 4, 4, 128, dtype=BF), normal(g, 4, 2, 128, dtype=BF)
    kc, vc = normal(g, 2, 2, 16, 128, dtype=BF), normal(g, 2, 2, 16, 128, dtype=BF)
    pos, f = i32([0, 1, 2, 3]), torch.ones(64, device=DEV)
    ok = dict(q=q, k=k, v=k, positions=pos, slots=pos, inv_freq=f, k_cache=kc, v_cache=vc)
    v.qk_norm_rope(**ok)
    wide = normal(g, 4, 4, 136, dtype=BF)
    for kw, err in ((dict(k=k[:3]), ValueError), (dict(v=k.float()), TypeError), (dict(positions=pos.long()), TypeError),
                    (dict(slots=pos[:3]), ValueError), (dict(k_cache=kc.half()), TypeError), (dict(v_cache=vc[:1]), ValueError),
                    (dict(q=q.half()), TypeError), (dict(inv_freq=f.double()), TypeError), (dict(inv_freq=f[:60]), v.MoeRoundError),
                    (dict(q_weight=f), ValueError), (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(q=wide[..., 1:129]), v.MoeRoundError), (dict(q_out=q[:, :, :]), None),
                    (dict(q_out=q.flip(0).view(-1)[:2048].view(4, 4, 128)[:, :, :64]), ValueError),
                    (dict(k_cache=kc[:, :, :1].expand(2, 2, 16, 128)), v.MoeRoundError), (dict(eps=-1.0), v.MoeRoundError)):
        if err is None:
            v.qk_norm_rope(**{**ok, **kw})
        else:
            with pytest.raises(err):
                v.qk_norm_rope(**{**ok, **kw})


def test_a_cache_past_32_bits():
    """Slots whose elements lie past 2^32: the last pages of a cache of more than 2^32 elements."""
    pages, kv, P, D = 4200, 64, 128, 128       # 4.4e9 elements, 8.8 GB
    kc = torch.empty(pages, kv, P, D, dtype=BF, device=DEV)
    vc = torch.empty(pages, kv, P, D, dtype=BF, device=DEV)
    g = gen(5)
    q, k, val = normal(g, 2, 1, D, dtype=BF), normal(g, 2, kv, D, dtype=BF), normal(g, 2, kv, D, dtype=BF)
    slots = i32([pages * P - 1, (pages - 2) * P + 5])
    v.qk_norm_rope(q, k, val, i32([5, 6]), slots, torch.ones(0, device=DEV), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(vc[pages - 1, :, P - 1], val[0]) and torch.equal(kc[pages - 1, :, P - 1], k[0])
    assert torch.equal(vc[pages - 2, :, 5], val[1]) and torch.equal(kc[pages - 2, :, 5], k[1])
