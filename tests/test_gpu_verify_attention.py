"""tree_attention against the float64 oracle (needs an MI355X).

Bound per element, with u = HALF of the type, A = sum_j p_j |v_j|, reach = the largest scale * sum_d |q_d k_jd|:
  u A       each probability is rounded once to the type for its product with the values;
  u |out|   the output is rounded once;
  e A       float32 arithmetic: a score sums 128 or 256 products (relative 2^-24 of reach times at most 64, in the
            matrix unit's order), the exponent 1.45 |s - m| is rounded to 2^-24 of reach, the exponential to
            2^-22, sums and joins of parts to some 2^-20 in all: e = 2^-18 (1 + reach), twice (p and the sum);
  n 2^-30 max|v|   probabilities below the type's normal range keep an absolute step only (float16, relative to
            the running maximum: 2^-25 of 2^-7).
"""
import numpy as np
import pytest
import torch

import verify_router_gemv_amd as v
from oracle import verify_oracle
from verify_helpers import DEV, HALF, close, gen, host, i32, normal, random_parents, say

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16


class Case:
    """A filled cache with requests of the given lengths; everything between the tokens is garbage (NaN)."""

    def __init__(self, cached, rows, heads=4, kv=2, D=128, P=16, dtype=BF, tree=True, nhd=False, seed=0, pad=0,
                 garbage=float("nan"), extra_pages=2, qscale=2.0, extra_cols=1):
        rng, g = np.random.default_rng(seed), gen(seed)
        cached, rows = np.asarray(cached), np.asarray(rows)
        B, T = len(cached), int(rows.sum()) + pad
        need = -(-(cached + rows) // P)
        pages = int(need.sum()) + extra_pages
        order = rng.permutation(pages)
        W = int(need.max(initial=0)) + extra_cols
        table = np.full((B, W), -1, np.int32)
        shape = (pages, P, kv, D) if nhd else (pages, kv, P, D)
        self.kc, self.vc = [torch.full(shape, garbage, dtype=dtype, device=DEV) for _ in range(2)]
        if nhd:
            self.kc, self.vc = self.kc.permute(0, 2, 1, 3), self.vc.permute(0, 2, 1, 3)
        used = 0
        for b in range(B):
            table[b, :need[b]] = order[used:used + need[b]]
            used += need[b]
            n = int(cached[b] + rows[b])
            idx = torch.arange(n, device=DEV)
            page = torch.from_numpy(table[b].astype(np.int64)).to(DEV)[idx // P]
            self.kc[page, :, idx % P] = normal(g, n, kv, D, dtype=dtype)
            self.vc[page, :, idx % P] = normal(g, n, kv, D, dtype=dtype)
        start = np.concatenate([[0], np.cumsum(rows)])
        self.masks = None
        if tree:
            _, _, _, m, _, _ = verify_oracle.round_slots(cached, rows, table, [], P, T, random_parents(rng, rows, T))
            self.masks = torch.from_numpy(m).to(DEV)
        self.q = normal(g, T, heads, D, dtype=dtype, scale=qscale)
        self.cached, self.start, self.table = i32(cached), i32(start), i32(table).view(B, W)
        self.max_rows, self.scale, self.dtype = max(1, min(64, int(rows.max(initial=1)))), D ** -0.5, dtype
        self.T, self.D = T, D

    def run(self, out=None, **kw):
        return v.tree_attention(self.q, self.kc, self.vc, self.table, self.cached, self.start, out,
                                **{**dict(masks=self.masks, max_rows=self.max_rows, scale=self.scale), **kw})

    def check(self, what="", rows=None, **kw):
        say(f"case attention {what} T={self.T} B={len(self.cached)} q={tuple(self.q.shape)} kc={tuple(self.kc.shape)} {self.dtype}")
        q = host(self.q)
        out = torch.full_like(self.q, 7.0)
        self.run(out, **kw)
        torch.cuda.synchronize()
        max_rows = kw.get("max_rows", self.max_rows)
        masks = kw.get("masks", self.masks)
        ref, spread, reach = verify_oracle.tree_attention(
            q, host(self.kc), host(self.vc), host(self.table), host(self.cached), host(self.start),
            None if masks is None else host(masks), max_rows, kw.get("scale", self.scale))
        none = np.isnan(ref).all(-1) & (np.abs(spread).sum(-1) == 0)     # rows of no request
        got = host(out)
        assert (got[none] == 7).all(), f"{what}: rows of no request were written"
        n = int((host(self.cached)).max(initial=0)) + 64
        u = HALF[self.dtype]
        vmax = np.nanmax(np.where(np.isfinite(host(self.vc)), np.abs(host(self.vc)), 0), initial=0)
        with np.errstate(invalid="ignore"):
            tol = u * spread + u * np.abs(ref) + 2.0 ** -17 * (1 + reach[..., None]) * spread + n * 2.0 ** -30 * vmax
        close(got[~none], ref[~none], tol[~none], what)
        return out


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (4, 2), (5, 1), (16, 2), (14, 2)])
def test_heads_and_types(dtype, D, heads, kv):
    Case([100, 0, 37], [1, 1, 1], heads, kv, D, dtype=dtype).check("one row")
    Case([70, 5, 300], [3, 8, 5], heads, kv, D, dtype=dtype, seed=1).check("trees")


@pytest.mark.parametrize("cached", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513, 1000])
def test_lengths(cached):
    Case([cached], [1], 2, 1, 128).check("decode")
    Case([cached, 3], [7, 2], 8, 2, 64, dtype=FH, P=32, seed=cached).check("tree")
    Case([cached, cached + 1], [40, 64], 4, 2, 128, P=64, tree=False, seed=cached).check("chain")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,group", [(1, 16), (2, 16), (3, 8), (16, 2), (17, 1), (33, 1), (64, 1), (16, 8), (20, 7), (64, 4), (64, 8)])
def test_row_tiles(D, rows, group):
    """Every tile height, and several row blocks of one request."""
    Case([200, 40, 999], [rows, max(1, rows // 2), rows], group, 1, D, P=16, seed=rows).check("rows")


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256, 1024])
def test_pages(P):
    Case([300, 31, 1029], [5, 1, 64], 4, 2, 64, P=P, dtype=FH).check("pages")
    Case([300, 31, 1029], [5, 1, 64], 4, 2, 128, P=P, nhd=True).check("pages, tokens before heads")


def test_long_context_in_many_parts():
    Case([40001, 3, 9000], [2, 1, 6], 2, 1, 128, P=64, seed=3).check("split")
    Case([6000], [64], 8, 1, 64, P=64, seed=4).check("split, several row blocks")
    Case([3000, 100], [64, 30], 6, 2, 256, P=128, dtype=FH, seed=5).check("split, several row blocks, wide heads")


def test_many_requests():
    rng = np.random.default_rng(6)
    for B in (63, 64, 65, 130, 300):
        Case(rng.integers(0, 90, B), rng.integers(0, 4, B), 2, 1, 64, seed=B, pad=2).check(f"{B} requests")
    Case(np.full(200, 20), np.full(200, 2), 4, 4, 64, seed=1).check("200 requests")
    rows = np.zeros(140, int)
    rows[[2, 100, 139]] = [3, 64, 1]
    Case(rng.integers(0, 900, 140), rows, 8, 1, 128, seed=2).check("most without rows")


def test_very_many_requests():
    rng = np.random.default_rng(7)
    for B in (128, 129, 1024, 1025, 4200):
        Case(rng.integers(0, 40, B), rng.integers(0, 4, B), 2, 2, 64, seed=B, pad=2).check(f"{B} requests")
    rows = np.zeros(1100, int)
    rows[[0, 7, 8, 500, 1099]] = [33, 64, 1, 20, 64]
    Case(rng.integers(0, 90, 1100), rows, 16, 1, 64, seed=3).check("several row blocks, most without rows")
    cached = np.zeros(1100, int)
    cached[600] = 9000
    Case(cached, np.ones(1100, int), 4, 2, 128, P=64, seed=4).check("one long context among many")


def test_peaked_scores():
    for dtype in (BF, FH):
        Case([3000, 64], [4, 2], 4, 2, 128, dtype=dtype, qscale=30.0, seed=7).check("peaked")
        Case([500], [4], 4, 2, 128, dtype=dtype, qscale=0.0, seed=8).check("flat")


def test_rising_scores():
    """Scores that grow along the context: the running maximum is raised in every tile."""
    for dtype in (BF, FH):
        c = Case([2000], [2], 2, 1, 128, P=64, dtype=dtype, seed=9)
        c.q[:] = 1.0
        for j in range(2002):
            page = int(c.table[0, j // 64])
            c.kc[page, :, j % 64] = 0.002 * j
        c.check("rising")


def test_rows_that_see_nothing():
    c = Case([0, 50, 0], [4, 3, 2], 4, 2, 128, seed=10)
    c.masks[:] = 0
    out = c.check("empty masks")
    assert (out[:4] == 0).all() and (out[7:9] == 0).all() and (out[4:7] != 0).any()
    c = Case([40], [3], 8, 1, 64)
    c.table[:] = -1
    assert (c.check("no pages") == 0).all()


def test_mask_bits_past_the_rows_count_for_nothing():
    c = Case([30, 30], [3, 64], 2, 1, 128, seed=11)
    c.masks[:3] = -1
    c.masks[5] = -(1 << 63)
    c.check("bits past the rows")


def test_pages_that_are_missing():
    c = Case([300, 200], [5, 3], 4, 2, 128, seed=12)
    c.table[0, 3] = -1
    c.table[0, 7] = c.kc.shape[0]
    c.table[1, 0] = 1 << 30
    c.table[1, 12] = -(1 << 31)
    c.check("bad pages")
    c = Case([300, 200], [5, 3], 4, 2, 128, P=64, seed=13, extra_cols=0)
    c.table = c.table[:, :4].contiguous()            # 256 tokens: the rows of request 0 lie past it
    c.check("a narrow table")


def test_infinity_and_nan_stay_with_the_rows_that_see_them():
    inf, nan = float("inf"), float("nan")
    for dtype in (BF, FH):
        for D, heads, rows in ((128, 4, 8), (64, 16, 20), (256, 4, 40)):
            c = Case([77, 20], [rows, 3], heads, 2, D, dtype=dtype, seed=14)
            P = 16
            c.masks[:rows] = torch.tensor([(1 << i) | 1 for i in range(rows)], device=DEV)   # siblings below row 0
            at = lambda i: (int(c.table[0, (77 + i) // P]), (77 + i) % P)  # noqa: E731
            p, o = at(2)
            c.vc[p, 0, o, 3] = nan
            c.vc[p, 1, o, 5] = inf
            p, o = at(5)
            c.kc[p, :, o] = nan
            p, o = at(rows - 1)
            c.vc[p, :, o, D - 1] = -inf
            c.kc[p, 0, o, 1] = inf
            out = host(c.check(f"siblings {D}"))
            bad = ~np.isfinite(out).all((1, 2))
            assert sorted(np.nonzero(bad)[0]) == sorted({2, 5, rows - 1})
            q = c.q.clone()
            c.q[4] = nan
            out = host(c.run())
            assert np.isnan(out[4]).all() and np.isfinite(out[[0, 1, 3, 6]]).all()
            c.q = q


def test_rows_of_no_request_and_past_max_rows_are_left():
    c = Case([40, 10], [6, 3], 4, 2, 128, pad=4, seed=15)
    c.check("padding")
    c.check("max_rows", max_rows=4)
    c.start[1:] += 2                                    # request 0 has two more rows
    c.start[2] = 9
    c.masks = None
    c.check("other row starts")


def test_odd_row_starts_stay_inside():
    c = Case([40, 10, 30], [6, 3, 2], 4, 2, 128, seed=16)
    for start in ([0, 6, 900, 11], [-5, 3, 3, 11], [11, 11, 11, 11], [4, 2, 5, 1 << 30]):
        c.start = i32(start)
        out = torch.full_like(c.q, 7.0)
        c.run(out)
        torch.cuda.synchronize()
        assert torch.isfinite(out.float()).all()


def test_negative_and_too_long_lengths_stay_inside():
    c = Case([40, 64], [2, 2], 4, 2, 128, P=64, seed=17, extra_cols=0)
    c.cached = i32([-3, (1 << 31) - 1])
    c.table[1] = c.table[1].clamp(min=0)
    c.kc.nan_to_num_(0.0)
    c.vc.nan_to_num_(0.0)
    out = c.run()
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()


def test_in_place_and_strided_rows():
    c = Case([90, 33], [5, 7], 6, 3, 128, seed=18)
    ref = c.run()
    wide = torch.zeros(c.T, 10, 136, dtype=BF, device=DEV)
    view = wide[:, 2:8, 8:]
    view.copy_(c.q)
    c.q = view
    out = torch.full((6, c.T, 128), 7.0, dtype=BF, device=DEV).transpose(0, 1)
    c.run(out)
    assert torch.equal(out, ref)
    c.run(view)
    assert torch.equal(view, ref) and (wide[:, :2] == 0).all() and (wide[:, 8:] == 0).all() and (wide[..., :8] == 0).all()


def test_repeated_runs_are_equal_and_rows_do_not_leak():
    c = Case([5000, 300], [8, 3], 16, 2, 128, seed=19)
    a = c.run()
    for _ in range(3):
        assert torch.equal(a, c.run())
    # another row's query changes nothing in this row
    q = c.q.clone()
    c.q[1:8] = 5.0
    assert torch.equal(a[0], c.run()[0])
    c.q = q


def test_two_streams_and_graphs_at_once():
    cs = [Case([3000 + 500 * i, 40], [6, 3], 8, 2, 128, seed=20 + i) for i in range(2)]
    eager = [c.run() for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs, graphs = [], []
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(c.run())
        graphs.append(graph)
    for i in range(4):
        for c in cs:
            c.q.copy_(normal(gen(40 + i), *c.q.shape, dtype=BF))
            c.cached[1] = 10 * i
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            assert torch.equal(o, c.run())
        both = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                both.append(c.run())
        torch.cuda.synchronize()
        for b, o in zip(both, outs):
            assert torch.equal(b, o)
    assert not torch.equal(outs[0], eager[0])


def test_a_cache_past_32_bits():
    """Pages whose elements lie past 2^32, in both caches."""
    pages, kv, P, D = 4200, 64, 128, 128
    kc = torch.zeros(pages, kv, P, D, dtype=BF, device=DEV)
    vc = torch.zeros(pages, kv, P, D, dtype=BF, device=DEV)
    g = gen(21)
    kc[pages - 2:] = normal(g, 2, kv, P, D, dtype=BF)
    vc[pages - 2:] = normal(g, 2, kv, P, D, dtype=BF)
    q = normal(g, 2, kv, D, dtype=BF)
    small = v.tree_attention(q, kc[pages - 2:].contiguous(), vc[pages - 2:].contiguous(), i32([[1, 0]]), i32([200]), i32([0, 2]))
    far = v.tree_attention(q, kc, vc, i32([[pages - 1, pages - 2]]), i32([200]), i32([0, 2]))
    assert torch.equal(small, far) and (far != 0).any()


def test_empty_calls_and_refusals():
    c = Case([40, 10], [6, 3], 4, 2, 128, seed=22)
    assert v.tree_attention(c.q[:0], c.kc, c.vc, c.table, c.cached, c.start).shape == (0, 4, 128)
    out = torch.full_like(c.q, 7.0)
    v.tree_attention(c.q, c.kc, c.vc, c.table[:0], c.cached[:0], c.start[:1], out)
    assert (out == 7).all()
    for kw, err in ((dict(masks=c.masks[:3]), ValueError), (dict(masks=c.masks.int()), TypeError), (dict(scale=0.0), v.MoeRoundError),
                    (dict(max_rows=65), v.MoeRoundError), (dict(max_rows=0), v.MoeRoundError), (dict(out=c.q[:4]), ValueError),
                    (dict(out=c.q.half()), TypeError), (dict(out=c.q[:, :1].expand(9, 4, 128)), v.MoeRoundError)):
        with pytest.raises(err):
            c.run(**kw)
    with pytest.raises(v.MoeRoundError):                 # pages of 8 tokens
        v.tree_attention(c.q, c.kc[:, :, :8], c.vc[:, :, :8], c.table, c.cached, c.start)
    with pytest.raises(v.MoeRoundError):                 # three heads over two
        v.tree_attention(c.q[:, :3], c.kc, c.vc, c.table, c.cached, c.start)
    with pytest.raises(ValueError, match="GPU"):
        v.tree_attention(c.q, c.kc, c.vc, c.table.cpu(), c.cached, c.start)
