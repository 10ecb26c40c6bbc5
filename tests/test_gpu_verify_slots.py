"""round_slots against the plain oracle: every output is a whole number and must be equal (needs an MI355X)."""
import numpy as np
import pytest
import torch

import verify_router_gemv_amd as v
from oracle import verify_oracle
from verify_helpers import DEV, host, i32, random_parents, say

pytestmark = pytest.mark.gpu


def make(rng, B, rows, context, P, width=None, spare=3):
    cached = rng.integers(0, context + 1, B)
    new = rng.integers(0, rows + 1, B)
    need = -(-(cached + new) // P)
    width = width or max(1, int(need.max(initial=1))) + 1
    pool = rng.permutation(int(need.sum()) + spare).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    used = 0
    for b in range(B):
        n = min(-(-int(cached[b]) // P), width)
        table[b, :n] = pool[used:used + n]
        used += n
    return cached.astype(np.int32), new.astype(np.int32), table, pool[used:]


def check(cached, rows, table, free, P, N, parents=None, head=None, what="", strided=False, out=None):
    say(f"case slots {what} B={len(cached)} P={P} N={N}")
    B, W = table.shape
    big = torch.full((B, W + 5), -99, dtype=torch.int32, device=DEV) if strided else None
    t = big[:, :W] if strided else torch.empty(B, W, dtype=torch.int32, device=DEV)
    t.copy_(torch.from_numpy(table))
    r = v.round_slots(i32(cached), i32(rows), t, i32(free), P, N,
                      parents=None if parents is None else i32(parents),
                      free_head=None if head is None else i32([head]), out=out)
    ref = verify_oracle.round_slots(cached, rows, table, free, P, N, parents, head or 0)
    for name, got, want in zip(("row_start", "slots", "positions", "masks", "counts"), r, ref):
        if want is None:
            assert got is None
        else:
            assert np.array_equal(got.cpu().numpy(), want), f"{what}: {name}"
    assert np.array_equal(t.cpu().numpy(), ref[5]), f"{what}: table"
    if strided:
        assert (big[:, W:] == -99).all()
    return r


@pytest.mark.parametrize("B,rows,context,P", [
    (1, 1, 0, 16), (1, 1, 1000, 16), (3, 8, 40, 16), (4, 64, 100, 1), (5, 64, 4000, 7), (64, 8, 500, 32),
    (65, 17, 300, 128), (257, 5, 64, 64), (1000, 3, 90, 16),
])
def test_trees(B, rows, context, P):
    rng = np.random.default_rng(B * 7 + rows)
    cached, new, table, free = make(rng, B, rows, context, P)
    N = int(new.sum()) + 9
    check(cached, new, table, free, P, N, random_parents(rng, new, N), what="tree", strided=B % 2 == 1)


@pytest.mark.parametrize("B,rows,context,P", [
    (1, 1, 0, 16), (1, 40000, 0, 16), (2, 3000, 65, 64), (3, 1, 131071, 256), (300, 200, 30, 16), (4096, 2, 9, 8),
    (9001, 3, 40, 16),
])
def test_chains(B, rows, context, P):
    rng = np.random.default_rng(B + rows)
    cached, new, table, free = make(rng, B, rows, context, P)
    check(cached, new, table, free, P, int(new.sum()) + (B % 3), what="chain")


def test_no_requests_and_no_rows():
    none = np.zeros(0, np.int32)
    check(none, none, np.zeros((0, 4), np.int32), np.arange(3, dtype=np.int32), 16, 5, what="B = 0")
    check(none, none, np.zeros((0, 4), np.int32), none, 16, 0, what="B = 0, N = 0")
    zero = np.zeros(3, np.int32)
    table = np.full((3, 4), 2, np.int32)
    check(zero, zero, table, none, 16, 4, parents=np.full(4, -1), what="no rows")
    check(np.array([5, 16, 17], np.int32), zero, table, none, 16, 0, what="N = 0")


def test_what_does_not_fit_is_left_out():
    rng = np.random.default_rng(5)
    cached, new, table, free = make(rng, 12, 60, 100, 16)
    N = int(new.sum())
    check(cached, new, table, free[:5], 16, N, what="too few pages")
    check(cached, new, table, free[:0], 16, N, what="no pages")
    check(cached, new, table[:, :4], free, 16, N, what="a narrow table")
    check(cached, new, table, free, 16, N // 2, random_parents(rng, new, N // 2), what="rows past the buffer")
    check(-cached, new, table, free, 16, N, what="negative lengths count as 0")
    check(cached, -new, table, free, 16, 7, what="negative rows count as 0")
    bad = random_parents(rng, new, N)
    bad[::5] = 77
    bad[::7] = -3
    check(cached, new, table, free, 16, N, bad, what="parents out of range")
    table[3, 0] = -1
    check(cached, new, table, free, 16, N, what="a missing page in the table")


def test_lengths_at_the_end_of_32_bits():
    last = 2 ** 31 - 1
    cached, new = np.array([last, last - 3, 5], np.int32), np.array([4, 8, 2], np.int32)
    table, free, N = i32(np.zeros((3, 4))), i32(np.arange(4)), 15
    for parents in (None, i32([-1, 0, 1, 2, -1, 0, 1, 2, 3, 4, 5, 6, -1, 0, -1])):
        s = v.round_slots(i32(cached), i32(new), table.clone(), free, 16, N, parents)
        want = [min(int(c) + i, last) for c, n in zip(cached, new) for i in range(n)] + [0]
        assert host(s.positions).tolist() == want
        assert (host(s.slots)[:12] == -1).all() and host(s.slots)[12:14].tolist() == [5, 6]


def test_more_than_64_rows_in_a_tree():
    rng = np.random.default_rng(6)
    cached, new, table, free = make(rng, 4, 300, 50, 16)
    new[:] = [65, 64, 300, 1]
    N = int(new.sum()) + 2
    check(cached, new, table, np.arange(100, dtype=np.int32), 16, N, random_parents(rng, new, N), what="wide trees")
    chain = np.concatenate([np.arange(r) - 1 for r in new] + [[-1, -1]]).astype(np.int32)
    check(cached, new, table, np.arange(100, dtype=np.int32), 16, N, chain, what="a chain as a tree")


def test_free_head_moves_along_the_list():
    rng = np.random.default_rng(7)
    cached, new, table, free = make(rng, 9, 50, 60, 16, spare=40)
    for head in (0, 1, 11, len(free), len(free) + 5, -2):
        check(cached, new, table, free, 16, int(new.sum()), head=head, what=f"head {head}")


def test_the_same_buffers_again():
    rng = np.random.default_rng(8)
    out = None
    for _ in range(3):
        cached, new, table, free = make(rng, 6, 9, 70, 16, width=12)
        out = check(cached, new, table, free, 16, 60, random_parents(rng, new, 60), out=out, what="reused")
    with pytest.raises(ValueError, match="out.masks"):
        v.round_slots(i32(cached), i32(new), i32(table), i32(free), 16, 60, out=out)
    with pytest.raises(ValueError, match="length"):
        v.round_slots(i32(cached), i32(new), i32(table), i32(free), 16, 61, parents=i32(np.zeros(61)), out=out)


def test_captured_round_follows_the_lengths():
    rng = np.random.default_rng(9)
    cached, new, table, free = make(rng, 7, 8, 100, 16, width=20)
    c, r, t, f = i32(cached), i32(new), i32(table), i32(np.arange(200))
    p = i32(np.full(64, -1))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        out = v.round_slots(c, r, t, f, 16, 64, parents=p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        v.round_slots(c, r, t, f, 16, 64, parents=p, out=out)
    for _ in range(4):
        cached, new, table, _ = make(rng, 7, 8, 100, 16, width=20)
        parents = random_parents(rng, new, 64)
        for d, x in ((c, cached), (r, new), (t, table), (p, parents)):
            d.copy_(torch.from_numpy(x))
        graph.replay()
        torch.cuda.synchronize()
        ref = verify_oracle.round_slots(cached, new, table, np.arange(200), 16, 64, parents)
        for got, want in zip((*out, t), ref):
            assert np.array_equal(got.cpu().numpy(), want)
