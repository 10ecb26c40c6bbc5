"""The operators of a verify round together, as a program calls them: slots, then per layer the norm, rotary
position and cache write, the attention and the MoE round, then the log probabilities; several rounds over one
cache, eagerly and as one captured graph, each stage against its oracle on the GPU's own inputs (needs an MI355X)."""
import numpy as np
import pytest
import torch

import oracle
import synth
import verify_router_gemv_amd as v
from moe_helpers import assert_close, oracle_view
from oracle import verify_oracle
from verify_helpers import DEV, HALF, close, gen, host, i32, normal, random_parents, say

pytestmark = pytest.mark.gpu


class Model:
    """Two layers of a small MoE transformer with random weights."""

    def __init__(self, seed=0, heads=8, kv=2, D=64, P=16, pages=96, vocab=5003):
        self.cfg = synth.ShapeConfig("small", H=512, E=16, k=4, I=256)
        H, g = self.cfg.H, gen(seed)
        self.heads, self.kv, self.D, self.P, self.vocab = heads, kv, D, P, vocab
        self.layers = []
        for l in range(2):
            moe = synth.make_layer(self.cfg, seed=seed, layer=l, device=DEV)
            self.layers.append(dict(
                moe=moe, wqkv=normal(g, H, (heads + 2 * kv) * D, scale=H ** -0.5), wo=normal(g, heads * D, H, scale=H ** -0.5),
                qw=1 + 0.1 * normal(g, D), kw=1 + 0.1 * normal(g, D),
                kc=torch.zeros(pages, kv, P, D, dtype=torch.bfloat16, device=DEV),
                vc=torch.zeros(pages, kv, P, D, dtype=torch.bfloat16, device=DEV),
                round=v.MoeRound([moe], H, self.cfg.I, self.cfg.E, self.cfg.k, max_rows=32, use_graph=False,
                                 exact=True, stream=torch.cuda.current_stream())))
        self.head = normal(g, H, vocab, scale=0.2)
        self.inv_freq = (1e4 ** (-torch.arange(0, D, 2, device=DEV).double() / D)).float()

    def run(self, x, cached, rows, table, free, head, parents, drafted, keep=None):
        N = x.shape[0]
        s = v.round_slots(cached, rows, table, free, self.P, N, parents=parents, free_head=head)
        for L in self.layers:
            qkv = (x @ L["wqkv"]).view(N, self.heads + 2 * self.kv, self.D)
            q, k, val = qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv], qkv[:, self.heads + self.kv:]
            qo = torch.zeros(N, self.heads, self.D, dtype=torch.bfloat16, device=DEV)
            v.qk_norm_rope(q, k, val, s.positions, s.slots, self.inv_freq, L["kc"], L["vc"], qo, q_weight=L["qw"], k_weight=L["kw"])
            a = v.tree_attention(qo, L["kc"], L["vc"], table, cached, s.row_start, masks=s.masks)
            h = x + a.view(N, -1).float() @ L["wo"]
            out = torch.empty_like(h)
            L["round"].run(h, self.cfg.k, out)
            if keep is not None:
                keep.append(dict(q=q, qo=qo, k=k, val=val, a=a, h=h, moe=out))
            x = h + out
        logits = x @ self.head
        return s, logits, v.token_logprobs(logits, drafted, top=3)


def one_round(m, rng, cached, table, free, head, N=32):
    rows = rng.integers(0, 9, len(cached))
    parents = random_parents(rng, rows, N)
    x = normal(gen(int(rng.integers(1 << 30))), N, m.cfg.H)
    return rows, parents, x, torch.from_numpy(rng.integers(0, m.vocab, (N, 3)).astype(np.int32)).to(DEV)


def test_rounds_stage_by_stage():
    m, rng = Model(), np.random.default_rng(0)
    cached = np.array([0, 30, 5], np.int32)
    free_np = rng.permutation(96).astype(np.int32)
    table_np = np.full((3, 8), -1, np.int32)
    # the committed context arrives as a prompt: one round of chains fills its pages
    table, free, head = i32(table_np), i32(free_np), i32([0])
    x = normal(gen(1), 35, m.cfg.H)
    for L in m.layers:
        L["round"].close()
        L["round"] = v.MoeRound([L["moe"]], m.cfg.H, m.cfg.I, m.cfg.E, m.cfg.k, max_rows=128, exact=True)
    drafted = torch.zeros(35, 1, dtype=torch.int32, device=DEV)
    s, _, _ = m.run(x, i32([0, 0, 0]), i32(cached), table, free, head, None, drafted)
    assert host(s.counts).tolist() == [35, 3]
    head += s.counts[1:]
    for step in range(4):
        rows, parents, x, drafted = one_round(m, rng, cached, table, free, head)
        say(f"case round {step} rows={rows.tolist()} cached={cached.tolist()}")
        before, head_np = host(table).copy(), int(head)
        keep = []
        s, logits, lp = m.run(x, i32(cached), i32(rows), table, free, head, i32(parents), drafted, keep)
        torch.cuda.synchronize()
        ref = verify_oracle.round_slots(cached, rows, before, free_np, m.P, 32, parents, head_np)
        for got, want in zip((*s, table), ref):
            assert np.array_equal(host(got), want), f"step {step}: slots"
        T = int(rows.sum())
        slots, u = host(s.slots)[:T], HALF[torch.bfloat16]
        for l, (L, k) in enumerate(zip(m.layers, keep)):
            y = verify_oracle.norm_rope(host(k["q"])[:T], host(L["qw"]), host(s.positions)[:T], host(m.inv_freq), 1e-6, False)
            close(host(k["qo"])[:T], y, u * np.abs(y) + 2.0 ** -16, f"step {step} layer {l}: queries")
            y = verify_oracle.norm_rope(host(k["k"])[:T], host(L["kw"]), host(s.positions)[:T], host(m.inv_freq), 1e-6, False)
            close(host(L["kc"])[slots // m.P, :, slots % m.P], y, u * np.abs(y) + 2.0 ** -16, f"step {step} layer {l}: keys")
            close(host(L["vc"])[slots // m.P, :, slots % m.P], host(k["val"])[:T], u * np.abs(host(k["val"])[:T]) + 2.0 ** -30, "values")
            out, spread, _ = verify_oracle.tree_attention(host(k["qo"]), host(L["kc"]), host(L["vc"]), host(table), cached,
                                                          host(s.row_start), host(s.masks), 64, m.D ** -0.5)
            close(host(k["a"])[:T], out[:T], 2.1 * u * spread[:T] + 2.0 ** -20, f"step {step} layer {l}: attention")
            assert (host(k["a"])[T:] == 0).all()
            moe, _, _, _ = oracle.moe_round([oracle_view(L["moe"])], k["h"].cpu().numpy(), m.cfg.k, residual=False)
            assert_close(k["moe"].cpu().numpy(), moe, f"step {step} layer {l}: MoE")
        w = verify_oracle.token_logprobs(host(logits), host(drafted), 3)
        close(host(lp.logprobs), w[0], 2e-5, "log probabilities")
        close(host(lp.entropy), w[1], 2e-4, "entropy")
        assert np.array_equal(host(lp.top_ids), w[2])
        head += s.counts[1:]
        # accept the first row of each tree and the chain below it: here simply some leading rows
        cached = cached + np.minimum(rows, rng.integers(0, 4, 3)).astype(np.int32)


def test_a_captured_round_equals_the_eager_one():
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        m, rng = Model(seed=1), np.random.default_rng(1)
        c, r, p, hd = i32([0, 0, 0]), i32([0, 0, 0]), i32(np.full(32, -1)), i32([0])
        table, free = i32(np.full((3, 8), -1)), i32(rng.permutation(96))
        x, drafted = normal(gen(2), 32, m.cfg.H), torch.zeros(32, 3, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        m.run(x, c, r, table, free, hd, p, drafted)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s, logits, lp = m.run(x, c, r, table, free, hd, p, drafted)
        cached = np.zeros(3, np.int32)
        for _ in range(4):
            rows, parents, x_new, d_new = one_round(m, rng, cached, table, free, hd)
            for d, new in ((c, i32(cached)), (r, i32(rows)), (p, i32(parents)), (x, x_new), (drafted, d_new)):
                d.copy_(new)
            torch.cuda.synchronize()
            saved = [t.clone() for L in m.layers for t in (L["kc"], L["vc"])] + [table.clone()]
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (*s, logits, *lp, table, *(t for L in m.layers for t in (L["kc"], L["vc"])))]
            for t, old in zip([*(t for L in m.layers for t in (L["kc"], L["vc"])), table], saved):
                t.copy_(old)
            es, elogits, elp = m.run(x, c, r, table, free, hd, p, drafted)
            torch.cuda.synchronize()
            want = (*es, elogits, *elp, table, *(t for L in m.layers for t in (L["kc"], L["vc"])))
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            hd += es.counts[1:]
            cached = cached + np.minimum(rows, 2).astype(np.int32)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_the_outputs_of_a_call_are_tensors_of_their_own(mode):
    with mode():
        x = normal(gen(3), 5, 999)
        tokens = torch.randint(999, (5, 2), device=DEV)
        lp = v.token_logprobs(x, tokens, top=4)
        s = v.round_slots(i32([3, 20]), i32([2, 3]), i32(np.zeros((2, 4))), i32([7]), 16, 6, i32([-1, 0, -1, 0, 0, -1]))
        for made in (lp, s):
            before = [t.clone() for t in made]
            for i, t in enumerate(made):
                assert t.is_contiguous() and not t.requires_grad
                t.add_(1)                        # changes none of the others
                for j, (other, old) in enumerate(zip(made, before)):
                    assert torch.equal(other, old + (j <= i)), f"{j} after a change of {i}"
                assert torch.equal(t.flatten().view(-1), t.clone().flatten())
        del lp, s, x                             # an output outlives its call's other tensors
        lp = v.token_logprobs(normal(gen(4), 3, 50), None, top=1).top_logprobs
        torch.cuda.synchronize()
        assert lp.shape == (3, 1) and bool((lp < 0).all())
