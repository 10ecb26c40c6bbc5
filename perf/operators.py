"""Cases of the verify round's operators around the MoE feed-forward, for timing and comparison.

Four operators: `round_slots` (block table, slot map, positions and tree masks of a round from the
requests' lengths), `qk_norm_rope` (norm and rotary position of the query and key heads, keys and
values written into the paged cache), `tree_attention` (each request's tree of drafted rows over the
paged cache) and `token_logprobs` (log probabilities of given tokens, entropy, top alternatives).
`run` evaluates a case in plain torch operations, or, with `own` set, through the package's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
THETA = 1000000.0


def listed():
    return [
        # one verify round of a few requests, each with a tree of up to 8 drafted rows
        dict(name="slots_verify", op="slots", requests=8, rows=8, context=4096, page=16, tree=True, pad=8),
        # a batch of prompts that enters the cache at once, every page taken from the free list
        dict(name="slots_prompts", op="slots", requests=1000, rows=1025, context=0, page=16, tree=False, pad=0),
        # the single row of plain decode
        dict(name="rope_one", op="rope", tokens=1, heads=16, kv_heads=2, dim=128, rot=128, page=16, type="bf16",
             cache="bf16", interleaved=False),
        # the widest verify round, float32 activations as the MoE round takes them
        dict(name="rope_verify", op="rope", tokens=64, heads=32, kv_heads=8, dim=128, rot=128, page=64, type="fp32",
             cache="bf16", interleaved=False),
        # a prompt with wide heads of which the first quarter is rotated
        dict(name="rope_prompt", op="rope", tokens=8191, heads=16, kv_heads=2, dim=256, rot=64, page=16, type="fp16",
             cache="fp16", interleaved=True),
        # plain decode of one request: the latency of a single token
        dict(name="attend_one", op="attend", requests=1, rows=1, context=1000, heads=16, kv_heads=2, dim=128, page=16,
             type="bf16"),
        # a batch of requests of uneven length, each verifying a tree of up to 8 rows
        dict(name="attend_verify", op="attend", requests=8, rows=8, context=8192, heads=32, kv_heads=4, dim=128,
             page=16, type="bf16"),
        # one request with a long context, a few drafted rows
        dict(name="attend_long", op="attend", requests=1, rows=5, context=131071, heads=32, kv_heads=8, dim=128,
             page=64, type="bf16"),
        # the widest trees: 64 rows of each request share its cache
        dict(name="attend_wide", op="attend", requests=4, rows=64, context=16384, heads=32, kv_heads=4, dim=128,
             page=64, type="fp16"),
        # one decoded row over a large vocabulary
        dict(name="logprobs_one", op="logprobs", tokens=1, vocab=248000, given=1, top=8, type="fp32"),
        # a verify round's rows, each with the tokens drafted below it
        dict(name="logprobs_verify", op="logprobs", tokens=24, vocab=151001, given=4, top=5, type="bf16"),
        # scoring a prompt: the log probability of every next token
        dict(name="logprobs_score", op="logprobs", tokens=2048, vocab=131072, given=1, top=1, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["slots", "rope", "attend", "attend", "logprobs"])
    most = max((work(c) for c in listed() if c["op"] == op), key=lambda w: w["bytes"] + w["flops"])
    while True:
        if op == "slots":
            tree = rng.random() < 0.6
            case = dict(op=op, requests=_log(rng, 1, 1000), rows=_log(rng, 1, 64 if tree else 2000),
                        context=_log(rng, 1, 65536) - 1, page=rng.choice([16, 32, 64, 128]), tree=tree,
                        pad=rng.choice([0, 1, 63]))
            if case["requests"] * (case["context"] + case["rows"]) > 1 << 24:
                continue
        elif op == "rope":
            dim = rng.choice([64, 128, 256])
            kv = rng.choice([1, 2, 4, 8])
            case = dict(op=op, tokens=_log(rng, 1, 8191), heads=kv * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv,
                        dim=dim, rot=rng.choice([dim, dim // 2]), page=rng.choice([16, 64, 128]), type="", cache="",
                        interleaved=rng.random() < 0.4)
            case["cache"] = rng.choice(["bf16", "fp16"])
            case["type"] = rng.choice([case["cache"], "fp32"])
        elif op == "attend":
            kv = rng.choice([1, 2, 4, 8])
            case = dict(op=op, requests=_log(rng, 1, 128), rows=_log(rng, 1, 64), context=_log(rng, 1, 131072) - 1,
                        heads=kv * rng.choice([1, 2, 4, 5, 7, 8, 16]), kv_heads=kv, dim=rng.choice([64, 128, 256]),
                        page=rng.choice([16, 32, 64, 128, 256]), type=rng.choice(["bf16", "fp16"]))
            keys = case["requests"] * (case["context"] + case["rows"] + case["page"])
            if keys * kv * case["dim"] > 1 << 27 or keys * case["rows"] * case["heads"] > 1 << 27:
                continue
        else:
            case = dict(op=op, tokens=_log(rng, 1, 2048), vocab=_log(rng, 1000, 260000), given=rng.choice([1, 2, 5, 16]),
                        top=rng.choice([0, 1, 4, 8, 16]), type=rng.choice(["bf16", "fp16", "fp32"]))
        w = work(case)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


def _lengths(case):
    """Cached lengths and new rows of each request: uneven, the same for every seed up to their order."""
    b = np.arange(case["requests"])
    cached = case["context"] - (b * (case["context"] // 2)) // case["requests"]
    rows = case["rows"] - (b % 3) * case["rows"] // 4
    return cached.astype(np.int64), rows.astype(np.int64)


def work(case):
    if case["op"] == "slots":
        cached, rows = _lengths(case)
        P = case["page"]
        total, pages = int(rows.sum()), int((-(-(cached + rows) // P) - -(-cached // P)).sum())
        n = total + case["pad"]
        tree = 12 * n if case["tree"] else 0
        return {"bytes": 12 * case["requests"] + 8 * n + tree + 8 * pages, "flops": 4 * n}
    if case["op"] == "rope":
        T, D, size = case["tokens"], case["dim"], TYPES[case["type"]].itemsize
        qkv = T * (case["heads"] + 2 * case["kv_heads"]) * D
        return {"bytes": qkv * (size + 2) + 8 * T + 8 * D + 2 * case["rot"], "flops": 10 * qkv}
    if case["op"] == "attend":
        cached, rows = _lengths(case)
        D, heads = case["dim"], case["heads"]
        keys, total = int((cached + rows).sum()), int(rows.sum())
        byte = 2 * 2 * keys * case["kv_heads"] * D + 2 * 2 * total * heads * D + 8 * total
        byte += 4 * int((-(-(cached + rows) // case["page"])).sum()) + 8 * case["requests"]
        return {"bytes": byte, "flops": 4 * heads * D * int((rows * (cached + rows)).sum())}
    n = case["tokens"] * case["vocab"]
    out = case["tokens"] * (12 * case["given"] + 8 * case["top"] + 4)
    return {"bytes": n * TYPES[case["type"]].itemsize + out, "flops": 5 * n}


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, type=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(type)


def _requests(case, seed, g):
    """Lengths in this seed's order, and a tree of drafted rows for each request (packed parents)."""
    cached, rows = _lengths(case)
    order = np.random.default_rng(seed).permutation(case["requests"])
    cached, rows = cached[order], rows[order]
    start = np.concatenate([[0], np.cumsum(rows)])
    within = torch.from_numpy(np.arange(start[-1]) - np.repeat(start[:-1], rows)).to(DEV)
    # a row hangs below one of the few rows before it: branching chains, as drafted trees are
    back = 1 + (torch.rand(int(start[-1]), generator=g, device=DEV) * 3).long()
    parents = (within - back).clamp(min=-1).int()
    return cached, rows, start, within, parents


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "slots":
        cached, rows, start, _, parents = _requests(case, seed, g)
        P, B = case["page"], case["requests"]
        old, all_ = -(-cached // P), -(-(cached + rows) // P)
        width = int(all_.max()) + 1
        pool = torch.randperm(int(all_.sum()) + 5, generator=g, device=DEV).int()
        table = np.full((B, width), -1, np.int64)
        used = 0
        for b in range(B):
            table[b, :old[b]] = np.arange(used, used + old[b])
            used += old[b]
        table = torch.from_numpy(table).to(DEV)
        table = torch.where(table >= 0, pool.long()[table.clamp(min=0)], table).int()
        total = int(start[-1]) + case["pad"]
        s.update(cached=torch.from_numpy(cached).int().to(DEV), rows=torch.from_numpy(rows).int().to(DEV), table=table,
                 free=pool[used:].contiguous(), page=P, total=total, parents=None, head=None)
        if case["tree"]:
            s["parents"] = torch.nn.functional.pad(parents, (0, case["pad"]), value=-1)
        return s
    if case["op"] == "rope":
        T, Hq, Hk, D, P = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
        pages = -(-T // P) + 3
        # query, key and value heads as one projection leaves them: side by side in each row
        qkv = _normal(g, T, (Hq + 2 * Hk) * D, type=TYPES[case["type"]]).view(T, Hq + 2 * Hk, D)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:],
                 positions=torch.randint(0, 1 << 18, (T,), generator=g, device=DEV).int(),
                 slots=torch.randperm(pages * P, generator=g, device=DEV)[:T].int(),
                 inv_freq=(THETA ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])).float(),
                 q_weight=1 + 0.1 * _normal(g, D), k_weight=1 + 0.1 * _normal(g, D),
                 k_cache=_normal(g, pages, Hk, P, D, type=TYPES[case["cache"]]),
                 v_cache=_normal(g, pages, Hk, P, D, type=TYPES[case["cache"]]),
                 q_out=torch.empty(T, Hq, D, dtype=TYPES[case["cache"]], device=DEV))
        if T > 1:  # a prompt's rows lie in consecutive places of its pages
            first = torch.randperm(pages, generator=g, device=DEV)[:, None] * P + torch.arange(P, device=DEV)
            s["slots"] = first.reshape(-1)[:T].int()
        return s
    if case["op"] == "attend":
        cached, rows, start, within, parents = _requests(case, seed, g)
        Hq, Hk, D, P, B = case["heads"], case["kv_heads"], case["dim"], case["page"], case["requests"]
        need = -(-(cached + rows) // P)
        pages, width = int(need.sum()), int(need.max())
        pool = torch.randperm(pages, generator=g, device=DEV)
        first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).to(DEV)
        column = torch.arange(width, device=DEV)
        table = pool[(first[:, None] + column).clamp(max=pages - 1)]
        table = torch.where(column < torch.from_numpy(need).to(DEV)[:, None], table, torch.full_like(table, -1)).int()
        total, R = int(start[-1]), case["rows"]
        s.update(q=_normal(g, total, Hq, D, type=TYPES[case["type"]]),
                 k_cache=_normal(g, pages, Hk, P, D, type=TYPES[case["type"]]),
                 v_cache=_normal(g, pages, Hk, P, D, type=TYPES[case["type"]]), table=table,
                 cached=torch.from_numpy(cached).int().to(DEV), row_start=torch.from_numpy(start).int().to(DEV),
                 masks=_ancestors(within, parents, start, R), max_rows=R, scale=1.5 / math.sqrt(D),
                 out=torch.zeros(total, Hq, D, dtype=TYPES[case["type"]], device=DEV))
        return s
    T, V = case["tokens"], case["vocab"]
    # a peak of likely tokens over a broad floor, as a language model's head gives them
    logits = 2.0 * _normal(g, T, V)
    peak = torch.randint(0, V, (T, 12), generator=g, device=DEV)
    logits.scatter_add_(1, peak, 6 + 4 * torch.rand(T, 12, generator=g, device=DEV))
    tokens = torch.randint(0, V, (T, case["given"]), generator=g, device=DEV)
    tokens[:, 0] = peak[:, 0]
    s.update(logits=logits.to(TYPES[case["type"]]), tokens=tokens.int(), top=case["top"])
    return s


def _ancestors(within, parents, start, rows):
    """Each row's visible rows of its request as the bits of an int64: itself and its ancestors."""
    if not len(within):
        return torch.zeros(0, dtype=torch.int64, device=DEV)
    request = torch.searchsorted(torch.from_numpy(start[1:]).to(DEV), torch.arange(len(within), device=DEV), right=True)
    step = torch.zeros(len(start) - 1, rows, rows, device=DEV)
    step[request, within, within] = 1
    step[request, within, parents.long().clamp(min=0)] = torch.where(parents >= 0, 1.0, step[request, within, 0])
    return _bits(_closure(step))[request, within]


def _closure(step):
    """Which rows a row reaches over any number of steps (up to 64)."""
    step = (step @ step).clamp(max=1)
    step = (step @ step).clamp(max=1)
    step = (step @ step).clamp(max=1)
    step = (step @ step).clamp(max=1)
    step = (step @ step).clamp(max=1)
    return (step @ step).clamp(max=1)


def _bits(reach):
    return ((reach > 0).long() << torch.arange(reach.shape[-1], device=DEV)).sum(-1)


def run(s):
    if own:
        import verify_router_gemv_amd as v
        op = s["case"]["op"]
        if op == "slots":
            r = v.round_slots(s["cached"], s["rows"], s["table"], s["free"], s["page"], s["total"], parents=s["parents"])
            out = [r.row_start, r.slots, r.positions, r.counts, s["table"]]
            return out if r.masks is None else out + [r.masks]
        if op == "rope":
            v.qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"], s["v_cache"],
                           s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                           interleaved=s["case"]["interleaved"])
            return [s["q_out"], s["k_cache"], s["v_cache"]]
        if op == "attend":
            v.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cached"], s["row_start"], s["out"],
                             masks=s["masks"], max_rows=s["max_rows"], scale=s["scale"])
            return s["out"]
        r = v.token_logprobs(s["logits"], s["tokens"], top=s["top"])
        return [r.logprobs, r.entropy, r.top_ids, r.top_logprobs]
    return {"slots": _slots, "rope": _rope, "attend": _attend, "logprobs": _logprobs}[s["case"]["op"]](s)


def _slots(s):
    P, table, total = s["page"], s["table"], s["total"]
    cached, rows = s["cached"].clamp(min=0).long(), s["rows"].clamp(min=0).long()
    B, W = table.shape
    ends = rows.cumsum(0)
    starts = ends - rows
    old = ((cached + P - 1) // P).clamp(max=W)
    need = ((cached + rows + P - 1) // P).clamp(max=W) - old
    taken = need.cumsum(0) - need
    column = torch.arange(W, device=DEV) - old[:, None]
    place = taken[:, None] + column
    fresh = torch.where(place < len(s["free"]), s["free"][place.clamp(0, len(s["free"]) - 1)], torch.full_like(table, -1))
    table.copy_(torch.where((column >= 0) & (column < need[:, None]), fresh, table))
    t = torch.arange(total, device=DEV)
    real = t < ends[-1]
    request = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    within = t - starts[request]
    index = cached[request] + within
    page = table[request, (index // P).clamp(max=W - 1)].long()
    slots = torch.where(real & (index // P < W) & (page >= 0), page * P + index % P, torch.full_like(t, -1)).int()
    row_start = torch.cat([starts[:1], ends]).clamp(max=total).int()
    counts = torch.stack([ends[-1], need.sum()]).int()
    if s["parents"] is None:
        positions = torch.where(real, index, torch.zeros_like(index)).int()
        return [row_start, slots, positions, counts, table]
    R = 64
    at = starts[:, None] + torch.arange(R, device=DEV)
    inside = torch.arange(R, device=DEV) < rows[:, None]
    parent = torch.where(inside, s["parents"][at.clamp(max=total - 1)].long(), torch.full_like(at, -1))
    step = torch.eye(R, device=DEV) + (parent[:, :, None] == torch.arange(R, device=DEV)).float()
    reach = _closure(step)
    bits, depth = _bits(reach), reach.sum(-1).long() - 1
    positions = torch.where(real, cached[request] + depth[request, within.clamp(max=R - 1)], torch.zeros_like(t)).int()
    masks = torch.where(real, bits[request, within.clamp(max=R - 1)], torch.zeros_like(t))
    return [row_start, slots, positions, counts, table, masks]


def _rope(s):
    D, rot = s["q"].shape[-1], 2 * len(s["inv_freq"])
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
        if s["case"]["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1).to(s["k_cache"].dtype)

    P = s["k_cache"].shape[2]
    page, place = s["slots"].long() // P, s["slots"].long() % P
    s["q_out"].copy_(turned(s["q"], s["q_weight"]))
    s["k_cache"][page, :, place] = turned(s["k"], s["k_weight"])
    s["v_cache"][page, :, place] = s["v"].to(s["v_cache"].dtype)
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _attend(s):
    q, table, R = s["q"], s["table"], s["max_rows"]
    T, Hq, D = q.shape
    Hk, P = s["k_cache"].shape[1:3]
    B, W = table.shape
    pages = table.clamp(min=0).long()
    keys = s["k_cache"][pages].permute(0, 2, 4, 1, 3).reshape(B, Hk, D, W * P).float()
    values = s["v_cache"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hk, W * P, D).float()
    start, cached = s["row_start"].long(), s["cached"].long()
    rows = start[1:] - start[:-1]
    row = torch.arange(R, device=DEV)
    at = (start[:-1, None] + row).clamp(max=T - 1)
    x = q[at].float().view(B, R, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    scores = (x @ keys).mul_(s["scale"]).view(B, Hk, Hq // Hk, R, W * P)
    node = torch.arange(W * P, device=DEV) - cached[:, None]
    drafted = (node >= 0) & (node < rows[:, None])
    bit = (s["masks"][at][:, :, None] >> node.clamp(0, 63)[:, None]) & 1
    seen = (node < 0)[:, None] | (drafted[:, None] & (bit == 1))
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hk, -1, W * P) @ values).view(B, Hk, Hq // Hk, R, D) / total.clamp(min=1e-30)
    t = torch.arange(T, device=DEV)
    request = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return out.to(q.dtype)[request, :, :, t - start[request]].reshape(T, Hq, D)


def _logprobs(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    z = top + total.log()
    logprobs = x.gather(1, s["tokens"].long()) - z
    entropy = total.squeeze(1).log() - (p * (x - top)).sum(-1) / total.squeeze(1)
    if not s["top"]:
        ids = torch.zeros(len(x), 0, dtype=torch.int32, device=DEV)
        return [logprobs, entropy, ids, torch.zeros(len(x), 0, device=DEV)]
    best, ids = x.sort(dim=-1, descending=True, stable=True)
    return [logprobs, entropy, ids[:, :s["top"]].int(), best[:, :s["top"]] - z]


def exact(case, seed):
    """The case's outputs from the definitions, request by request, in 64 bits."""
    s = prepare(case, seed)
    return {"slots": _exact_slots, "rope": _exact_rope, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_slots(s):
    P, total = s["page"], s["total"]
    cached, rows, table, free = (s[n].cpu().numpy().astype(np.int64) for n in ("cached", "rows", "table", "free"))
    parents = s["parents"].cpu().numpy() if s["parents"] is not None else None
    slots, positions = np.full(total, -1, np.int32), np.zeros(total, np.int32)
    masks, row_start, taken, t = np.zeros(total, np.uint64), [0], 0, 0
    for b in range(len(cached)):
        c, n = int(cached[b]), int(rows[b])
        for page in range(-(-c // P), -(-(c + n) // P)):
            table[b, page] = free[taken]
            taken += 1
        index = np.arange(c, c + n)
        slots[t:t + n] = table[b, index // P] * P + index % P
        positions[t:t + n] = index
        if parents is not None:
            depth, mask = [], []
            for i in range(n):
                up = int(parents[t + i])
                depth.append(0 if up < 0 else depth[up] + 1)
                mask.append((1 << i) | (0 if up < 0 else mask[up]))
            positions[t:t + n] = c + np.array(depth, np.int32)
            masks[t:t + n] = np.array(mask, np.uint64)
        t += n
        row_start.append(t)
    i32 = lambda x: torch.as_tensor(np.asarray(x), device=DEV).int()  # noqa: E731
    out = [i32(row_start), i32(slots), i32(positions), i32([t, taken]), i32(table)]
    return out if parents is None else out + [torch.from_numpy(masks.view(np.int64)).to(DEV)]


def _exact_rope(s):
    half = len(s["inv_freq"])
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]

    def head(x, weight):
        x = x.double()
        x = weight.double() * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        part = x[..., :2 * half]
        if s["case"]["interleaved"]:
            pairs = torch.view_as_complex(part.reshape(*part.shape[:-1], half, 2).contiguous()) * turn
            part = torch.view_as_real(pairs).reshape(part.shape)
        else:
            pairs = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
            part = torch.cat([pairs.real, pairs.imag], -1)
        return torch.cat([part, x[..., 2 * half:]], -1)

    caches = []
    for cache, new in ((s["k_cache"], head(s["k"], s["k_weight"])), (s["v_cache"], s["v"].double())):
        pages, Hk, P, D = cache.shape
        flat = cache.double().transpose(1, 2).reshape(pages * P, Hk, D)
        flat[s["slots"].long()] = new
        caches.append(flat.view(pages, P, Hk, D).transpose(1, 2).contiguous())
    return [head(s["q"], s["q_weight"]), *caches]


def _exact_attend(s):
    q, P = s["q"].double(), s["k_cache"].shape[2]
    Hq, Hk, D = q.shape[1], s["k_cache"].shape[1], q.shape[2]
    start, cached = s["row_start"].tolist(), s["cached"].tolist()
    out = torch.zeros_like(q)
    for b in range(len(cached)):
        n, c = start[b + 1] - start[b], cached[b]
        index = torch.arange(c + n, device=DEV)
        page, place = s["table"][b].long()[index // P], index % P
        mask = s["masks"][start[b]:start[b + 1]]
        bit = torch.arange(n, device=DEV)
        unseen = torch.cat([torch.zeros(n, c, dtype=torch.bool, device=DEV), ((mask[:, None] >> bit) & 1) == 0], 1)
        for h in range(Hk):
            k, v = s["k_cache"][page, h, place].double(), s["v_cache"][page, h, place].double()
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            x = q[start[b]:start[b + 1], heads].reshape(-1, D)
            score = s["scale"] * (x @ k.t().contiguous())
            score = score.masked_fill(unseen.repeat_interleave(Hq // Hk, 0), -math.inf)
            out[start[b]:start[b + 1], heads] = (torch.softmax(score, -1) @ v).view(n, -1, D)
    return out


def _exact_logprobs(s):
    x = s["logits"]
    z = torch.cat([torch.logsumexp(row.double(), -1) for row in x.split(128)])
    entropy = torch.cat([lz - (torch.softmax(row.double(), -1) * row.double()).sum(-1)
                         for row, lz in zip(x.split(128), z.split(128))])
    ids = torch.empty(len(x), s["top"], dtype=torch.int64, device=DEV)
    left = x.float()
    column = torch.arange(x.shape[1], device=DEV)
    for j in range(s["top"]):
        best = left.amax(-1, keepdim=True)
        ids[:, j] = torch.where(left == best, column, x.shape[1]).amin(-1)
        left = left.scatter(1, ids[:, j:j + 1], -math.inf)
    return [x.gather(1, s["tokens"].long()).double() - z[:, None], entropy, ids.int(),
            x.gather(1, ids).double() - z[:, None]]
