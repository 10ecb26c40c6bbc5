"""The verify-round operators without a GPU: exported symbols and argument structs, refusals of the C entries
and of the binding, and hand-worked pins of their float64 oracle."""
import ctypes
import math
import os
import re
import struct
import subprocess

import numpy as np
import pytest
import torch

import verify_router_gemv_amd as v
from conftest import ROOT
from oracle import verify_oracle
from verify_router_gemv_amd import binding, verify_ops

HEADER = os.path.join(ROOT, "include", "verify_ops.h")
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from verify_router_gemv_amd import build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    verify_ops._native()
    lib = binding.load()
    args, vp, i64 = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int64
    for name, res, sig in (
            ("verify_round_slots", ctypes.c_int32, [args, vp]),
            ("verify_qk_norm_rope", ctypes.c_int32, [args, vp]),
            ("verify_tree_attention_workspace", i64, [args]),
            ("verify_tree_attention", ctypes.c_int32, [args, vp, i64, vp]),
            ("verify_token_logprobs_workspace", i64, [args]),
            ("verify_token_logprobs", ctypes.c_int32, [args, vp, i64, vp]),
            ("verify_last_hip_error", ctypes.c_int32, [])):
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, sig
    return lib


def declared():
    return sorted(set(re.findall(r"MOE_ROUND_API\s+[\w\s\*]+?\b(verify_\w+)\s*\(", open(HEADER).read())))


def test_library_exports_exactly_the_declared_symbols(lib):
    assert len(declared()) == 7
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if " T verify_" in l) == declared()


STRUCTS = {k: f"verify_{k}_args" for k in ("slots", "rope", "attention", "logprobs")}


def fields(kind):
    """(name, struct code) of the header's fields, read from its text."""
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % ((STRUCTS[kind],) * 2), open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    out = []
    for line in body.split(";"):
        line = " ".join(line.split())
        if not line:
            continue
        kind_, names = re.match(r"((?:const )?(?:void|float|int32_t|int64_t)\s*\*?)\s*(.*)", line).groups()
        code = "P" if "*" in kind_ else {"int64_t": "q", "int32_t": "i", "float": "f"}[kind_.strip()]
        out += [(n.strip(), code) for n in names.split(",")]
    return out


def layout(kind):
    """The struct's packing: the header's fields in order, each at its own alignment."""
    return struct.Struct("@" + "".join(c for _, c in fields(kind)))


def pack(kind, f):
    return layout(kind).pack(*[f[n] for n, _ in fields(kind)])


P16 = 0x100000   # a made-up aligned address: every check here comes before any GPU call


def base(kind):
    f = {n: P16 if c == "P" else 0 for n, c in fields(kind)}
    f["struct_bytes"] = (layout(kind).size + 7) // 8 * 8
    if kind == "slots":
        f.update(n_requests=2, width=4, table_stride=4, n_free=3, page_size=16, total_rows=5)
    elif kind == "rope":
        f.update(q=0x1000000, q_row=512, q_head=128, k_row=256, k_head=128, v_row=256, v_head=128, o_row=512,
                 o_head=128, kc_page=4096, kc_head=2048, kc_token=128, vc_page=4096, vc_head=2048, vc_token=128,
                 n_pages=7, n_rows=3, heads=4, kv_heads=2, dim=128, page_size=16, n_freq=64, in_type=1, cache_type=1,
                 eps=1e-6)
    elif kind == "attention":
        f.update(q_row=512, q_head=128, o_row=512, o_head=128, kc_page=4096, kc_head=2048, kc_token=128, vc_page=4096,
                 vc_head=2048, vc_token=128, table_stride=90, n_pages=7, n_rows=3, n_requests=2, heads=4, kv_heads=2,
                 dim=128, page_size=16, width=90, max_rows=8, type=1, scale=0.1)
    else:
        f.update(row_stride=1000, n_rows=3, vocab=1000, n_tokens=2, top=4, type=1)
    return f


def call(lib, kind, **kw):
    f = {**base(kind), **kw}
    args = pack(kind, f)
    if kind == "slots":
        return lib.verify_round_slots(args, None)
    if kind == "rope":
        return lib.verify_qk_norm_rope(args, None)
    if kind == "attention":
        return lib.verify_tree_attention(args, None, 0, None)
    return lib.verify_token_logprobs(args, None, 0, None)


BAD = [
    ("slots", dict(struct_bytes=120), INVALID), ("slots", dict(reserved=1), INVALID),
    ("slots", dict(n_requests=-1), INVALID), ("slots", dict(width=0), INVALID), ("slots", dict(page_size=0), INVALID),
    ("slots", dict(total_rows=-1), INVALID), ("slots", dict(n_free=-1), INVALID), ("slots", dict(table_stride=3), INVALID),
    ("slots", dict(masks=0), INVALID), ("slots", dict(parents=0), INVALID), ("slots", dict(cached=0), INVALID),
    ("slots", dict(rows=P16 + 2), INVALID), ("slots", dict(table=0), INVALID), ("slots", dict(free_pages=0), INVALID),
    ("slots", dict(slots=0), INVALID), ("slots", dict(counts=0), INVALID), ("slots", dict(row_start=0), INVALID),
    ("slots", dict(masks=P16 + 4), INVALID), ("slots", dict(free_head=P16 + 1), INVALID),
    ("slots", dict(n_requests=65537), UNSUPPORTED), ("slots", dict(page_size=65537), UNSUPPORTED),
    ("slots", dict(total_rows=16777217), UNSUPPORTED), ("slots", dict(total_rows=16777216), UNSUPPORTED),
    ("rope", dict(n_rows=16777216), UNSUPPORTED), ("logprobs", dict(n_rows=16777216), UNSUPPORTED),
    ("rope", dict(struct_bytes=0), INVALID), ("rope", dict(heads=0), INVALID), ("rope", dict(kv_heads=0), INVALID),
    ("rope", dict(n_pages=0), INVALID), ("rope", dict(page_size=0), INVALID), ("rope", dict(eps=-1.0), INVALID),
    ("rope", dict(eps=math.nan), INVALID), ("rope", dict(eps=math.inf), INVALID), ("rope", dict(interleaved=2), INVALID),
    ("rope", dict(q=0), INVALID), ("rope", dict(k=P16 + 8), INVALID), ("rope", dict(q_row=513), INVALID),
    ("rope", dict(v_head=-128), INVALID), ("rope", dict(kc_token=1 << 25), INVALID), ("rope", dict(kc_token=0), INVALID),
    ("rope", dict(vc_page=0), INVALID), ("rope", dict(o_head=0), INVALID), ("rope", dict(positions=0), INVALID),
    ("rope", dict(slots=P16 + 1), INVALID), ("rope", dict(q_weight=P16 + 4), INVALID),
    ("rope", dict(q_out=0x1000000 + 256), INVALID),                      # overlaps q
    ("rope", dict(q_out=0x1000000, o_row=1024), INVALID),                # q itself, other strides
    ("rope", dict(q_out=0x1000000, in_type=0), INVALID),                 # q itself, another type
    ("rope", dict(dim=96), UNSUPPORTED), ("rope", dict(n_freq=60), UNSUPPORTED), ("rope", dict(n_freq=72), UNSUPPORTED),
    ("rope", dict(in_type=2), UNSUPPORTED), ("rope", dict(cache_type=0), UNSUPPORTED), ("rope", dict(in_type=3), UNSUPPORTED),
    ("rope", dict(heads=1025), UNSUPPORTED),
    ("attention", dict(struct_bytes=1), INVALID), ("attention", dict(heads=3), INVALID), ("attention", dict(kv_heads=0), INVALID),
    ("attention", dict(width=0), INVALID), ("attention", dict(n_pages=0), INVALID), ("attention", dict(max_rows=0), INVALID),
    ("attention", dict(scale=0.0), INVALID), ("attention", dict(scale=-1.0), INVALID), ("attention", dict(scale=math.nan), INVALID),
    ("attention", dict(scale=math.inf), INVALID), ("attention", dict(table_stride=89), INVALID),
    ("attention", dict(q=0), INVALID), ("attention", dict(out=P16 + 8), INVALID), ("attention", dict(masks=P16 + 4), INVALID),
    ("attention", dict(o_row=0), INVALID), ("attention", dict(kc_token=132), INVALID), ("attention", dict(table=0), INVALID),
    ("attention", dict(cached=0), INVALID), ("attention", dict(row_start=P16 + 2), INVALID),
    ("attention", dict(width=64, out=P16 + 256), INVALID),               # overlaps q (no workspace is needed)
    ("attention", dict(width=64, o_row=1024), INVALID),                  # q itself, other strides
    ("attention", dict(), INVALID),                                      # the context may split: no workspace given
    ("attention", dict(dim=80), UNSUPPORTED), ("attention", dict(type=0), UNSUPPORTED),
    ("attention", dict(page_size=8), UNSUPPORTED), ("attention", dict(page_size=48), UNSUPPORTED),
    ("attention", dict(max_rows=65), UNSUPPORTED), ("attention", dict(heads=130), UNSUPPORTED),
    ("attention", dict(n_rows=1 << 20, heads=64, kv_heads=1, q=1 << 40), UNSUPPORTED),          # the join's threads
    ("attention", dict(width=64, n_requests=65536, max_rows=64, heads=1024, kv_heads=64, q=1 << 40), UNSUPPORTED),  # the blocks
    ("attention", dict(width=1 << 27, table_stride=1 << 27), UNSUPPORTED),
    ("logprobs", dict(struct_bytes=80), INVALID), ("logprobs", dict(vocab=0), INVALID), ("logprobs", dict(n_tokens=-1), INVALID),
    ("logprobs", dict(row_stride=999), INVALID), ("logprobs", dict(tokens_64=2), INVALID), ("logprobs", dict(logits=0), INVALID),
    ("logprobs", dict(logits=P16 + 1), INVALID), ("logprobs", dict(tokens=0), INVALID), ("logprobs", dict(tokens=P16 + 4, tokens_64=1), INVALID),
    ("logprobs", dict(top_ids=0), INVALID), ("logprobs", dict(logprobs=0), INVALID), ("logprobs", dict(vocab=3, top=4), INVALID),
    ("logprobs", dict(top=17), UNSUPPORTED), ("logprobs", dict(type=3), UNSUPPORTED),
]


@pytest.mark.parametrize("kind,kw,expect", BAD, ids=lambda x: str(x) if not isinstance(x, dict) else "-".join(x) or "workspace")
def test_bad_arguments_are_refused_before_any_gpu_call(lib, kind, kw, expect):
    assert call(lib, kind, **kw) == expect


def test_null_structs_and_empty_calls(lib):
    assert lib.verify_round_slots(None, None) == INVALID
    assert lib.verify_qk_norm_rope(None, None) == INVALID
    assert lib.verify_tree_attention(None, None, 0, None) == INVALID
    assert lib.verify_token_logprobs(None, None, 0, None) == INVALID
    assert lib.verify_tree_attention_workspace(None) == INVALID
    assert lib.verify_token_logprobs_workspace(None) == INVALID
    assert call(lib, "rope", n_rows=0, q=0, k=0, v=0, q_out=0, positions=0, slots=0) == 0
    assert call(lib, "attention", n_rows=0, q=0, out=0) == 0
    assert call(lib, "attention", n_requests=0, table=0, cached=0) == 0
    assert call(lib, "logprobs", n_rows=0, logits=0) == 0
    assert lib.verify_last_hip_error() == 0


def test_workspace_sizes(lib):
    def need(**kw):
        f = {**base("attention"), **kw}
        return lib.verify_tree_attention_workspace(pack("attention", f))
    assert need(width=64) == 0            # 1024 tokens: one part
    assert need(width=65) > 0
    assert need(width=64, n_requests=128) == 0 and need(width=64, n_requests=129) == 129 * 8   # the cut's plan
    assert need(n_rows=0) == 0 and need(scale=0.0) == INVALID
    f = base("logprobs")
    assert lib.verify_token_logprobs_workspace(pack("logprobs", f)) > 0
    assert lib.verify_token_logprobs_workspace(pack("logprobs", {**f, "n_rows": 0})) == 0
    assert lib.verify_token_logprobs_workspace(pack("logprobs", {**f, "vocab": 0})) == INVALID


def test_binding_refuses_host_tensors_and_wrong_types():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        v.round_slots(i32(2), i32(2), i32(2, 4), i32(3), 16, 5)
    with pytest.raises(TypeError):
        v.round_slots(i32(2), i32(2), torch.zeros(2, 4), i32(3), 16, 5)
    with pytest.raises(TypeError):
        v.round_slots([1, 2], i32(2), None, i32(3), 16, 5)
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    cache = torch.zeros(7, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        v.qk_norm_rope(x, x[:, :2], x[:, 2:], i32(3), i32(3), torch.zeros(64), cache, cache)
    with pytest.raises(ValueError, match="GPU"):
        v.tree_attention(x, cache, cache, i32(2, 4), i32(2), i32(3))
    with pytest.raises(TypeError):
        v.tree_attention(x.float(), cache, cache, i32(2, 4), i32(2), i32(3))
    with pytest.raises(ValueError, match="GPU"):
        v.token_logprobs(torch.zeros(3, 100))
    with pytest.raises(TypeError):
        v.token_logprobs(torch.zeros(3, 100, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        v.token_logprobs(torch.zeros(100))


# ---------------------------------------------------------------------------
# hand-worked pins of the oracle
# ---------------------------------------------------------------------------

def test_oracle_slots_by_hand():
    # pages of 4; request 0 has 3 tokens on page 9 and gets 3 rows, request 1 is new with 2
    table = [[9, -1, -1], [-1, -1, -1]]
    rs, slots, pos, masks, counts, out = verify_oracle.round_slots(
        [3, 0], [3, 2], table, [5, 6, 7], 4, 7, parents=[-1, 0, 0, -1, -1, 99, 99])
    assert rs.tolist() == [0, 3, 5] and counts.tolist() == [5, 2]
    assert out.tolist() == [[9, 5, -1], [6, -1, -1]]
    assert slots.tolist() == [39, 20, 21, 24, 25, -1, -1]
    assert pos.tolist() == [3, 4, 4, 0, 0, 0, 0]
    assert masks.tolist() == [1, 3, 5, 1, 2, 0, 0]
    # a chain, too few pages, a narrow table, rows past the buffer
    rs, slots, pos, masks, counts, out = verify_oracle.round_slots([0, 2], [3, 9], [[-1], [8]], [1], 2, 6)
    assert masks is None and rs.tolist() == [0, 3, 6] and counts.tolist() == [12, 1]
    assert slots.tolist() == [2, 3, -1, -1, -1, -1] and pos.tolist() == [0, 1, 2, 2, 3, 4]
    assert out.tolist() == [[1], [8]]


def test_oracle_rope_by_hand():
    x = np.array([[[3.0, 4.0, 5.0, 6.0]]])
    y = verify_oracle.norm_rope(x, None, [2], [math.pi / 4], 0.0, False)     # a quarter turn of (0, 1)
    assert np.allclose(y, [[[-4, 3, 5, 6]]])
    y = verify_oracle.norm_rope(x, None, [1], [math.pi / 2, math.pi], 0.0, False)   # (0, 2) and (1, 3)
    assert np.allclose(y, [[[-5, -4, 3, -6]]])
    y = verify_oracle.norm_rope(x, None, [1], [math.pi / 2, math.pi], 0.0, True)    # (0, 1) and (2, 3)
    assert np.allclose(y, [[[-4, 3, -5, -6]]])
    y = verify_oracle.norm_rope(x, [1, 1, 2, 2], [0], [1.0], 0.0, False)
    assert np.allclose(y, x / math.sqrt(86 / 4) * [1, 1, 2, 2])


def test_oracle_attention_by_hand():
    # one head of 2, pages of 2; tokens 0, 1 cached, rows 0 and 1 siblings: each sees itself only
    k = np.zeros((3, 1, 2, 2))
    val = np.zeros((3, 1, 2, 2))
    val[2, 0] = [[1, 0], [2, 0]]
    val[0, 0] = [[6, 1], [9, np.nan]]
    q = np.zeros((3, 1, 2))
    out, _, _ = verify_oracle.tree_attention(q, k, val, np.array([[2, 0, 7]]), [2], [0, 2], np.array([1, 2, 0]), 64, 1.0)
    assert np.allclose(out[0, 0], [3, 1 / 3]) and math.isnan(out[1, 0, 1]) and np.isnan(out[2]).all()
    k[2, 0, 1] = [math.log(3), 0]
    q[0, 0] = [1, 0]
    out, _, _ = verify_oracle.tree_attention(q, k, val, np.array([[2, 0]]), [2], [0, 1], None, 64, 1.0)
    assert np.allclose(out[0, 0], [(1 + 3 * 2 + 6) / 5, 1 / 5])
    out, _, _ = verify_oracle.tree_attention(q, k, val, np.array([[-1, 3]]), [2], [0, 1], None, 64, 1.0)
    assert (out[0] == 0).all()


def test_oracle_logprobs_by_hand():
    x = np.array([[0, math.log(3), -np.inf, math.log(3)], [-np.inf] * 4])
    lp, h, ids, tlp = verify_oracle.token_logprobs(x, np.array([[0, 2, 4], [0, 1, -1]]), 3)
    assert np.allclose(lp[0], [-math.log(7), -np.inf, -np.inf]) and (lp[1] == -np.inf).all()
    assert np.allclose(h, [math.log(7) - 6 / 7 * math.log(3), 0])
    assert ids.tolist() == [[1, 3, 0], [0, 1, 2]]
    assert np.allclose(tlp[0], np.log([3 / 7, 3 / 7, 1 / 7])) and (tlp[1] == -np.inf).all()
