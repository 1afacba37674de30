"""Drafted trees over a paged cache: what is timed and compared.

An actor's drafts are verified against a target whose keys and values lie in a paged cache.  Three
operators lie between the drafter and `rl_infra_gb300.ops.verify_draft`:

  append   keys and values of drafted (or prompted) tokens into the cache, keys and queries rotated by
           their positions on the way (`ops.cache_append`)
  attend   attention of a tree of drafted tokens over the cache (`ops.tree_attention`); one node a
           sequence is the step of plain decoding
  keep     the accepted path of each tree moved to where the sequence goes on (`ops.cache_keep`)

`own` chooses between the plain forms below (elementary torch operations in 32 bits, angles in 64,
rounded once at the end) and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# -- the cases --------------------------------------------------------------------------------
# b sequences, n new tokens each, hkv heads of keys and g query heads to each, d entries a head, pages of
# `page` slots, up to ctx tokens of context.

def listed():
    return [
        # one token of one sequence: latency
        dict(name="append_one", op="append", b=1, n=1, hkv=8, g=4, d=128, page=16, ctx=1000, dtype="bf16",
             rot=128, pairs=False, tree=False, far=0),
        # a serving batch's drafted trees, far into their sequences
        dict(name="append_tree", op="append", b=64, n=24, hkv=8, g=4, d=128, page=64, ctx=2000, dtype="f16",
             rot=128, pairs=False, tree=True, far=120000),
        # 32 bits, an odd page, heads of 80 entries of which 32 are rotated in neighbouring pairs
        dict(name="append_partial", op="append", b=7, n=333, hkv=12, g=1, d=80, page=24, ctx=500, dtype="f32",
             rot=32, pairs=True, tree=False, far=0),
        # prompts of odd length
        dict(name="append_prompt", op="append", b=4, n=8191, hkv=8, g=4, d=128, page=64, ctx=700, dtype="bf16",
             rot=128, pairs=False, tree=False, far=0),
        # one token over a short context: latency
        dict(name="attend_one", op="attend", b=1, n=1, hkv=8, g=4, d=128, page=16, ctx=1023, dtype="bf16", tree=False),
        # a decoding batch of ragged sequences
        dict(name="attend_decode", op="attend", b=64, n=1, hkv=8, g=4, d=128, page=16, ctx=5000, dtype="bf16", tree=False),
        # drafted trees of a serving batch
        dict(name="attend_tree", op="attend", b=16, n=24, hkv=8, g=4, d=64, page=64, ctx=8000, dtype="f16", tree=True),
        # a chain of drafts over one long sequence
        dict(name="attend_long", op="attend", b=1, n=8, hkv=8, g=4, d=128, page=64, ctx=262145, dtype="bf16", tree=False),
        # 32 bits, odd heads and pages, no shared heads
        dict(name="attend_odd", op="attend", b=5, n=13, hkv=12, g=1, d=80, page=24, ctx=3001, dtype="f32", tree=True),
        # large trees of a large target: 512 rows to each head of keys
        dict(name="attend_wide", op="attend", b=32, n=64, hkv=8, g=8, d=128, page=64, ctx=6000, dtype="bf16", tree=True),
        # what a verified serving batch keeps
        dict(name="keep_batch", op="keep", b=64, n=24, most=6, hkv=8, d=128, page=64, ctx=300, dtype="bf16"),
        # actors of a large rollout
        dict(name="keep_large", op="keep", b=1024, n=48, most=12, hkv=8, d=128, page=16, ctx=30, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "keep"])
    while True:
        d = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128, 256])
        case = dict(op=op, hkv=rng.choice([1, 2, 3, 4, 8, 8, 12]), d=d, page=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                    dtype=rng.choice(["f32", "f16", "bf16", "bf16"]))
        if op == "append":
            case.update(b=_log(rng, 1, 256), n=_log(rng, 1, 8192), g=rng.choice([1, 2, 4, 5, 8]), ctx=_log(rng, 1, 3000),
                        rot=rng.choice([d, d, d // 2, 0]), pairs=rng.random() < 0.3, far=rng.choice([0, 1000000]))
            case["tree"] = case["n"] <= 64 and rng.random() < 0.6
        elif op == "attend":
            case.update(b=_log(rng, 1, 128), n=_log(rng, 1, 96), g=rng.choice([1, 2, 4, 5, 8]), ctx=_log(rng, 1, 200000))
            case["tree"] = case["n"] > 1 and rng.random() < 0.6
        else:
            case.update(b=_log(rng, 1, 1024), n=rng.randint(2, 64), ctx=_log(rng, 1, 1000))
            case["most"] = min(case["n"], rng.randint(1, 12))
        like = [c for c in listed() if c["op"] == op]
        slots = case["b"] * (case["ctx"] + case["n"]) * case["hkv"] * d * BYTES[case["dtype"]]
        if slots <= 1 << 30 and all(work(case)[k] <= max(work(c)[k] for c in like) for k in ("bytes", "flops")):
            return case


def _lens(b, ctx):
    """Tokens that sequence i has: between half of ctx and ctx, one in 16 (past the first few) has none."""
    return [0 if i % 16 == 5 else ctx - (i * 7919 * ctx // 20011) % max(1, ctx // 2) for i in range(b)]


def _counts(b, n):
    """New tokens that sequence i has: n, one in 8 half of them."""
    return [(n + 1) // 2 if i % 8 == 3 else n for i in range(b)]


def work(case):
    e, b, n, hkv, d = BYTES[case["dtype"]], case["b"], case["n"], case["hkv"], case["d"]
    if case["op"] == "keep":
        kept = sum(1 + i % case["most"] for i in range(b))
        return {"bytes": kept * hkv * d * e * 4 + kept * 4 + b * 16, "flops": 0}
    lens, counts = _lens(b, case["ctx"]), _counts(b, n)
    new = sum(counts)
    rows = (case["g"] + 2) * hkv
    if case["op"] == "append":
        return {"bytes": new * (rows * d * e * 2 + 4) + b * 8, "flops": new * (case["g"] + 1) * hkv * case["rot"] * 3}
    seen, heads = sum(lens) + new, case["g"] * hkv
    return {"bytes": seen * hkv * d * e * 2 + new * heads * (2 * d * e + 4) + (n * n if case["tree"] else 0),
            "flops": sum(4 * c * heads * d * (s + (c + 1) // 2) for s, c in zip(lens, counts))}


# -- the inputs -------------------------------------------------------------------------------

def _cache(case, g, used):
    """Keys, values [pages, page, hkv, d], scattered pages, and the table of each sequence's pages."""
    b, page, dt = case["b"], case["page"], DTYPES[case["dtype"]]
    width = -(-max(used) // page)
    pages = b * width
    shape = (pages, page, case["hkv"], case["d"])
    k, v = torch.empty(shape, dtype=dt, device="cuda"), torch.empty(shape, dtype=dt, device="cuda")
    part = max(1, (1 << 27) // (page * case["hkv"] * case["d"]))
    for t in (k, v):
        for r in range(0, pages, part):
            t[r:r + part] = torch.randn((min(part, pages - r), *shape[1:]), generator=g, device="cuda").to(dt)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).reshape(b, width)
    return k, v, table


def _tree(n, g):
    """Depths [n] and ancestors [n, n] (bool, themselves among them) of a tree whose node 0 is the root."""
    at = torch.arange(n, device="cuda")
    parent = (torch.rand(n, generator=g, device="cuda") * at).long().clamp_min(0)
    up = torch.zeros(n, n, device="cuda")
    up[at, at] = 1.0
    up[at[1:], parent[1:]] = 1.0
    for _ in range(max(1, n - 1).bit_length()):
        up = (up @ up).clamp_(max=1.0)
    mask = up > 0.5
    return mask.sum(1) - 1, mask


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    b, n, hkv, d, dt = case["b"], case["n"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    lens, counts = _lens(b, case["ctx"]), _counts(b, n)
    k_cache, v_cache, table = _cache(case, g, [s + n for s in lens])
    s = dict(case=case, k_cache=k_cache, v_cache=v_cache, table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    if case["op"] == "keep":
        # node 0 is the token that was drawn before; a path goes on to ever later nodes
        s["kept"] = torch.tensor([1 + i % case["most"] for i in range(b)], dtype=torch.int32, device="cuda")
        rest = torch.rand(b, n, generator=g, device="cuda")
        rest[:, 0] = -1.0
        s["path"] = rest.argsort(1)[:, :case["most"]].sort(1).values.to(torch.int32)
        return s
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    s["q"] = randn(b, n, case["g"] * hkv, d)
    depth = mask = None
    if case["tree"]:
        depth, mask = _tree(n, g)
    s["mask"] = mask
    if case["op"] == "append":
        # all three are parts of one projection's output, as a model has them
        qkv = randn(b, n, (case["g"] + 2) * hkv, d)
        s["q"], s["k"], s["v"] = qkv.split([case["g"] * hkv, hkv, hkv], dim=2)
        at = depth if depth is not None else torch.arange(n, device="cuda")
        s["positions"] = (s["lens"][:, None] + at + case["far"]).to(torch.int32)
        rot = case["rot"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float() if rot else None
    return s


# -- the plain forms --------------------------------------------------------------------------

def _rotated(x, cos, sin, pairs):
    """x [b, n, h, d] in 32 bits with its first entries rotated by cos, sin [b, n, rot / 2]."""
    if cos is None:
        return x.float()
    half = cos.shape[-1]
    xf, cos, sin = x.float(), cos[:, :, None], sin[:, :, None]
    if pairs:
        first, second = xf[..., 0:2 * half:2], xf[..., 1:2 * half:2]
        turned = torch.stack([first * cos - second * sin, second * cos + first * sin], -1).flatten(-2)
    else:
        first, second = xf[..., :half], xf[..., half:2 * half]
        turned = torch.cat([first * cos - second * sin, second * cos + first * sin], -1)
    return torch.cat([turned, xf[..., 2 * half:]], -1)


def _place(table, slots, page):
    """Page and slot in it of each sequence's slots [b, m]."""
    return table.gather(1, slots // page).long(), slots % page


def _plain_append(s):
    case, n = s["case"], s["case"]["n"]
    cos = sin = None
    if s["inv_freq"] is not None:
        angle = s["positions"].double()[..., None] * s["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
    at = torch.arange(n, device="cuda")
    valid = at < s["counts"][:, None]
    page, slot = _place(s["table"], s["lens"].long()[:, None] + at, case["page"])
    page, slot = page[valid], slot[valid]
    s["k_cache"][page, slot] = _rotated(s["k"], cos, sin, case["pairs"]).to(s["k"].dtype)[valid]
    s["v_cache"][page, slot] = s["v"][valid]
    q = torch.where(valid[..., None, None], _rotated(s["q"], cos, sin, case["pairs"]), 0.0).to(s["q"].dtype)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case = s["case"]
    b, n, hkv, g, d = case["b"], case["n"], case["hkv"], case["g"], case["d"]
    slots = s["table"].shape[1] * case["page"]
    k = s["k_cache"][s["table"].long()].reshape(b, slots, hkv, d).float().permute(0, 2, 3, 1)
    q = s["q"].float().reshape(b, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * g, d)
    scores = (q @ k) * d ** -0.5
    node = torch.arange(slots, device="cuda") - s["lens"][:, None]                   # of each slot: < 0 context
    inside = (node >= 0) & (node < s["counts"][:, None])
    tree = s["mask"] if s["mask"] is not None else torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    seen = (node < 0)[:, None] | (inside[:, None] & tree[:, node.clamp(0, n - 1)].permute(1, 0, 2))
    seen &= (torch.arange(n, device="cuda") < s["counts"][:, None])[..., None]       # [b, n, slots]
    seen = seen[:, None, :, None].expand(b, 1, n, g, slots).reshape(b, 1, n * g, slots)
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    mass = p.sum(-1, keepdim=True)
    v = s["v_cache"][s["table"].long()].reshape(b, slots, hkv, d).float().permute(0, 2, 1, 3)
    o = (p @ v) / torch.where(mass > 0, mass, 1.0)
    lse = (top + torch.log(mass))[..., 0]
    o = o.reshape(b, hkv, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, hkv * g, d)
    return {"out": o.to(s["q"].dtype), "lse": lse.reshape(b, hkv, n, g).permute(0, 2, 1, 3).reshape(b, n, hkv * g)}


def _plain_keep(s):
    case = s["case"]
    at = torch.arange(case["most"], device="cuda")
    valid = at < s["kept"][:, None]
    start = s["lens"].long()[:, None]
    source, target = (_place(s["table"], start + x, case["page"]) for x in (s["path"].long(), at.expand_as(valid)))
    for cache in (s["k_cache"], s["v_cache"]):
        cache[target[0][valid], target[1][valid]] = cache[source[0][valid], source[1][valid]]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain(s):
    return {"append": _plain_append, "attend": _plain_attend, "keep": _plain_keep}[s["case"]["op"]](s)


# -- the library's calls ----------------------------------------------------------------------

def _own(s):
    from rl_infra_gb300 import ops
    case = s["case"]
    if case["op"] == "append":
        got = ops.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], q=s["q"],
                               positions=s["positions"], counts=s["counts"], inv_freq=s["inv_freq"],
                               interleaved=case["pairs"])
        return {"q": got["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "attend":
        return ops.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], mask=s["mask"],
                                  counts=s["counts"])
    ops.cache_keep(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["path"], s["kept"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    return _own(state) if own else _plain(state)


# -- the definitions in 64 bits ---------------------------------------------------------------

def _exact_append(s):
    case = s["case"]
    k_out, v_out, q_out = s["k_cache"].double(), s["v_cache"].double(), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    table, page = s["table"].tolist(), case["page"]
    half = case["rot"] // 2
    for i, (start, count) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
        if count == 0:
            continue
        where = torch.arange(start, start + count, device="cuda")
        cells = torch.tensor(table[i], device="cuda")[where // page] * page + where % page

        def turn(x):
            x = x[i, :count].double().clone()
            if half:
                phase = torch.outer(s["positions"][i, :count].double(), s["inv_freq"].double())[:, None]
                one = slice(0, 2 * half, 2) if case["pairs"] else slice(0, half)
                two = slice(1, 2 * half, 2) if case["pairs"] else slice(half, 2 * half)
                z = torch.polar(torch.ones_like(phase), phase) * torch.complex(x[..., one], x[..., two])
                x[..., one], x[..., two] = z.real, z.imag
            return x

        k_out.view(-1, case["hkv"], case["d"])[cells] = turn(s["k"])
        v_out.view(-1, case["hkv"], case["d"])[cells] = s["v"][i, :count].double()
        q_out[i, :count] = turn(s["q"])
    return {"q": q_out, "k_cache": k_out, "v_cache": v_out}


def _exact_attend(s):
    case = s["case"]
    n, hkv, g, d = case["n"], case["hkv"], case["g"], case["d"]
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for i, (length, count) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
        total = length + count
        pages = s["table"][i, :-(-total // case["page"])].long()
        keys = s["k_cache"][pages].flatten(0, 1)[:total]
        values = s["v_cache"][pages].flatten(0, 1)[:total]
        tree = torch.zeros(count, total, dtype=torch.bool, device="cuda")
        tree[:, :length] = True
        if s["mask"] is None:
            tree[:, length:] = torch.arange(count, device="cuda")[None] <= torch.arange(count, device="cuda")[:, None]
        else:
            tree[:, length:] = s["mask"][:count, :count]
        for h in range(hkv):
            heads = slice(h * g, (h + 1) * g)
            logits = torch.einsum("nge,te->ngt", s["q"][i, :count, heads].double(), keys[:, h].double()) / math.sqrt(d)
            logits.masked_fill_(~tree[:, None], -math.inf)
            norm = torch.logsumexp(logits, -1)
            lse[i, :count, heads] = norm
            out[i, :count, heads] = torch.einsum("ngt,te->nge", torch.exp(logits - norm[..., None]), values[:, h].double())
    return {"out": out, "lse": lse}


def _exact_keep(s):
    page, out = s["case"]["page"], {}
    table, path = s["table"].long(), s["path"].tolist()
    lens, kept = s["lens"].tolist(), s["kept"].tolist()
    source = [(i, lens[i] + path[i][j]) for i in range(len(kept)) for j in range(kept[i])]
    target = [(i, lens[i] + j) for i in range(len(kept)) for j in range(kept[i])]

    def cells(places):
        row, slot = torch.tensor(places, device="cuda").unbind(1)
        return table[row, slot // page] * page + slot % page

    for name in ("k_cache", "v_cache"):
        flat = s[name].double().flatten(0, 1)
        out[name] = flat.index_copy(0, cells(target), flat[cells(source)]).reshape(s[name].shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "keep": _exact_keep}[case["op"]](s)
