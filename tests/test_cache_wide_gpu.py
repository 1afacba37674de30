"""Attention over a paged cache where a head of keys has many rows: the kernel on the tensor cores' own
instruction, and the one with few rows at its borders."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from rl_infra_gb300 import build, capi, ops  # noqa: E402
from tests import cache_oracle as co  # noqa: E402
from tests.ops_oracle import TINY, close  # noqa: E402
from tests.test_cache_gpu import INF, NAN, TYPES, attend_case, cache, check_attend, fill, host, i32, rand, tree  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n, g", [(33, 1), (8, 8), (64, 2), (43, 3), (64, 3), (32, 8), (129, 2), (64, 8), (20, 25)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[0, 100], [127, 300], [1]])
def test_rows(kind, n, g, d, lens):
    """Every number of row tiles and of key tiles in a part, odd and even."""
    attend_case(31, kind, len(lens), n, 1, g, d, 16, lens, masks="tree")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [8, 40, 72, 80, 104, 120, 192, 33])
@pytest.mark.parametrize("n, page", [(35, 64), (70, 24)])
def test_odd_heads(kind, d, n, page):
    attend_case(32, kind, 2, n, 2, 2, d, page, [200, 33], masks="each")


@pytest.mark.parametrize("page", [1, 2, 5, 12, 48, 128, 256, 300])
@pytest.mark.parametrize("n, g", [(5, 2), (40, 1), (100, 2)])
def test_pages(page, n, g):
    attend_case(33, "bf16", 2, n, 2, g, 128, page, [340, 129], masks="tree")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n, g", [(40, 1), (40, 6)])
@pytest.mark.parametrize("d", [64, 128])
def test_one_long_sequence(kind, n, g, d):
    attend_case(34, kind, 1, n, 1, g, d, 64, [20000], masks="tree")


@pytest.mark.parametrize("n, g", [(40, 1), (40, 5)])
def test_ragged(n, g):
    r = np.random.default_rng(35)
    lens, counts = r.integers(0, 700, 21), r.integers(0, n + 1, 21)
    lens[3], counts[3], counts[4], lens[5], counts[6] = 0, 0, 0, 0, 1
    attend_case(35, "bf16", 21, n, 2, g, 64, 16, lens, counts, "each")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [3.0, 0.0, -1.0])
def test_maxima_that_rise(kind, scale):
    """Scores that grow along the sequence, so that each tile raises the maximum; and scales that are not positive."""
    r = np.random.default_rng(36)
    kc, vc, table = cache(r, 1, 700, 16, 1, 64, kind)
    fill(r, kc, vc, table, [700], kind)
    tab = table.cpu().numpy()
    for s in range(700):
        p, x = co.place(tab[0], s, 16, kc.shape[0])
        kc[p, x] *= 0.002 * s
    q = rand(r, 1, 50, 4, 64, kind=kind)
    got = ops.tree_attention(q, kc, vc, table, i32([650]), scale=scale)
    check_attend(got, co.attend(host(q), host(kc), host(vc), tab, [650], scale=scale, kind=kind), kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d, n, g", [(64, 40, 1), (128, 20, 3), (128, 100, 2), (64, 60, 5), (128, 20, 2), (256, 40, 1)])
def test_masked_places_take_no_part(kind, d, n, g):
    r = np.random.default_rng(37)
    lens = [200, 0, 126]
    kc, vc, table = cache(r, 3, 320, 16, 1, d, kind)
    fill(r, kc, vc, table, [x + n for x in lens], kind)
    mask = np.stack([tree(r, n) for _ in range(3)])
    mask[:, :, 2] = False                      # nobody sees node 2
    mask[1, 4] = False                         # this row of the sequence without context sees nothing
    mask[:, :, 5] &= np.arange(n)[None] % 2 == 1
    tab = table.cpu().numpy()
    low = torch.finfo(TYPES[kind]).min
    for i, ln in enumerate(lens):
        p, s = co.place(tab[i], ln + 2, 16, kc.shape[0])
        kc[p, s], vc[p, s] = torch.tensor([NAN, INF, -INF, low] * (d // 4), device="cuda"), NAN
        vc[p, s, :, 1::2] = INF
        p, s = co.place(tab[i], ln + 5, 16, kc.shape[0])
        vc[p, s, :, 3], vc[p, s, :, 4], vc[p, s, :, 5] = INF, NAN, low / 4
    q = rand(r, 3, n, g, d, kind=kind)
    got = ops.tree_attention(q, kc, vc, table, i32(lens), mask=torch.from_numpy(mask).cuda())
    want = co.attend(host(q), host(kc), host(vc), tab, lens, mask, kind=kind)
    assert np.isnan(want["out"]).any() and np.isinf(want["out"]).any() and np.isinf(want["lse"]).any()
    check_attend(got, want, kind)
    # what is not finite was one call's: the next one, without it, has none
    for i, ln in enumerate(lens):
        p, s = co.place(tab[i], ln + 5, 16, kc.shape[0])
        vc[p, s] = 1.0
    assert torch.isfinite(ops.tree_attention(q, kc, vc, table, i32(lens), mask=torch.from_numpy(mask).cuda())["out"]).all()


@pytest.mark.parametrize("n, g", [(40, 1), (40, 6), (6, 2)])
def test_bad_pages(n, g):
    r = np.random.default_rng(38)
    kc, vc, table = cache(r, 2, 400, 16, 1, 64, "bf16")
    fill(r, kc, vc, table, [400, 400], "bf16")
    table[0, 1], table[0, 9], table[1, 0], table[1, 20] = -1, 1 << 30, -(1 << 31), kc.shape[0]
    q = rand(r, 2, n, g, 64, kind="bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.tree_attention(q, kc, vc, table, i32([330, 300]), status=status)
    check_attend(got, co.attend(host(q), host(kc), host(vc), table.cpu().numpy(), [330, 300], kind="bf16"), "bf16")
    assert status.item() == capi.PER_DEVFLAG_BAD_INDEX


def test_layouts_and_outputs():
    """Heads before slots; a cache that is part of a larger one; outputs and queries with gaps; nothing beside the
    rows is written."""
    r = np.random.default_rng(39)
    b, n, hkv, g, d, page = 2, 40, 2, 3, 64, 16
    kc, vc, table = cache(r, b, 400, page, hkv, d, "bf16")
    fill(r, kc, vc, table, [390, 200], "bf16")
    q = rand(r, b, n, hkv * g, d, kind="bf16")
    lens = i32([350, 160])
    want = ops.tree_attention(q, kc, vc, table, lens)
    k2 = kc.transpose(1, 2).contiguous().transpose(1, 2)                       # [pages, heads, slots, D]
    both = torch.stack([kc, vc], 1).contiguous()                               # [pages, 2, slots, heads, D]
    wide = torch.nn.functional.pad(q, (0, 24))[..., :d]
    store = torch.full((b, n, hkv * g, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    odd = torch.full((b, n, hkv * g, d + 1), 3.0, dtype=torch.bfloat16, device="cuda")
    for kk, vv, qq, out in ((k2, vc, q, None), (both[:, 0], both[:, 1], wide, store[..., :d]), (kc, vc, q, odd[..., :d])):
        got = ops.tree_attention(qq, kk, vv, table, lens, out=None if out is None else {"out": out})
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    assert (store[..., d:] == 3).all() and (odd[..., d:] == 3).all()


def test_many_calls_at_once():
    """Calls of every kernel under way on two streams give what they give alone."""
    r = np.random.default_rng(40)
    kc, vc, table = cache(r, 6, 900, 16, 2, 128, "bf16")
    fill(r, kc, vc, table, [900] * 6, "bf16")
    lens = i32([850, 100, 0, 613, 127, 128])
    qs = [rand(r, 6, n, 2 * g, 128, kind="bf16") for n, g in ((1, 4), (8, 4), (40, 1), (40, 4))]
    want = [ops.tree_attention(q, kc, vc, table, lens) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[ops.tree_attention(q, kc, vc, table, lens, stream=s) for q in qs] for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    for row in got:
        for x, y in zip(row, want):
            assert torch.equal(x["out"], y["out"]) and torch.equal(x["lse"], y["lse"])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n, g", [(1, 4), (4, 8), (16, 4), (40, 6)])
@pytest.mark.parametrize("b", [1, 3, 40, 150])
def test_room_for_more(kind, n, g, b):
    """Short sequences of every number of tiles, in a table just wide enough and in one with room for long ones: other
    cuts of the work, the same results to the last roundings."""
    r = np.random.default_rng(41)
    lens, counts = r.integers(0, 500, b), r.integers(0, n + 1, b)
    lens[0], counts[0] = 499, n
    kc, vc, table = cache(r, b, 500 + n, 16, 2, 64, kind)
    fill(r, kc, vc, table, lens + counts, kind)
    q = rand(r, b, n, 2 * g, 64, kind=kind)
    wide = torch.nn.functional.pad(table, (0, 5000), value=-1)
    one = ops.tree_attention(q, kc, vc, table, i32(lens), counts=i32(counts))
    two = ops.tree_attention(q, kc, vc, wide, i32(lens), counts=i32(counts))
    some = min(b, 4)
    want = co.attend(host(q[:some]), host(kc), host(vc), table.cpu().numpy(), lens[:some], None, counts[:some], kind=kind)
    for got in (one, two):
        check_attend({k: t[:some] for k, t in got.items()}, want, kind)
    torch.testing.assert_close(one["out"], two["out"], rtol=2e-2 if kind == "bf16" else 1e-4, atol=1e-2 if kind == "bf16" else 1e-5)
    torch.testing.assert_close(one["lse"], two["lse"], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("kind, n, g", [("f32", 4, 2), ("bf16", 4, 2), ("f16", 40, 2), ("bf16", 100, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_nodes_behind_the_tables_end(kind, n, g, masked):
    """Nodes that the table has no slot for are seen by nobody; they themselves see what is there."""
    r = np.random.default_rng(42)
    kc, vc, table = cache(r, 2, 112, 16, 1, 64, kind)
    fill(r, kc, vc, table, [112, 112], kind)
    lens = [112 - n // 2, 112]
    q = rand(r, 2, n, g, 64, kind=kind)
    mask = np.ones((n, n), bool) if masked else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.tree_attention(q, kc, vc, table, i32(lens), mask=torch.from_numpy(mask).cuda() if masked else None, status=status)
    check_attend(got, co.attend(host(q), host(kc), host(vc), table.cpu().numpy(), lens, mask, kind=kind), kind)
    assert status.item() == capi.PER_DEVFLAG_BAD_INDEX


@pytest.mark.parametrize("kind, n, g, d", [("bf16", 1024, 2, 64), ("f32", 300, 1, 32), ("f16", 1024, 1, 256)])
def test_the_most_nodes(kind, n, g, d):
    attend_case(43, kind, 1, n, 1, g, d, 64, [100], masks="tree" if n < 1024 else None)


def test_a_first_call_can_be_captured():
    """In a new process, whose first call of each kernel is under capture."""
    code = """
import torch
from rl_infra_gb300 import ops
kc = torch.randn(40, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
vc, table = torch.randn_like(kc), torch.arange(40, device="cuda", dtype=torch.int32)[None]
lens = torch.tensor([500], device="cuda", dtype=torch.int32)
qs = [torch.randn(1, n, 2 * g, 64, device="cuda", dtype=torch.bfloat16) for n, g in ((1, 4), (9, 2), (60, 2))]
new = torch.randn(1, 60, 2, 64, device="cuda", dtype=torch.bfloat16)
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=side):
    ops.cache_append(new, new, kc, vc, table, lens)
    got = [ops.tree_attention(q, kc, vc, table, lens) for q in qs]
    ops.cache_keep(kc, vc, table, lens, lens[None], torch.zeros_like(lens))
graph.replay()
torch.cuda.synchronize()
for q, x in zip(qs, got):
    assert torch.equal(x["out"], ops.tree_attention(q, kc, vc, table, lens)["out"])
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n, g", [(40, 1), (40, 5)])
def test_scores_of_minus_infinity(kind, n, g):
    """Whole tiles of keys that score -inf, first, in between and last; then nothing else."""
    r = np.random.default_rng(44)
    kc, vc, table = cache(r, 1, 700, 16, 1, 64, kind)
    fill(r, kc, vc, table, [700], kind)
    tab = table.cpu().numpy()
    for s in [*range(0, 260), *range(400, 520), *range(530, 640, 3)]:
        kc[co.place(tab[0], s, 16, kc.shape[0])] = -INF
    q = rand(r, 1, n, g, 64, kind=kind).abs()
    got = ops.tree_attention(q, kc, vc, table, i32([650]))
    check_attend(got, co.attend(host(q), host(kc), host(vc), tab, [650], kind=kind), kind)
    kc.fill_(-INF)
    got = ops.tree_attention(q, kc, vc, table, i32([650]))
    assert (got["out"] == 0).all() and (got["lse"] == -INF).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n, g, d", [(1, 4, 64), (6, 4, 64), (12, 4, 128), (40, 1, 64), (20, 5, 128), (40, 4, 64), (40, 5, 128), (3, 2, 256),
                                     (9, 5, 33)])
@pytest.mark.parametrize("nats, ctx", [(14, 8000), (16, 8000), (17.5, 8000), (18, 30000), (19, 8000)])
def test_one_key_far_above_the_others(kind, n, g, d, nats, ctx):
    """A key that takes nearly all of the mass and whose value is 0, first or last: the output is what the many others
    have left, each of them w = exp(-nats) of the maximum.  All scores are exact, so that out is sum(v) over
    exp(nats) + the others: off by out's rounding and p's (half a step each), and 2^-12 for the references and sums.  A
    float16 below 2^-14 is off by 2^-25: p is w 2^15 where a head of keys has few rows, and at least w 2^11.5 on the tensor
    cores' own instruction."""
    r = np.random.default_rng(45)
    kc, vc, table = cache(r, 1, ctx + n, 16, 1, d, kind)
    kc.zero_()
    vc.copy_((rand(r, *vc.shape, kind="f32").abs() * 100 + 1).to(TYPES[kind]))
    q = torch.zeros(1, n, g, d, dtype=TYPES[kind], device="cuda")
    q[..., 0] = 1
    tab = table.cpu().numpy()
    mask = torch.zeros(n, n, dtype=torch.bool, device="cuda")
    for at in (0, ctx - 1):
        top = co.place(tab[0], at, 16, kc.shape[0])
        keep = kc[top].clone(), vc[top].clone()
        kc[top[0], top[1], 0, 0], vc[top] = nats, 0
        got = ops.tree_attention(q, kc, vc, table, i32([ctx]), mask=mask, scale=1.0)
        values = host(vc[table[0].long()].reshape(-1, d)[:ctx])
        want = values.sum(0) / (np.exp(nats) + ctx - 1)
        half = torch.finfo(TYPES[kind]).eps / 2
        err = np.abs(host(got["out"]) - want) / want
        rounds = half if kind == "bf16" else max(half, 2.0 ** -25 / (np.exp(-nats) * 2 ** (11.5 if n * g > 32 and d <= 128 else 15)))
        assert err.max() <= half + rounds + 2.0 ** -12, err.max()
        np.testing.assert_allclose(host(got["lse"]), np.log(np.exp(nats) + ctx - 1), rtol=1e-5)
        kc[top], vc[top] = keep


@pytest.mark.parametrize("kind, big", [("bf16", 6e4), ("bf16", 1e9), ("bf16", 1e18), ("f16", 6e4), ("f16", 2e3)])
@pytest.mark.parametrize("n, g, d", [(3, 4, 64), (40, 1, 64), (40, 1, 128), (40, 5, 128), (70, 2, 64)])
@pytest.mark.parametrize("steps", [(1.0, 1.0, 1.0), (1e-6, 1.0, 3.0), (1.0, 1e-3, 1e-7)])
def test_large_scores(kind, big, n, g, d, steps):
    """Scores of up to 2^30 and past it, in stretches of keys of different size (references that go far at once, later,
    or twice): a row whose first score is ahead of the second by far more than binary32's noise gives that key's value,
    off by half a step of the type for its p (2^x for any x, over a sum that is not rounded) and half a step for out."""
    r = np.random.default_rng(46)
    half = torch.finfo(TYPES[kind]).eps / 2
    ctx = 900
    kc, vc, table = cache(r, 1, ctx + n, 16, 1, d, kind)
    fill(r, kc, vc, table, [ctx + n], kind)
    kc.copy_((r.uniform() + rand(r, *kc.shape, kind="f32").clamp(-4, 4)) * big / 5)
    tab = table.cpu().numpy()
    for s in range(ctx + n):
        p, x = co.place(tab[0], s, 16, kc.shape[0])
        kc[p, x] *= steps[min(s // 300, 2)] / max(steps)
    q = (rand(r, 1, n, g, d, kind="f32").clamp(-4, 4) * big / 5).to(TYPES[kind])
    got = ops.tree_attention(q, kc, vc, table, i32([ctx]))
    keys, values = (host(t[table[0].long()].reshape(-1, d)) for t in (kc, vc))
    out, lse, sure = host(got["out"]), host(got["lse"]), 0
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for i in range(n):
        x, y = keys[:ctx + i + 1], values[:ctx + i + 1]
        for h in range(g):
            s = x @ host(q)[0, i, h] * d ** -0.5
            noise = 2.0 ** -23 * (d + 8) * (np.abs(x) @ np.abs(host(q)[0, i, h])).max() * d ** -0.5
            first, second = np.argmax(s), np.partition(s, -2)[-2]
            assert abs(lse[0, i, h] - s[first]) <= noise + 8
            if s[first] - second > 2 * noise + 30:
                sure += 1
                np.testing.assert_allclose(out[0, i, h], y[first], rtol=2.01 * half, atol=TINY[kind])
    assert sure > n * g // 2


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n, g, d", [(40, 1, 64), (20, 4, 128), (40, 5, 64), (40, 4, 128)])
@pytest.mark.parametrize("far", [1, -1])
@pytest.mark.parametrize("ctx", [700, 80])
def test_scores_far_from_zero(kind, n, g, d, far, ctx):
    """Scores of far 2^23 + j and small j, which binary32 holds, as 2^30 + 128 j times a scale of 2^-7: a softmax of j alone.
    p and out are off by half a step of the type each, 2^-12 for sums (no j is 16 below the maximum).  A sequence of more than
    one tile is joined from parts whose references, in log2, are binary32: steps of 1 there, each off by up to a half, so that a
    part's weight is off by a factor f of 2^-0.5 to 2^0.5, and sum(w f v) / sum(w f) from its value without f by up to
    max(f) / min(f) = 2 times the weighted mean of |v - value|."""
    r = np.random.default_rng(47)
    kc, vc, table = cache(r, 1, ctx + n, 16, 1, d, kind)
    vc.copy_(rand(r, *vc.shape, kind="f32").abs() + 1)
    kc.zero_()
    j = torch.from_numpy(r.integers(0, 8, kc.shape[:3]).astype(np.float32)).cuda()
    tab = table.cpu().numpy()
    for s in range(ctx):                       # maxima that rise from tile to tile
        p, x = co.place(tab[0], s, 16, kc.shape[0])
        j[p, x] += s // 90
    kc[..., 0], kc[..., 1] = 2.0 ** 15, j
    q = torch.zeros(1, n, g, d, dtype=TYPES[kind], device="cuda")
    q[..., 0], q[..., 1] = far * 2.0 ** 15, 128
    mask = torch.zeros(n, n, dtype=torch.bool, device="cuda")
    got = ops.tree_attention(q, kc, vc, table, i32([ctx]), mask=mask, scale=2.0 ** -7)
    line = lambda t: host(t[table[0].long()]).reshape(-1, *t.shape[3:])[:ctx]
    p = np.exp(line(j) - line(j).max())
    want = p / p.sum() @ line(vc)
    half = torch.finfo(TYPES[kind]).eps / 2
    joins = 2 * (p / p.sum() @ np.abs(line(vc) - want)) / want if ctx + n > 128 else 0
    err = np.abs(host(got["out"]) - want) / want
    assert (err <= 2 * half + 2.0 ** -12 + joins).all(), err.max()
    np.testing.assert_allclose(host(got["lse"]), far * 2.0 ** 23 + np.log(p.sum()) + line(j).max(), atol=2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n, g, d, page", [(1, 4, 64, 16), (2, 3, 128, 16), (7, 2, 96, 8), (9, 2, 256, 16), (20, 2, 80, 16), (12, 8, 128, 16),
                                           (5, 2, 33, 7), (40, 2, 130, 3)])
def test_infinite_entries(kind, n, g, d, page):
    """Keys with infinite entries score -inf, inf or NaN by their signs and the query's, in every type; so do queries with
    infinite entries.  Where nothing scores inf or NaN, a row gives what the other keys give."""
    r = np.random.default_rng(48)
    ctx = 300
    kc, vc, table = cache(r, 1, ctx + n, page, 1, d, kind)
    fill(r, kc, vc, table, [ctx + n], kind)
    tab = table.cpu().numpy()
    q = rand(r, 1, n, g, d, kind=kind)
    q[..., :3] = q[..., :3].abs() + 0.01
    q[0, n - 1, 0, 1] = -1.0                   # this row scores inf somewhere
    gone = [0, 5, 6, 77, 130, 131, 200, ctx - 1, ctx]      # the last is node 0's
    for s in gone:
        kc[co.place(tab[0], s, page, kc.shape[0])][..., 1] = -INF
    kc[co.place(tab[0], 6, page, kc.shape[0])][..., 2] = -INF
    kc[co.place(tab[0], 200, page, kc.shape[0])][..., 0] = -INF
    got = {name: host(t) for name, t in ops.tree_attention(q, kc, vc, table, i32([ctx])).items()}
    assert np.isnan(got["out"][0, n - 1, 0]).all() and np.isnan(got["lse"][0, n - 1, 0])
    # the same without those keys: pages of one slot, and node 0 seen by nobody
    left = np.setdiff1d(np.arange(ctx + n), gone[:-1])
    line = [host(t[table[0].long()]).reshape(-1, 1, 1, d)[left] for t in (kc, vc)]
    line[0][~np.isfinite(line[0])] = 0
    mask = np.tri(n, dtype=bool)
    mask[:, 0] = False
    qs = host(q)
    qs[0, n - 1, 0] = 0
    want = co.attend(qs, *line, np.arange(len(left))[None], [ctx - len(gone) + 1], mask, kind=kind)
    for name in ("out", "lse"):
        got[name][0, n - 1, 0] = want[name][0, n - 1, 0]
    close(got["out"], want["out"], want["bout"], kind)
    close(got["lse"], want["lse"], want["blse"])
    # an infinite query: every score of its row is inf, -inf or NaN
    fill(r, kc, vc, table, [ctx + n], kind)
    q = rand(r, 1, n, g, d, kind=kind).abs()
    kc.abs_().neg_()
    q[0, 0, 0, 0] = INF
    got = ops.tree_attention(q, kc, vc, table, i32([ctx]))
    assert (got["out"][0, 0, 0] == 0).all() and got["lse"][0, 0, 0] == -INF
    assert torch.isfinite(got["out"]).all() and torch.isfinite(got["lse"].flatten()[1:]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("b, n, g, d, page, ctx", [(3, 1, 4, 128, 16, 1000), (1, 4, 4, 64, 16, 9000), (2, 3, 1, 256, 8, 700), (1, 16, 1, 40, 16, 130)])
def test_few_rows_keep_p_in_two_parts(kind, b, n, g, d, page, ctx):
    """Up to 16 rows: out is off by its own rounding, binary32's and what two roundings leave of p (half a step squared)."""
    r = np.random.default_rng(49)
    kc, vc, table = cache(r, b, ctx + n, page, 2, d, kind)
    fill(r, kc, vc, table, [ctx + n] * b, kind)
    q, lens = rand(r, b, n, 2 * g, d, kind=kind), np.full(b, ctx)
    got = ops.tree_attention(q, kc, vc, table, i32(lens))
    args = host(q), host(kc)
    tab = table.cpu().numpy()
    want = co.attend(*args, host(vc), tab, lens, kind="f32")
    size = co.attend(*args, np.abs(host(vc)), tab, lens, kind="f32")["out"]
    close(host(got["out"]), want["out"], want["bout"] + size * (torch.finfo(TYPES[kind]).eps / 2) ** 2, kind)
