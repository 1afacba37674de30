"""The paged cache's operators against their definitions in 64 bits (tests/cache_oracle.py), element by
element, at the sizes, masks and layouts where they can go wrong."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from rl_infra_gb300 import build, capi, ops  # noqa: E402
from tests import cache_oracle as co  # noqa: E402
from tests.ops_oracle import close  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


def host(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rand(g, *shape, kind="f32", scale=1.0):
    return torch.from_numpy((g.normal(size=shape) * scale).astype(np.float32)).cuda().to(TYPES[kind])


def cache(g, b, room, page, hkv, d, kind, spare=3, stale=NAN):
    """Caches of stale slots, and a table of scattered pages for `room` slots a sequence."""
    width = -(-room // page)
    pages = b * width + spare
    k = torch.full((pages, page, hkv, d), stale, dtype=TYPES[kind], device="cuda")
    return k, k.clone(), i32(g.permutation(pages)[:b * width].reshape(b, width))


def fill(g, kc, vc, table, totals, kind):
    """Random entries in each sequence's first totals[i] slots."""
    page = kc.shape[1]
    for i, n in enumerate(totals):
        at = np.arange(n)
        p = torch.from_numpy(table[i].cpu().numpy()[at // page].astype(np.int64)).cuda()
        s = torch.from_numpy(at % page).cuda()
        kc[p, s] = rand(g, n, *kc.shape[2:], kind=kind)
        vc[p, s] = rand(g, n, *kc.shape[2:], kind=kind)


def tree(g, n):
    mask = np.zeros((n, n), bool)
    for i in range(n):
        if i:
            mask[i] = mask[g.integers(0, i)]
        mask[i, i] = True
    return mask


def check_attend(got, want, kind):
    close(host(got["out"]), want["out"], want["bout"], kind)
    close(host(got["lse"]), want["lse"], want["blse"])


def attend_case(seed, kind, b, n, hkv, g, d, page, lens, counts=None, masks=None, **kw):
    r = np.random.default_rng(seed)
    lens = np.asarray(lens)
    totals = lens + (n if counts is None else np.asarray(counts))
    kc, vc, table = cache(r, b, int(max(totals.max(), 1)), page, hkv, d, kind)
    fill(r, kc, vc, table, totals, kind)
    q = rand(r, b, n, hkv * g, d, kind=kind)
    mask = {None: None, "tree": tree(r, n), "each": np.stack([tree(r, n) for _ in range(b)])}[masks]
    got = ops.tree_attention(q, kc, vc, table, i32(lens), mask=None if mask is None else torch.from_numpy(mask).cuda(),
                             counts=None if counts is None else i32(counts), **kw)
    want = co.attend(host(q), host(kc), host(vc), table.cpu().numpy(), lens, mask, counts, kind=kind, **kw)
    check_attend(got, want, kind)
    return got


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b, n, hkv, g, d, page, lens, masks", [
    (1, 1, 1, 1, 64, 16, [0], None),                    # a sequence's first token
    (1, 1, 2, 4, 128, 16, [1], None),
    (3, 1, 2, 4, 128, 16, [63, 64, 65], None),          # around a tile
    (2, 5, 2, 3, 64, 24, [100, 7], "tree"),             # 15 rows; pages that end inside a tile
    (2, 8, 1, 4, 128, 8, [130, 0], "each"),             # 32 rows
    (2, 11, 3, 2, 80, 16, [200, 31], "tree"),
    (1, 24, 1, 4, 128, 64, [300], "tree"),              # 96 rows
    (2, 70, 1, 2, 64, 32, [5, 129], "tree"),            # nodes over two tiles
    (2, 33, 2, 5, 96, 16, [64, 1], None),
    (1, 9, 1, 1, 256, 16, [150], "tree"),
    (2, 40, 1, 2, 256, 5, [33, 90], "each"),
    (1, 3, 2, 2, 32, 1, [77], None),                    # pages of one slot
    (1, 16, 1, 8, 72, 128, [500], "tree"),              # 128 rows
    (1, 40, 1, 8, 128, 64, [700], "tree"),              # 320 rows
    (2, 5, 2, 2, 33, 7, [45, 12], "tree"),              # heads off every boundary
    (1, 2, 1, 1, 1, 3, [10], None),
    (2, 7, 1, 3, 255, 16, [70, 3], None),
])
def test_attention(kind, b, n, hkv, g, d, page, lens, masks):
    attend_case(1, kind, b, n, hkv, g, d, page, lens, masks=masks)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n, g", [(1, 1), (6, 5), (12, 8)])
def test_one_long_sequence_is_joined_from_many_parts(kind, n, g):
    attend_case(2, kind, 1, n, 1, g, 64, 16, [20011], masks="tree" if n > 1 else None)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ragged_batch(kind):
    r = np.random.default_rng(3)
    lens, counts = r.integers(0, 400, 37), r.integers(0, 7, 37)
    lens[5], counts[5], counts[6], lens[7] = 0, 0, 0, 0
    attend_case(3, kind, 37, 6, 2, 2, 64, 16, lens, counts, "each")


def test_more_sequences_than_threads():
    r = np.random.default_rng(4)
    attend_case(4, "f16", 300, 2, 1, 2, 32, 8, r.integers(0, 40, 300), r.integers(0, 3, 300))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
def test_scales(scale):
    attend_case(5, "f16", 2, 4, 1, 2, 64, 16, [90, 20], scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 40])
def test_masked_places_take_no_part(kind, d):
    """A node that others do not see holds infinities and NaN; a row that sees nothing gives 0."""
    r = np.random.default_rng(6)
    n, g, lens = 6, 3, [70, 0, 3]
    kc, vc, table = cache(r, 3, 80, 16, 1, d, kind)
    fill(r, kc, vc, table, [76, 6, 9], kind)
    mask = np.stack([tree(r, n) for _ in range(3)])
    mask[:, :, 2] = False                      # nobody sees node 2, not even itself
    mask[1, 4] = False                         # this row of the sequence without context sees nothing
    mask[2, 1, :] = False
    mask[:, 3, 5] = True                       # and node 5's infinity goes to rows 3 and 5 only
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
    assert (host(got["out"])[1, 4] == 0).all()


def test_scores_of_minus_infinity():
    r = np.random.default_rng(7)
    kc, vc, table = cache(r, 1, 20, 4, 1, 16, "bf16")
    fill(r, kc, vc, table, [20], "bf16")
    q = rand(r, 1, 2, 1, 16, kind="bf16").abs()
    tab = table.cpu().numpy()
    for s in range(0, 18, 2):
        kc[co.place(tab[0], s, 4, kc.shape[0])] = -INF
    check_attend(ops.tree_attention(q, kc, vc, table, i32([18])),
                 co.attend(host(q), host(kc), host(vc), tab, [18], kind="bf16"), "bf16")
    kc.fill_(-INF)
    got = ops.tree_attention(q, kc, vc, table, i32([18]))
    assert (got["out"] == 0).all() and (got["lse"] == -INF).all()


@pytest.mark.parametrize("kind, lead, pad", [("bf16", 0, 8), ("bf16", 1, 0), ("f16", 3, 5), ("f32", 2, 3), ("f32", 0, 4)])
def test_strides_and_alignment(kind, lead, pad):
    """Heads before slots, gaps between rows, tensors that begin off a boundary."""
    r = np.random.default_rng(8)
    b, n, hkv, g, d, page = 2, 5, 2, 3, 64, 8
    kc, vc, table = cache(r, b, 60, page, hkv, d, kind)
    fill(r, kc, vc, table, [55, 30], kind)
    q = rand(r, b, n, hkv * g, d, kind=kind)

    def moved(t, order):
        """The same values in another nesting of the axes, rows `pad` apart, `lead` from a boundary."""
        t = t.permute(order)
        store = torch.full((lead + t.numel() // d * (d + pad),), 3.0, dtype=t.dtype, device="cuda")
        view = store[lead:].view(*t.shape[:3], d + pad)[..., :d]
        view.copy_(t)
        back = [order.index(i) for i in range(4)]
        return view.permute(back), store

    (k2, _), (v2, _), (q2, _) = moved(kc, [0, 2, 1, 3]), moved(vc, [2, 0, 1, 3]), moved(q, [1, 0, 2, 3])
    table2 = torch.nn.functional.pad(table, (0, 3), value=99)[:, :table.shape[1]]
    out, store = moved(torch.zeros_like(q), [2, 1, 0, 3])
    mask = torch.from_numpy(tree(r, n)).cuda()
    got = ops.tree_attention(q2, k2, v2, table2, i32([50, 25]), mask=mask, out={"out": out})
    assert got["out"] is out
    want = co.attend(host(q), host(kc), host(vc), table.cpu().numpy(), [50, 25], mask.cpu().numpy(), kind=kind)
    check_attend(got, want, kind)
    gaps = store[lead:].view(-1, d + pad)[:, d:]
    assert (gaps == 3).all() and (store[:lead] == 3).all()


def test_a_result_does_not_depend_on_where_pages_lie():
    r = np.random.default_rng(9)
    kc, vc, table = cache(r, 4, 300, 16, 2, 128, "bf16")
    fill(r, kc, vc, table, [300] * 4, "bf16")
    q = rand(r, 4, 8, 8, 128, kind="bf16")
    lens = i32([290, 100, 0, 250])
    one = ops.tree_attention(q, kc, vc, table, lens)
    turn = torch.from_numpy(r.permutation(kc.shape[0])).cuda()
    two = ops.tree_attention(q, kc[turn], vc[turn], torch.argsort(turn)[table.long()].int(), lens)
    again = ops.tree_attention(q, kc, vc, table, lens)
    for name in ("out", "lse"):
        assert torch.equal(one[name], two[name]) and torch.equal(one[name], again[name])


def test_bad_pages_and_lengths_are_left_out():
    r = np.random.default_rng(10)
    kc, vc, table = cache(r, 5, 100, 16, 1, 64, "f32")
    fill(r, kc, vc, table, [100] * 5, "f32")
    table[0, 1], table[1, 0], table[1, 6] = -1, 1 << 20, -7
    lens, counts = [90, 95, -3, 111, 40], [3, 3, 2, 3, 9]      # seven pages hold 112 slots
    q = rand(r, 5, 4, 2, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.tree_attention(q, kc, vc, table, i32(lens), counts=i32(counts), status=status)
    want = co.attend(host(q), host(kc), host(vc), table.cpu().numpy(), lens, None, counts)
    check_attend(got, want, "f32")
    assert want["flag"] and status.item() == capi.PER_DEVFLAG_BAD_INDEX
    status.zero_()
    ops.tree_attention(q[4:], kc, vc, table[4:], i32([40]), status=status)
    assert status.item() == 0


def test_empty_calls():
    kc = torch.zeros(0, 16, 2, 64, device="cuda")
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    got = ops.tree_attention(torch.ones(2, 3, 4, 64, device="cuda"), kc, kc, table, i32([0, 0]), counts=i32([0, 0]))
    assert (got["out"] == 0).all() and (got["lse"] == -INF).all()
    assert ops.tree_attention(torch.ones(0, 3, 4, 64, device="cuda"), kc, kc, table[:0], i32([]))["out"].shape == (0, 3, 4, 64)
    assert ops.tree_attention(torch.ones(2, 0, 4, 64, device="cuda"), kc, kc, table, i32([0, 0]))["lse"].shape == (2, 0, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.ones(2, 1, 2, 64, device="cuda")
    ops.cache_append(new, new, kc, kc, table, i32([0, 0]), status=status)
    assert status.item() == capi.PER_DEVFLAG_BAD_INDEX      # there is no page
    ops.cache_append(new[:, :0], new[:, :0], kc, kc, table, i32([0, 0]))


# -- append ------------------------------------------------------------------------------------

def append_case(seed, kind, b, n, hkv, hq, d, page, starts, rot, pairs, counts=None, positions=None, far=0):
    r = np.random.default_rng(seed)
    starts = np.asarray(starts)
    kc, vc, table = cache(r, b, int(starts.max()) + n, page, hkv, d, kind, stale=5.0)
    qkv = rand(r, b, n, hq + 2 * hkv, d, kind=kind)
    q, k, v = qkv.split([hq, hkv, hkv], dim=2)
    inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32) if rot else None
    if positions is None and far:
        positions = starts[:, None] + r.integers(0, n, (b, n)) + far
    k0, v0 = host(kc), host(vc)
    got = ops.cache_append(k, v, kc, vc, table, i32(starts), q=q if hq else None,
                           positions=None if positions is None else i32(positions),
                           counts=None if counts is None else i32(counts),
                           inv_freq=None if inv is None else torch.from_numpy(inv).cuda(), interleaved=pairs)
    want = co.append(host(k), host(v), host(q) if hq else None, k0, v0, table.cpu().numpy(), starts, positions, counts,
                     inv, pairs)
    close(host(kc), want["k"], want["bk"], kind)
    untouched = (want["k"] == k0) & (want["bk"] == 0)
    assert (host(kc)[untouched] == k0[untouched]).all()
    np.testing.assert_array_equal(host(vc), want["v"])
    if hq:
        close(host(got["q"]), want["q"], want["bq"], kind)
    else:
        assert got == {}


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("b, n, hkv, hq, d, page, starts, rot", [
    (1, 1, 1, 1, 64, 16, [0], 64), (2, 3, 2, 8, 128, 16, [15, 31], 128), (3, 9, 2, 0, 80, 24, [0, 20, 47], 32),
    (2, 40, 1, 3, 33, 7, [5, 0], 10), (1, 130, 3, 6, 96, 32, [64], 96), (2, 5, 1, 1, 256, 8, [3, 9], 128),
    (2, 4, 2, 2, 1, 3, [1, 2], 0), (1, 2, 1, 2, 2, 1, [4], 2), (2, 6, 2, 4, 64, 16, [7, 8], 0), (1, 3, 1, 5, 72, 16, [2], 24),
])
def test_append(kind, pairs, b, n, hkv, hq, d, page, starts, rot):
    append_case(11, kind, b, n, hkv, hq, d, page, starts, rot, pairs)


@pytest.mark.parametrize("far", [1 << 20, 2_000_000_000])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_append_far_positions(far, kind):
    append_case(12, kind, 3, 20, 2, 4, 128, 16, [3, 9, 0], 128, False, counts=[20, 0, 7], far=far)


def test_append_negative_positions_and_frequencies():
    r = np.random.default_rng(13)
    append_case(13, "f32", 2, 4, 1, 2, 64, 8, [0, 3], 64, True, positions=r.integers(-(1 << 31), 0, (2, 4)))


@pytest.mark.parametrize("f", [0.0, -0.25, 1.0, 3.7, -1e-3, 1e-20, 1e-38, 1e-45])
def test_append_frequencies(f):
    r = np.random.default_rng(14)
    kc, vc, table = cache(r, 1, 8, 8, 1, 2, "f32", stale=0.0)
    k = rand(r, 1, 8, 1, 2)
    pos = np.array([[0, 1, 2, 1000, -5, 99999, 1 << 22, -(1 << 24)]])
    inv = np.array([f], np.float32)
    ops.cache_append(k, k, kc, vc, table, i32([0]), positions=i32(pos), inv_freq=torch.from_numpy(inv).cuda())
    want = co.append(host(k), host(k), None, np.zeros(kc.shape), np.zeros(kc.shape), table.cpu().numpy(), [0], pos, None, inv)
    close(host(kc), want["k"], want["bk"] * (1 + 2.0 ** -38 * abs(f) * 2.0 ** 24))


def test_append_carries_what_is_not_finite_and_takes_no_frequency_that_is_not():
    kc, vc, table = cache(np.random.default_rng(0), 1, 4, 4, 1, 4, "bf16", stale=0.0)
    k = torch.tensor([NAN, 1.0, INF, -INF], device="cuda").to(torch.bfloat16).view(1, 1, 1, 4)
    ops.cache_append(k, k, kc, vc, table, i32([1]))
    p = int(table[0, 0])
    for c in (kc, vc):
        assert torch.equal(c[p, 1, 0].view(torch.int16), k.view(4).view(torch.int16)) and (c[p, [0, 2, 3]] == 0).all()
    one = torch.ones(1, 1, 1, 4, device="cuda")
    kc, vc = torch.zeros(1, 4, 1, 4, device="cuda"), torch.zeros(1, 4, 1, 4, device="cuda")
    ops.cache_append(one, one, kc, vc, i32([[0]]), i32([3]), inv_freq=torch.tensor([INF, 0.0], device="cuda"))
    assert kc[0, 3, 0, [0, 2]].isnan().all() and (kc[0, 3, 0, [1, 3]] == 1).all()


def test_append_in_place_and_into_other_layouts():
    r = np.random.default_rng(15)
    inv = torch.tensor([1.0, 0.1, 0.01, 0.001], device="cuda")
    for kind, lead in (("bf16", 0), ("f16", 1), ("f32", 0)):
        q, k = rand(r, 2, 3, 4, 16, kind=kind), rand(r, 2, 3, 2, 16, kind=kind)
        want = {}
        for layout in (0, 1):
            store = torch.full((lead + 6 * 8 * 2 * 16,), 9.0, dtype=TYPES[kind], device="cuda")
            kc = store[lead:].view(6, 8, 2, 16) if layout == 0 else store[lead:].view(6, 2, 8, 16).transpose(1, 2)
            vc = kc.clone()
            mine = q.clone()
            table = i32([[4, 1], [0, 5]])
            got = ops.cache_append(k, k, kc, vc, table, i32([6, 2]), q=mine, inv_freq=inv, out={"q": mine})
            assert got["q"] is mine
            want.setdefault("q", mine), want.setdefault("k", kc.contiguous()), want.setdefault("v", vc.contiguous())
            for name, t in (("q", mine), ("k", kc), ("v", vc)):
                assert torch.equal(want[name], t)
        ref = co.append(host(k), host(k), host(q), np.full((6, 8, 2, 16), 9.0), np.full((6, 8, 2, 16), 9.0),
                        [[4, 1], [0, 5]], [6, 2], None, None, host(inv))
        close(host(want["q"]), ref["q"], ref["bq"], kind)
        close(host(want["k"]), ref["k"], ref["bk"], kind)


def test_append_leaves_bad_places_alone():
    r = np.random.default_rng(16)
    kc, vc, table = cache(r, 4, 16, 8, 1, 8, "f32", stale=0.0)
    table[0, 1], table[1, 0] = -1, kc.shape[0]
    starts, counts = [6, 7, -1, 15], [4, 4, 4, 9]
    k, q = rand(r, 4, 4, 1, 8), rand(r, 4, 4, 2, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.cache_append(k, k, kc, vc, table, i32(starts), q=q, counts=i32(counts), status=status)
    want = co.append(host(k), host(k), host(q), np.zeros(kc.shape), np.zeros(kc.shape), table.cpu().numpy(), starts, None, counts)
    np.testing.assert_array_equal(host(kc), want["k"])
    np.testing.assert_array_equal(host(vc), want["v"])
    np.testing.assert_array_equal(host(got["q"]), want["q"])
    assert want["flag"] and status.item() == capi.PER_DEVFLAG_BAD_INDEX


# -- keep --------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b, hkv, d, page, most, nodes", [
    (1, 1, 64, 16, 1, 4), (5, 2, 128, 16, 6, 24), (3, 3, 33, 7, 9, 20), (2, 1, 1, 1, 20, 30), (3, 2, 256, 64, 40, 64),
    (2, 8, 128, 24, 17, 90),
])
def test_keep(kind, b, hkv, d, page, most, nodes):
    r = np.random.default_rng(17)
    lens = r.integers(0, 50, b)
    kc, vc, table = cache(r, b, 50 + nodes, page, hkv, d, kind)
    fill(r, kc, vc, table, lens + nodes, kind)
    path = np.stack([np.sort(r.permutation(nodes)[:most]) for _ in range(b)])
    kept = r.integers(0, most + 1, b)
    kept[0] = most
    want = co.keep(host(kc), host(vc), table.cpu().numpy(), lens, path, kept)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.cache_keep(kc, vc, table, i32(lens), i32(path), i32(kept), nodes=nodes, status=status)
    np.testing.assert_array_equal(host(kc), want["k"])
    np.testing.assert_array_equal(host(vc), want["v"])
    assert not want["flag"] and status.item() == 0


@pytest.mark.parametrize("path, kept, nodes", [
    ([0, 2, 2, 5], 4, 8), ([1, 0, 3, 4], 4, 8), ([0, 3, 8, 9], 4, 8), ([-1, 1, 2, 3], 2, 8), ([0, 1, 3, 6], 9, 8),
    ([2, 3, 5, 6], -1, 8), ([0, 2, 4, 30], 4, 64),
])
def test_keep_ends_where_a_path_is_none(path, kept, nodes):
    r = np.random.default_rng(18)
    kc, vc, table = cache(r, 1, 24, 8, 2, 16, "f32", stale=0.0)
    fill(r, kc, vc, table, [24], "f32")
    want = co.keep(host(kc), host(vc), table.cpu().numpy(), [5], np.array([path]), [kept], nodes)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.cache_keep(kc, vc, table, i32([5]), i32([path]), i32([kept]), nodes=nodes, status=status)
    np.testing.assert_array_equal(host(kc), want["k"])
    np.testing.assert_array_equal(host(vc), want["v"])
    assert want["flag"] and status.item() == capi.PER_DEVFLAG_BAD_INDEX


# -- together ----------------------------------------------------------------------------------

def test_a_verified_round():
    """A prompt, a drafted chain and what is accepted of it, over a cache, give what one pass over the whole
    sequence gives; then a tree whose path is kept."""
    r = np.random.default_rng(19)
    b, hkv, g, d, page = 3, 2, 2, 64, 16
    kc, vc, table = cache(r, b, 64, page, hkv, d, "f32")
    inv = torch.from_numpy((100.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)).cuda()
    tokens = rand(r, b, 40, (g + 2) * hkv, d)
    parts = lambda t: t.split([g * hkv, hkv, hkv], dim=2)       # noqa: E731
    lens = i32([20, 17, 11])
    q, k, v = parts(tokens[:, :20])
    ops.cache_append(k, v, kc, vc, table, i32([0, 0, 0]), counts=lens, inv_freq=inv)
    # a tree of 7 nodes: 0 - 1 - 3 - 6 is the path; 2, 4, 5 branch off
    mask = torch.zeros(7, 7, dtype=torch.bool, device="cuda")
    for i, up in enumerate([-1, 0, 0, 1, 1, 2, 3]):
        if up >= 0:
            mask[i] = mask[up]
        mask[i, i] = True
    depth = mask.sum(1).int() - 1
    drafted = rand(r, b, 7, (g + 2) * hkv, d)
    q, k, v = parts(drafted)
    turned = ops.cache_append(k, v, kc, vc, table, lens, q=q, positions=lens[:, None] + depth, inv_freq=inv)["q"]
    out = ops.tree_attention(turned, kc, vc, table, lens, mask=mask)["out"]
    path = i32([[0, 1, 3, 6]] * b)
    probs = torch.softmax(out[:, [0, 1, 3, 6]].flatten(2)[..., :50], -1)
    got = ops.verify_draft(probs, None, probs[:, :3].argmax(-1), torch.zeros(b, 3, device="cuda"), torch.zeros(b, device="cuda"))
    assert got["accepted"].tolist() == [3] * b
    kept = got["accepted"] + 1
    ops.cache_keep(kc, vc, table, lens, path, kept, nodes=7)
    # the same sequences in one go, in a cache of their own
    k2, v2, table2 = cache(r, b, 64, 8, hkv, d, "f32")
    whole = torch.stack([torch.cat([tokens[i, :n], drafted[i, [0, 1, 3, 6]], tokens[i, n:36]]) for i, n in enumerate(lens.tolist())])
    q2, kk, vv = parts(whole[:, :24])
    total = lens + 4
    turned2 = ops.cache_append(kk, vv, k2, v2, table2, i32([0] * b), q=q2, counts=total, inv_freq=inv)["q"]
    out2 = ops.tree_attention(turned2, k2, v2, table2, i32([0] * b), counts=total)["out"]
    for i, n in enumerate(lens.tolist()):
        torch.testing.assert_close(out[i, [0, 1, 3, 6]], out2[i, n:n + 4], rtol=1e-4, atol=1e-5)
        for s in range(n + 4):
            p, x = co.place(table[i].tolist(), s, page, kc.shape[0])
            p2, x2 = co.place(table2[i].tolist(), s, 8, k2.shape[0])
            assert torch.equal(kc[p, x], k2[p2, x2]) and torch.equal(vc[p, x], v2[p2, x2])


def test_captured_and_replayed():
    """Append, attention and keep in one graph, its inputs changed between replays; two graphs at once on their
    own streams."""
    r = np.random.default_rng(20)
    graphs = []
    for _ in range(2):
        kc, vc, table = cache(r, 4, 700, 16, 2, 64, "bf16", stale=0.0)
        fill(r, kc, vc, table, [600] * 4, "bf16")
        s = dict(k=rand(r, 4, 5, 2, 64, kind="bf16"), q=rand(r, 4, 5, 8, 64, kind="bf16"), kc=kc, vc=vc, table=table,
                 lens=i32([500, 3, 64, 0]), path=i32([[0, 2, 4]] * 4), kept=i32([3, 1, 2, 0]),
                 inv=torch.rand(32, device="cuda"), stream=torch.cuda.Stream())

        def go(s=s):
            turned = ops.cache_append(s["k"], s["k"], s["kc"], s["vc"], s["table"], s["lens"], q=s["q"], inv_freq=s["inv"])["q"]
            got = ops.tree_attention(turned, s["kc"], s["vc"], s["table"], s["lens"])
            ops.cache_keep(s["kc"], s["vc"], s["table"], s["lens"], s["path"], s["kept"])
            return got

        go()
        torch.cuda.synchronize()
        s["go"], s["graph"] = go, torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            s["got"] = go()
        graphs.append(s)
    for turn in range(3):
        for s in graphs:
            s["lens"].copy_(i32(r.integers(0, 590, 4)))
            s["q"].copy_(rand(r, 4, 5, 8, 64, kind="bf16"))
        torch.cuda.synchronize()
        before = [(s["kc"].clone(), s["vc"].clone()) for s in graphs]
        torch.cuda.synchronize()
        for s in graphs:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s, (k0, v0) in zip(graphs, before):
            got = {n: t.clone() for n, t in s["got"].items()}
            after = s["kc"].clone(), s["vc"].clone()
            s["kc"].copy_(k0), s["vc"].copy_(v0)
            want = s["go"]()
            assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
            assert torch.equal(after[0], s["kc"]) and torch.equal(after[1], s["vc"])


def test_another_stream_and_given_outputs():
    r = np.random.default_rng(21)
    kc, vc, table = cache(r, 2, 9000, 16, 1, 64, "f16")
    fill(r, kc, vc, table, [9000, 300], "f16")
    q, lens = rand(r, 2, 4, 4, 64, kind="f16"), i32([8980, 5])
    want = ops.tree_attention(q, kc, vc, table, lens)
    side = torch.cuda.Stream()
    work = torch.empty(ops.tree_attention_work(q, kc, vc, table), dtype=torch.uint8, device="cuda")
    assert work.numel() and not ops.tree_attention_work(q, kc, vc, table[:, :1])
    out = {"out": torch.empty_like(q), "lse": torch.empty(2, 4, 4, device="cuda")}
    side.wait_stream(torch.cuda.current_stream())
    got = ops.tree_attention(q, kc, vc, table, lens, out=out, work=work, stream=side)
    side.synchronize()
    assert got["out"] is out["out"] and got["lse"] is out["lse"]
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    with pytest.raises(capi.PerError, match="work"):
        ops.tree_attention(q, kc, vc, table, lens, work=work[:-1])


def test_a_cache_past_32_bits_of_elements():
    """Offsets beyond 2^32 elements: pages at the far end of a large cache."""
    hkv, d, page = 8, 128, 64
    pages = (1 << 32) // (page * hkv * d) + 40
    kc = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    r = np.random.default_rng(22)
    table = i32([[pages - 1, 3, pages - 7]])
    new = rand(r, 1, 150, hkv, d, kind="bf16")
    ops.cache_append(new, new, kc, vc, table, i32([0]))
    small_k = kc[table[0].long()].contiguous()
    small_v = vc[table[0].long()].contiguous()
    q = rand(r, 1, 6, 16, d, kind="bf16")
    got = ops.tree_attention(q, kc, vc, table, i32([144]))
    want = ops.tree_attention(q, small_k, small_v, i32([[0, 1, 2]]), i32([144]))
    assert torch.equal(got["out"], want["out"]) and torch.equal(small_v.view(-1, hkv, d)[:150], new[0])
    ops.cache_keep(kc, vc, table, i32([140]), i32([[1, 4, 9]]), i32([3]))
    for j, x in enumerate((1, 4, 9)):
        assert torch.equal(vc[pages - 7, 140 - 128 + j], new[0, 140 + x])


def test_refusals():
    r = np.random.default_rng(23)
    kc, vc, table = cache(r, 2, 32, 16, 2, 64, "bf16", stale=0.0)
    q, k, lens = rand(r, 2, 3, 4, 64, kind="bf16"), rand(r, 2, 3, 2, 64, kind="bf16"), i32([3, 4])
    bad = [
        lambda: ops.tree_attention(q.float(), kc, vc, table, lens),
        lambda: ops.tree_attention(q[:, :, :3], kc, vc, table, lens),
        lambda: ops.tree_attention(q, kc, vc[:-1], table, lens),
        lambda: ops.tree_attention(q, kc, vc, table.long(), lens),
        lambda: ops.tree_attention(q, kc, vc, table[:1], lens),
        lambda: ops.tree_attention(q, kc, vc, table, lens.long()),
        lambda: ops.tree_attention(q, kc, vc, table, lens, mask=torch.ones(3, 4, dtype=torch.bool, device="cuda")),
        lambda: ops.tree_attention(q, kc, vc, table, lens, mask=torch.ones(3, 3, device="cuda")),
        lambda: ops.tree_attention(q, kc, vc, table, lens, scale=INF),
        lambda: ops.tree_attention(q, kc, vc, table, lens, work=torch.empty(0, device="cuda")),
        lambda: ops.tree_attention(q.transpose(2, 3), kc, vc, table, lens),
        lambda: ops.tree_attention(torch.zeros(2, 1025, 4, 64, dtype=torch.bfloat16, device="cuda"), kc, vc, table, lens),
        lambda: ops.cache_append(k, k[:, :2], kc, vc, table, lens),
        lambda: ops.cache_append(k, k, kc[..., :32], vc[..., :32], table, lens),
        lambda: ops.cache_append(k, k, kc, vc, table, None),
        lambda: ops.cache_append(k, k, kc, vc, table, lens, inv_freq=torch.ones(33, device="cuda")),
        lambda: ops.cache_append(k, k, kc, vc, table, lens, positions=i32([1, 2])),
        lambda: ops.cache_append(k, k, kc[:1].expand(5, -1, -1, -1), vc[:1].expand(5, -1, -1, -1), table, lens),
        lambda: ops.cache_append(k, k, kc, vc, table, lens, q=q, out={"q": q[:, :1].expand(-1, 3, -1, -1)}),
        lambda: ops.cache_keep(kc, vc, table, lens, i32([[0, 1]] * 3), i32([1, 1])),
        lambda: ops.cache_keep(kc, vc, table, lens, i32([[0, 1]] * 2), None),
        lambda: ops.cache_keep(kc, vc, table, lens, torch.zeros(2, 1025, dtype=torch.int32, device="cuda"), i32([1, 1])),
    ]
    before = kc.clone(), vc.clone()
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, capi.PerError)):
            call()
            pytest.fail(f"call {i} was not refused")
    assert torch.equal(before[0], kc) and torch.equal(before[1], vc)
    with pytest.raises(RuntimeError, match="no gradient"):
        ops.tree_attention(q.clone().requires_grad_(), kc, vc, table, lens)
    with torch.no_grad():
        ops.tree_attention(q.clone().requires_grad_(), kc, vc, table, lens)


def test_dual_tensors_are_refused():
    """A tensor with a tangent of forward-mode differentiation does not pass as a constant, under no_grad neither."""
    import torch.autograd.forward_ad as fw
    kc = torch.zeros(4, 16, 1, 32, device="cuda")
    vc, table, lens = kc.clone(), i32([[1, 2]]), i32([3])
    q, one = torch.ones(1, 2, 1, 32, device="cuda"), torch.ones(1, 2, 1, 32, device="cuda")
    inv = torch.ones(4, device="cuda")
    with fw.dual_level():
        dual = lambda t: fw.make_dual(t, torch.ones_like(t))
        for call in (lambda: ops.tree_attention(dual(q), kc, vc, table, lens), lambda: ops.tree_attention(q, kc, dual(vc), table, lens),
                     lambda: ops.cache_append(dual(one), one, kc, vc, table, lens), lambda: ops.cache_append(one, one, kc, vc, table, lens, q=dual(q)),
                     lambda: ops.cache_append(one, one, kc, vc, table, lens, inv_freq=dual(inv)),
                     lambda: ops.cache_keep(dual(kc), vc, table, lens, i32([[0]]), i32([1]))):
            for grad in (True, False):
                with torch.set_grad_enabled(grad), pytest.raises(RuntimeError, match="no gradient"):
                    call()
        assert (ops.tree_attention(q, kc, vc, table, lens)["out"] == 0).all()
    assert (kc == 0).all()
    ops.tree_attention(q, kc, vc, table, lens)
