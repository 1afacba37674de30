"""The paged cache's operators on the host side: what the C calls and the binding refuse (nothing is enqueued, so no GPU
is needed), and the 64-bit definitions against other ways to the same values."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from rl_infra_gb300 import build, capi
from tests import cache_oracle as co

torch = pytest.importorskip("torch")

ONE = 1 << 12          # a pointer that is never followed: each call is refused before a launch
I3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


def _cache(**kw):
    c = capi.per_cache(pages=8, page=16, width=4, heads=2, dim=64, type=capi.PER_TYPE_BF16, stride_table=4,
                       stride_k=I3(2048, 128, 64), stride_v=I3(2048, 128, 64))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE = [(dict(pages=1 << 31), "pages"), (dict(page=0), "page"), (dict(page=(1 << 20) + 1), "page"),
         (dict(width=1 << 28), "width"), (dict(heads=0), "heads"), (dict(heads=4097), "heads"), (dict(dim=0), "dim"),
         (dict(dim=257), "dim"), (dict(type=3), "type")]
OVERLAP = [dict(stride_k=I3(2048, 128, 63)), dict(stride_v=I3(2047, 128, 64)), dict(stride_k=I3(0, 128, 64)),
           dict(stride_v=I3(2048, 64, 64))]


def _append(cache=None, args=None, **kw):
    s = capi.per_append_shape(cache=_cache(**(cache or {})), batch=2, tokens=3, q_heads=4, rot=64,
                              stride_in=(I3 * 2)(I3(384, 128, 64), I3(384, 128, 64)), stride_q=I3(768, 256, 64),
                              stride_q_out=I3(768, 256, 64), stride_positions=3)
    for k, v in kw.items():
        setattr(s, k, v)
    a = dict(k=ONE, v=ONE, q=ONE, kc=ONE, vc=ONE, qo=2 * ONE, table=ONE, starts=ONE, counts=None, pos=None, inv=ONE)
    a.update(args or {})
    return capi.per_cache_append(ctypes.byref(s), a["k"], a["v"], a["q"], a["kc"], a["vc"], a["qo"], a["table"],
                                 a["starts"], a["counts"], a["pos"], a["inv"], None, None)


@pytest.mark.parametrize("cache, kw, args, said", [(c, {}, {}, said) for c, said in CACHE] + [
    (c, {}, {}, "overlap") for c in OVERLAP] + [
    ({}, dict(batch=(1 << 20) + 1), {}, "batch"), ({}, dict(batch=1 << 16, tokens=1 << 16), {}, "2^31"),
    ({}, dict(q_heads=4097), {}, "q_heads"), ({}, dict(rot=63), {}, "rot"), ({}, dict(rot=66), {}, "rot"),
    ({}, dict(flags=2), {}, "flags"), ({}, dict(reserved=1), {}, "flags"),
    ({}, dict(stride_q_out=I3(768, 255, 64)), {}, "overlap"),
    ({}, dict(stride_q_out=I3(768, 256, 64), stride_q=I3(768, 256, 128)), dict(q=2 * ONE), "strides"),
    ({}, {}, dict(k=None), "required"), ({}, {}, dict(v=None), "required"), ({}, {}, dict(starts=None), "required"),
    ({}, {}, dict(kc=None), "required"), ({}, {}, dict(table=None), "required"), ({}, {}, dict(q=None), "required"),
    ({}, {}, dict(qo=None), "required"), ({}, {}, dict(inv=None), "required"), ({}, {}, dict(k=ONE + 1), "misaligned"),
    ({}, {}, dict(vc=ONE + 1), "misaligned"), ({}, {}, dict(starts=ONE + 2), "misaligned"),
    ({}, {}, dict(inv=ONE + 2), "misaligned"),
])
def test_append_refuses(cache, kw, args, said):
    assert _append(cache, args, **kw) == capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error() and capi.per_last_op_error().startswith("per_cache_append")


def _attend(cache=None, args=None, **kw):
    s = capi.per_attend_shape(cache=_cache(**(cache or {})), batch=2, nodes=3, q_heads=4, scale=0.125,
                              stride_q=I3(768, 256, 64), stride_out=I3(768, 256, 64))
    for k, v in kw.items():
        setattr(s, k, v)
    a = dict(q=ONE, kc=ONE, vc=ONE, table=ONE, lens=ONE, out=2 * ONE, lse=None, work=None)
    a.update(args or {})
    return capi.per_tree_attention(ctypes.byref(s), a["q"], a["kc"], a["vc"], a["table"], a["lens"], None, None, a["out"],
                                   a["lse"], a["work"], None, None)


@pytest.mark.parametrize("cache, kw, args, said", [(c, {}, {}, said) for c, said in CACHE] + [
    ({}, dict(batch=(1 << 20) + 1), {}, "batch"), ({}, dict(nodes=1025), {}, "nodes"), ({}, dict(q_heads=0), {}, "q_heads"),
    ({}, dict(q_heads=5), {}, "q_heads"), ({}, dict(q_heads=130), {}, "q_heads"),
    ({}, dict(scale=float("nan")), {}, "scale"), ({}, dict(scale=float("-inf")), {}, "scale"),
    ({}, dict(scale=3e38), {}, "scale"), (dict(width=1 << 25, heads=4096, page=31), dict(batch=1 << 20, q_heads=4096), {}, "2^50"),
    ({}, dict(stride_out=I3(768, 256, 63)), {}, "overlap"), ({}, dict(stride_out=I3(0, 256, 64)), {}, "overlap"),
    ({}, {}, dict(q=None), "required"), ({}, {}, dict(lens=None), "required"), ({}, {}, dict(out=None), "required"),
    ({}, {}, dict(vc=None), "required"), ({}, {}, dict(table=None), "required"), ({}, {}, dict(q=ONE + 1), "misaligned"),
    ({}, {}, dict(lse=ONE + 2), "misaligned"), ({}, {}, dict(work=ONE + 8), "misaligned"),
])
def test_attention_refuses(cache, kw, args, said):
    assert _attend(cache, args, **kw) == capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error() and capi.per_last_op_error().startswith("per_tree_attention")


def _keep(cache=None, args=None, **kw):
    s = capi.per_keep_shape(cache=_cache(**(cache or {})), batch=2, nodes=9, most=3, stride_path=3)
    for k, v in kw.items():
        setattr(s, k, v)
    a = dict(kc=ONE, vc=ONE, table=ONE, lens=ONE, path=ONE, kept=ONE)
    a.update(args or {})
    return capi.per_cache_keep(ctypes.byref(s), a["kc"], a["vc"], a["table"], a["lens"], a["path"], a["kept"], None, None)


@pytest.mark.parametrize("cache, kw, args, said", [(c, {}, {}, said) for c, said in CACHE] + [
    (c, {}, {}, "overlap") for c in OVERLAP] + [
    ({}, dict(batch=(1 << 20) + 1), {}, "batch"), ({}, dict(nodes=(1 << 20) + 1), {}, "nodes"),
    ({}, dict(most=1025), {}, "most"), ({}, dict(reserved=1), {}, "flags"), ({}, {}, dict(lens=None), "required"),
    ({}, {}, dict(path=None), "required"), ({}, {}, dict(kept=None), "required"), ({}, {}, dict(kc=None), "required"),
    ({}, {}, dict(kc=ONE + 1), "misaligned"), ({}, {}, dict(path=ONE + 2), "misaligned"),
])
def test_keep_refuses(cache, kw, args, said):
    assert _keep(cache, args, **kw) == capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error() and capi.per_last_op_error().startswith("per_cache_keep")


def test_null_shapes_and_empty_calls():
    assert capi.per_cache_append(None, *[ONE] * 11, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_tree_attention(None, *[ONE] * 10, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_cache_keep(None, *[ONE] * 6, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_tree_attention_work(None, None, None)[0] == capi.PER_ERR_INVALID_ARG
    none = dict.fromkeys(("k", "v", "q", "kc", "vc", "qo", "table", "starts", "inv"))
    assert _append(args=none, batch=0) == capi.PER_OK and _append(args=none, tokens=0) == capi.PER_OK
    none = dict.fromkeys(("q", "kc", "vc", "table", "lens", "out"))
    assert _attend(args=none, batch=0) == capi.PER_OK and _attend(args=none, nodes=0) == capi.PER_OK
    none = dict.fromkeys(("kc", "vc", "table", "lens", "path", "kept"))
    assert _keep(args=none, batch=0) == capi.PER_OK and _keep(args=none, most=0) == capi.PER_OK
    s = capi.per_attend_shape(cache=_cache(), batch=0, nodes=3, q_heads=4, scale=1.0)
    assert capi.per_tree_attention_work(ctypes.byref(s), None, None) == (capi.PER_OK, 0)


def test_binding_wants_cuda_tensors():
    from rl_infra_gb300 import ops
    z, i = torch.zeros(1, 2, 1, 8), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must"):
        ops.tree_attention(z, z, z, torch.zeros(1, 1, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="k must"):
        ops.cache_append(z, z, z, z, torch.zeros(1, 1, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="k_cache must"):
        ops.cache_keep(z, z, torch.zeros(1, 1, dtype=torch.int32), i, torch.zeros(1, 1, dtype=torch.int32), i)


# -- the definitions ---------------------------------------------------------------------------

def test_attention_against_a_dense_softmax():
    g = np.random.default_rng(0)
    kc, vc = g.normal(size=(9, 4, 2, 8)), g.normal(size=(9, 4, 2, 8))
    table = g.permutation(9)[:6].reshape(2, 3)
    q = g.normal(size=(2, 3, 4, 8))
    lens, counts = [6, 2], [3, 2]
    mask = np.array([[1, 0, 0], [1, 1, 0], [1, 0, 1]], bool)
    got = co.attend(q, kc, vc, table, lens, mask, counts)
    assert not got["flag"]
    for b in range(2):
        keys = kc[table[b]].reshape(12, 2, 8)[:lens[b] + counts[b]]
        values = vc[table[b]].reshape(12, 2, 8)[:lens[b] + counts[b]]
        for h in range(4):
            s = q[b, :counts[b], h] @ keys[:, h // 2].T / np.sqrt(8)
            s[:, lens[b]:] += np.where(mask[:counts[b], :counts[b]], 0, -np.inf)
            p = np.exp(s)
            np.testing.assert_allclose(got["lse"][b, :counts[b], h], np.log(p.sum(1)), rtol=1e-12)
            np.testing.assert_allclose(got["out"][b, :counts[b], h], p / p.sum(1, keepdims=True) @ values[:, h // 2], rtol=1e-10, atol=1e-12)
        assert (got["out"][b, counts[b]:] == 0).all() and (got["lse"][b, counts[b]:] == -np.inf).all()


@pytest.mark.parametrize("pairs", [False, True])
def test_rotated_scores_depend_on_distances_alone(pairs):
    g = np.random.default_rng(1)
    inv = (100.0 ** (-np.arange(4) / 4)).astype(np.float32)
    q, k = g.normal(size=(1, 1, 1, 10)), g.normal(size=(1, 1, 1, 10))
    zero = np.zeros((1, 1, 1, 10))
    scores = []
    for far in (0, 1000, 123456):
        got = co.append(k, k, q, zero, zero, [[0]], [0], np.array([[far]]), None, inv, pairs)
        turned = co.append(k, k, q, zero, zero, [[0]], [0], np.array([[far + 7]]), None, inv, pairs)
        scores.append((got["k"][0, 0, 0] * turned["q"][0, 0, 0]).sum())
        np.testing.assert_array_equal(got["k"][..., 8:], k[..., 8:])
        np.testing.assert_allclose(np.linalg.norm(got["k"]), np.linalg.norm(k), rtol=1e-12)
    np.testing.assert_allclose(scores, scores[0], rtol=1e-9)


def test_keep_against_a_list():
    g = np.random.default_rng(2)
    kc = g.normal(size=(5, 3, 1, 2))
    table = np.array([[4, 1, 3, 0]])
    line = [kc[table[0, s // 3], s % 3, 0, 0] for s in range(12)]
    path = np.array([[0, 2, 3, 6]])
    got = co.keep(kc, kc, table, [4], path, [4])
    moved = line[:4] + [line[4 + x] for x in path[0]] + line[8:]
    assert [got["k"][table[0, s // 3], s % 3, 0, 0] for s in range(12)] == moved and not got["flag"]


@pytest.mark.parametrize("kw, said", [(dict(wait_limit_ms=10001), "wait_limit_ms"), (dict(withhold=9), "withhold")])
def test_attention_refuses_limits(kw, said):
    assert _attend({}, {}, **kw) == capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error()
    s = capi.per_attend_shape(cache=_cache(), batch=2, nodes=3, q_heads=4, scale=1.0, **kw)
    assert capi.per_tree_attention_work(ctypes.byref(s), None, None)[0] == capi.PER_ERR_INVALID_ARG


def test_shared_memory_that_is_cast_asks_for_its_alignment():
    """Dynamic shared memory of bytes lies where the compiler likes unless it asks: what casts it to wider words must."""
    import re
    from pathlib import Path
    seen = 0
    for f in sorted(Path(build.CSRC).glob("*.cu*")):
        for line in re.findall(r"extern __shared__.*", f.read_text()):
            if re.search(r"\bchar\b", line):
                seen += 1
                assert re.search(r"__align__\((16|\d{3,4})\)", line), f"{f.name}: {line}"
    assert seen


def test_one_memory_for_keys_and_values_is_refused():
    """append and keep write both, from different threads; attention reads them and may have one for both."""
    for call, name in ((_append, "per_cache_append"), (_keep, "per_cache_keep")):
        assert call() == capi.PER_ERR_INVALID_ARG
        assert "same memory" in capi.per_last_op_error() and capi.per_last_op_error().startswith(name)
