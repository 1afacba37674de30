"""Attention over a paged cache when a wait inside a kernel runs out: the call ends by itself, its status says so, and
the next call is right again.  The arrival is withheld on the host's word; nothing faults and nothing hangs."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from rl_infra_gb300 import build, capi, ops  # noqa: E402
from tests.test_cache_gpu import TYPES, cache, fill, i32, rand  # noqa: E402

CODES = {"f32": capi.PER_TYPE_F32, "f16": capi.PER_TYPE_F16, "bf16": capi.PER_TYPE_BF16}
KEYS, VALUES, RELEASE, MEET, QUERIES, SCORES, P, OUTPUTS = range(1, 9)
LIMIT = 20             # milliseconds


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


def attend(kind, q, kc, vc, table, lens, status, **kw):
    """out and lse by the C call."""
    (b, n, hq, d), (pages, page, hkv, _), width = q.shape, kc.shape, table.shape[1]
    i3 = ctypes.c_int64 * 3
    c = capi.per_cache(pages=pages, page=page, width=width, heads=hkv, dim=d, type=CODES[kind], stride_table=width,
                       stride_k=i3(*kc.stride()[:3]), stride_v=i3(*vc.stride()[:3]))
    s = capi.per_attend_shape(cache=c, batch=b, nodes=n, q_heads=hq, scale=d ** -0.5, stride_q=i3(*q.stride()[:3]),
                              stride_out=i3(*q.stride()[:3]), **kw)
    done, size = capi.per_tree_attention_work(ctypes.byref(s), kc.data_ptr(), vc.data_ptr())
    assert done == capi.PER_OK
    work = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
    s.work_bytes = size
    out, lse = torch.zeros_like(q), torch.zeros(b, n, hq, device="cuda")
    assert capi.per_tree_attention(ctypes.byref(s), q.data_ptr(), kc.data_ptr(), vc.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                   None, None, out.data_ptr(), lse.data_ptr(), work.data_ptr(), status.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream) == capi.PER_OK
    torch.cuda.synchronize()
    return out, lse


def runs_out(kind, b, n, hkv, g, d, page, ctx, withhold, ends=True):
    r = np.random.default_rng(61)
    kc, vc, table = cache(r, b, ctx + n, page, hkv, d, kind)
    kc.copy_(torch.randn(kc.shape, device="cuda"))
    vc.copy_(torch.randn(vc.shape, device="cuda"))
    q, lens = rand(r, b, n, hkv * g, d, kind=kind), i32(np.maximum(ctx - 7 * np.arange(b), 0))
    want = ops.tree_attention(q, kc, vc, table, lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    attend(kind, q, kc, vc, table, lens, status, wait_limit_ms=LIMIT, withhold=withhold)
    assert status.item() == (capi.PER_DEVFLAG_TIMEOUT if ends else 0)
    status.zero_()
    for kw in (dict(wait_limit_ms=LIMIT), {}):
        out, lse = attend(kind, q, kc, vc, table, lens, status, **kw)
        assert status.item() == 0
        assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("withhold", [KEYS, VALUES, MEET])
@pytest.mark.parametrize("b, n, hkv, g, d, page, ctx", [
    (1, 1, 2, 4, 128, 16, 1000),           # a cluster's CTAs share a sequence
    (2, 1, 1, 2, 64, 16, 20),              # one tile
    (40, 1, 2, 4, 128, 16, 3000),          # more tiles a CTA than its ring holds
    (3, 7, 2, 4, 64, 8, 9000), (2, 6, 1, 2, 256, 16, 2000),
])
def test_few_rows(kind, withhold, b, n, hkv, g, d, page, ctx):
    runs_out(kind, b, n, hkv, g, d, page, ctx, withhold)


@pytest.mark.parametrize("kind, n, g", [("bf16", 1, 4), ("f32", 1, 4), ("f16", 6, 4)])
def test_few_rows_release(kind, n, g):
    runs_out(kind, 40, n, 2, g, 128, 16, 3000, RELEASE)
    runs_out(kind, 1, n, 2, g, 128, 16, 40, RELEASE, ends=False)       # no tile has to wait for another's place
    runs_out(kind, 1, n, 2, g, 128, 16, 40, SCORES, ends=False)        # not a barrier of this kernel


def test_any_layout_has_no_waits():
    runs_out("bf16", 1, 3, 2, 2, 33, 7, 500, KEYS, ends=False)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("withhold", [KEYS, VALUES, MEET, QUERIES, SCORES, P, OUTPUTS])
@pytest.mark.parametrize("b, n, hkv, g, d, page, ctx", [
    (1, 40, 1, 1, 64, 16, 60),             # one tile
    (2, 20, 2, 4, 64, 16, 700), (40, 20, 2, 4, 128, 16, 3000),      # rows that both groups share
    (2, 40, 1, 6, 128, 64, 500), (24, 40, 2, 4, 64, 16, 3000),      # rows of each group's own
])
def test_many_rows(kind, withhold, b, n, hkv, g, d, page, ctx):
    runs_out(kind, b, n, hkv, g, d, page, ctx, withhold)


@pytest.mark.parametrize("n, g, d", [(20, 4, 128), (40, 4, 128), (40, 4, 64)])
def test_many_rows_release(n, g, d):
    runs_out("bf16", 40, n, 2, g, d, 16, 3000, RELEASE)
    runs_out("bf16", 1, n, 2, g, d, 16, 40, RELEASE, ends=False)
