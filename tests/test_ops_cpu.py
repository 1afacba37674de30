"""The operators' host side: what the C calls and the binding refuse (nothing is enqueued, so no GPU is
needed), and the 64-bit definitions against differences and brute force."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from rl_infra_gb300 import build, capi
from tests import ops_oracle as oo

torch = pytest.importorskip("torch")

ONE = 1 << 12          # a pointer that is never followed: each call is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


def _distill_shape(**kw):
    s = capi.per_distill_shape(rows=2, vocab=8, top=2, type=0, top_type=0, stride_logits=8, stride_top=2, stride_idx=2,
                               stride_grad=8, temperature=1.0, flags=0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw, args, said", [
    (dict(rows=1 << 31), {}, "rows"), (dict(vocab=0), {}, "vocab"), (dict(vocab=(1 << 18) + 1), {}, "vocab"),
    (dict(top=0), {}, "top"), (dict(top=1025), {}, "top"), (dict(type=3), {}, "type"), (dict(top_type=9), {}, "type"),
    (dict(flags=2), {}, "flags"), (dict(temperature=0.0), {}, "temperature"), (dict(temperature=-1.0), {}, "temperature"),
    (dict(temperature=float("nan")), {}, "temperature"), (dict(temperature=float("inf")), {}, "temperature"),
    (dict(stride_grad=7), {}, "overlap"), (dict(stride_grad=0), {}, "overlap"),
    ({}, dict(x=None), "required"), ({}, dict(top=None), "required"), ({}, dict(idx=None), "required"),
    ({}, dict(loss=None), "required"), ({}, dict(grad=None), "required"), ({}, dict(x=ONE + 2), "misaligned"),
    ({}, dict(loss=ONE + 2), "misaligned"), (dict(flags=1), dict(idx=ONE + 4), "misaligned"),
    (dict(stride_grad=16), dict(grad=ONE), "stride"),
])
def test_distill_refuses(kw, args, said):
    a = dict(x=ONE, top=2 * ONE, idx=3 * ONE, loss=4 * ONE, grad=5 * ONE)
    a.update(args)
    s = capi.per_distill_step(ctypes.byref(_distill_shape(**kw)), a["x"], a["top"], a["idx"], None, None, a["loss"], None,
                              a["grad"], None, None)
    assert s == capi.PER_ERR_INVALID_ARG
    assert said in capi.per_last_op_error() and capi.per_last_op_error().startswith("per_distill_step")


def test_null_shapes_are_refused():
    assert capi.per_distill_forward(None, ONE, ONE, ONE, None, ONE, ONE, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_distill_backward(None, ONE, ONE, ONE, None, ONE, None, ONE, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_verify_draft(None, ONE, ONE, ONE, None, ONE, ONE, ONE, ONE, None, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_scan_forward(None, ONE, ONE, None, None, ONE, None, None) == capi.PER_ERR_INVALID_ARG
    assert capi.per_scan_backward(None, ONE, ONE, ONE, None, None, ONE, None, ONE, ONE, None, None) == capi.PER_ERR_INVALID_ARG


def test_backward_needs_lse_and_empty_batches_are_no_ops():
    s = _distill_shape()
    assert capi.per_distill_backward(ctypes.byref(s), ONE, ONE, ONE, None, None, None, ONE, None, None) == capi.PER_ERR_INVALID_ARG
    s.rows = 0
    assert capi.per_distill_step(ctypes.byref(s), None, None, None, None, None, None, None, None, None, None) == capi.PER_OK
    v = capi.per_verify_shape(batch=0, drafts=2, vocab=8)
    assert capi.per_verify_draft(ctypes.byref(v), *[None] * 11) == capi.PER_OK
    for c in (capi.per_scan_shape(steps=4, batch=0, channels=3), capi.per_scan_shape(steps=4, batch=3, channels=0)):
        assert capi.per_scan_forward(ctypes.byref(c), *[None] * 7) == capi.PER_OK
        assert capi.per_scan_backward(ctypes.byref(c), *[None] * 11) == capi.PER_OK


@pytest.mark.parametrize("kw, args, said", [
    (dict(batch=(1 << 20) + 1), {}, "batch"), (dict(drafts=1025), {}, "drafts"), (dict(vocab=0), {}, "vocab"),
    (dict(vocab=(1 << 18) + 1), {}, "vocab"), (dict(type=3), {}, "type"), (dict(flags=2), {}, "flags"),
    (dict(reserved=1), {}, "flags"), ({}, dict(p=None), "required"), ({}, dict(tokens=None), "required"),
    ({}, dict(u=None), "required"), ({}, dict(us=None), "required"), ({}, dict(out=None), "required"),
    ({}, dict(p=ONE + 2), "misaligned"), (dict(flags=1), dict(tokens=ONE + 4), "misaligned"),
    ({}, dict(out=ONE + 1), "misaligned"),
])
def test_verify_refuses(kw, args, said):
    sh = capi.per_verify_shape(batch=2, drafts=2, vocab=8, type=0)
    for k, v in kw.items():
        setattr(sh, k, v)
    a = dict(p=ONE, q=ONE, tokens=ONE, u=ONE, us=ONE, acc=ONE, out=ONE)
    a.update(args)
    s = capi.per_verify_draft(ctypes.byref(sh), a["p"], a["q"], a["tokens"], None, a["u"], a["us"], a["acc"], a["out"], None,
                              None, None)
    assert s == capi.PER_ERR_INVALID_ARG and said in capi.per_last_op_error()


@pytest.mark.parametrize("kw, args, said", [
    (dict(steps=1 << 31), {}, "steps"), (dict(batch=1 << 16, channels=1 << 16), {}, "below 2^31"), (dict(type=3), {}, "type"),
    (dict(flags=4), {}, "flags"), ({}, dict(a=None), "required"), ({}, dict(x=None), "required"),
    ({}, dict(h=None), "required"), ({}, dict(a=ONE + 2), "misaligned"), ({}, dict(h0=ONE + 2), "misaligned"),
    (dict(stride_h=(ctypes.c_int64 * 2)(40, 7)), {}, "overlap"), (dict(stride_h=(ctypes.c_int64 * 2)(31, 8)), {}, "overlap"),
    (dict(stride_h=(ctypes.c_int64 * 2)(8, 15)), {}, "overlap"), (dict(stride_h=(ctypes.c_int64 * 2)(32, 0)), {}, "overlap"),
])
def test_scan_refuses(kw, args, said):
    sh = capi.per_scan_shape(steps=4, batch=2, channels=8, type=0, stride_h=(ctypes.c_int64 * 2)(32, 8))
    for k, v in kw.items():
        setattr(sh, k, v)
    a = dict(a=ONE, x=ONE, h=ONE, h0=None)
    a.update(args)
    s = capi.per_scan_forward(ctypes.byref(sh), a["a"], a["x"], a["h0"], None, a["h"], None, None)
    assert s == capi.PER_ERR_INVALID_ARG and said in capi.per_last_op_error()


def test_scan_backward_needs_x_with_a_gate():
    sh = capi.per_scan_shape(steps=4, batch=2, channels=8, type=0, flags=capi.PER_SCAN_SIGMOID)
    for n in ("ga", "gx"):
        setattr(sh, "stride_" + n, (ctypes.c_int64 * 2)(32, 8))
    assert capi.per_scan_backward(ctypes.byref(sh), ONE, None, ONE, None, None, ONE, None, ONE, ONE, None, None) == \
        capi.PER_ERR_INVALID_ARG
    assert "x is required" in capi.per_last_op_error()


def test_binding_wants_cuda_tensors():
    from rl_infra_gb300 import ops
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="logits"):
        ops.distill_forward(z, z, z.int())
    with pytest.raises(ValueError, match="target_probs"):
        ops.verify_draft(torch.zeros(1, 2, 8), None, torch.zeros(1, 1).int(), torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(ValueError, match="a must"):
        ops.scan_forward(torch.zeros(1, 2, 8), torch.zeros(1, 2, 8))
    with pytest.raises(TypeError):
        ops.scan_step(None, z, z)


# -- the definitions ---------------------------------------------------------------------------

def _differences(f, x, at, step=1e-5):
    out = []
    for i in at:
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out.append((f(hi) - f(lo)) / (2 * step))
    return np.array(out)


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("own_norm", [True, False])
def test_distill_gradient_against_differences(tau, own_norm):
    g = np.random.default_rng(0)
    x, t = g.normal(size=(1, 12)), g.normal(size=(1, 4))
    idx = np.array([[3, 11, -1, 3]])           # one place twice, one entry left out
    tl = None if own_norm else np.array([2.5])
    got = oo.distill(x, t, idx, tau, np.array([0.7]), tl)
    want = _differences(lambda z: 0.7 * oo.distill(z, t, idx, tau, None, tl)["loss"][0], x, [(0, j) for j in range(12)])
    np.testing.assert_allclose(got["grad"][0], want, rtol=1e-8, atol=1e-9)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_gradient_against_differences(sigmoid, reverse):
    g = np.random.default_rng(1)
    a, x = g.normal(size=(2, 5, 3)) * 0.7, g.normal(size=(2, 5, 3))
    h0, gh, gl = g.normal(size=(2, 3)), g.normal(size=(2, 5, 3)), g.normal(size=(2, 3))
    resets = np.zeros((2, 5), np.uint8)
    resets[0, 2] = resets[1, 0] = 1

    def value(a_, x_, h_):
        got = oo.scan(a_, x_, h_, resets, sigmoid, reverse)
        return (got["h"] * gh).sum() + (got["last"] * gl).sum()

    h = oo.scan(a, x, h0, resets, sigmoid, reverse)["h"]
    got = oo.scan_backward(a, x, h, gh, h0, resets, gl, sigmoid, reverse)
    at = [(i, j, k) for i in range(2) for j in range(5) for k in range(3)]
    np.testing.assert_allclose(got["grad_a"].ravel(), _differences(lambda z: value(z, x, h0), a, at), rtol=1e-7, atol=1e-8)
    np.testing.assert_allclose(got["grad_x"].ravel(), _differences(lambda z: value(a, z, h0), x, at), rtol=1e-7, atol=1e-8)
    at = [(i, k) for i in range(2) for k in range(3)]
    np.testing.assert_allclose(got["grad_h0"].ravel(), _differences(lambda z: value(a, x, z), h0, at), rtol=1e-7, atol=1e-8)


def test_verification_emits_the_targets_distribution():
    """Drawing the draft's token, its test and the residual's draw over a grid of random numbers gives
    the target's distribution."""
    p = np.array([0.5, 0.3, 0.2], np.float32)
    q = np.array([0.2, 0.2, 0.6], np.float32)
    n = 200
    grid = ((np.arange(n) + 0.5) / n).astype(np.float32)
    count = np.zeros(3)
    for tok in range(3):
        uu, ss = np.meshgrid(grid, grid, indexing="ij")
        b = n * n
        got = oo.verify(np.broadcast_to(p, (b, 2, 3)), np.broadcast_to(q, (b, 1, 3)), np.full((b, 1), tok),
                        uu.reshape(b, 1), ss.reshape(b))
        first = got["tokens"][:, 0]
        count += q[tok] * np.bincount(first, minlength=3) / b
    np.testing.assert_allclose(count, p, atol=2.0 / n)
