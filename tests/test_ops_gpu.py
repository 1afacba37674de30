"""The operators' kernels against their definitions in 64 bits, element by element, at sizes and masks
where they can go wrong.  Bounds come from tests/ops_oracle.py: what a 32-bit evaluation of the
formulas may be off, in any order of summation, plus one rounding to the output's type."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from rl_infra_gb300 import build, capi, ops  # noqa: E402
from tests import ops_oracle as oo  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


def host(t):
    return t.detach().to(torch.float64 if t.dtype.is_floating_point else torch.int64).cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def rand(g, *shape, kind="f32", scale=1.0, shift=0.0):
    return torch.from_numpy((g.normal(size=shape) * scale + shift).astype(np.float32)).cuda().to(TYPES[kind])


def padded(t, pad, lead=0):
    """The same values with `pad` elements behind each row of the last axis and `lead` before the first."""
    rows = t.numel() // t.shape[-1] if t.shape[-1] else 0
    w = t.shape[-1] + pad
    store = torch.full((lead + rows * w,), 7.0, device=t.device).to(t.dtype)
    strides, s = [1], w
    for n in reversed(t.shape[:-1]):
        strides.insert(0, s)
        s *= n
    view = store.as_strided(t.shape, strides, lead)
    view.copy_(t)
    return view


# -- distillation ------------------------------------------------------------------------------

def teacher(g, n, v, k, kind="f32", wide=False):
    k = min(k, v)
    idx = np.stack([g.permutation(v)[:k] for _ in range(n)])
    return rand(g, n, k, kind=kind, scale=2.0, shift=3.0), torch.from_numpy(idx).cuda().to(torch.int64 if wide else torch.int32)


def check_distill(x, t, idx, tau=1.0, scale=None, tlse=None, part="all", kind="f32", **kw):
    want = oo.distill(host(x), host(t), host(idx), tau, None if scale is None else host(scale),
                      None if tlse is None else host(tlse))
    fwd = ops.distill_forward(x, t, idx, temperature=tau, teacher_lse=tlse, **kw)
    oo.close(f32(fwd["lse"]), want["lse"], want["blse"])
    oo.close(f32(fwd["loss"]), want["loss"], want["bloss"])
    step = ops.distill_step(x, t, idx, scale, temperature=tau, teacher_lse=tlse, **kw)
    oo.close(f32(step["lse"]), want["lse"], want["blse"])
    oo.close(f32(step["loss"]), want["loss"], want["bloss"])
    oo.close(f32(step["grad"]), want["grad"], want["bgrad"], kind)
    back = ops.distill_backward(x, t, idx, fwd["lse"], scale, temperature=tau, teacher_lse=tlse, **kw)
    oo.close(f32(back["grad"]), want["grad"], want["bgrad"], kind)
    return step


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n, v, k", [(1, 1, 1), (3, 2, 2), (5, 31, 4), (4, 64, 64), (7, 257, 5), (33, 1009, 8), (3, 4096, 100),
                                     (2, 8200, 33), (2, 16384, 1024), (3, 20011, 64), (2, 65537, 7)])
def test_distill(kind, n, v, k):
    g = np.random.default_rng(n + v)
    x = rand(g, n, v, kind=kind, scale=2.0)
    t, idx = teacher(g, n, v, k)
    check_distill(x, t, idx, scale=rand(g, n).abs(), kind=kind)


@pytest.mark.parametrize("v", [100003, 131072, 200000, 262144, 262143])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_distill_large_vocabularies(kind, v):
    g = np.random.default_rng(v)
    x = rand(g, 2, v, kind=kind, scale=3.0)
    t, idx = teacher(g, 2, v, 50)
    idx[0, :4] = torch.tensor([0, v - 1, v // 2, v // 4], device="cuda")
    check_distill(x, t, idx, tau=2.0, kind=kind)


@pytest.mark.parametrize("tau", [0.3, 1.0, 4.0])
@pytest.mark.parametrize("tkind, wide", [("f32", True), ("f16", False), ("bf16", True)])
def test_distill_types_of_the_teacher(tau, tkind, wide):
    g = np.random.default_rng(3)
    x = rand(g, 6, 777, kind="bf16", scale=2.0)
    t, idx = teacher(g, 6, 777, 12, kind=tkind, wide=wide)
    tl = tau * torch.logsumexp(t.float() / tau, 1) + 0.3     # the teacher's own normaliser: the top K hold less than 1
    check_distill(x, t, idx, tau=tau, tlse=tl, scale=rand(g, 6), kind="bf16")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad, lead", [(1, 0), (3, 5), (8, 8), (24, 1), (0, 3)])
@pytest.mark.parametrize("v", [130, 4104])
def test_distill_strides_and_alignment(kind, pad, lead, v):
    g = np.random.default_rng(pad * 10 + lead)
    x = rand(g, 5, v, kind=kind, scale=2.0)
    t, idx = teacher(g, 5, v, 9)
    xp, tp, ip = padded(x, pad, lead), padded(t, 2, 1), padded(idx, 3)
    grad = padded(torch.zeros_like(x), 2, 1)
    want = check_distill(x, t, idx, kind=kind)
    got = ops.distill_step(xp, tp, ip, out={"grad": grad})
    assert torch.equal(got["loss"], want["loss"])
    assert torch.equal(grad, want["grad"])
    whole = grad.as_strided((5, v + 2), (v + 2, 1), 1)
    assert (whole[:4, v:] == 7).all(), "written between the rows"
    # in the logits' place
    got = ops.distill_step(xp, tp, ip, out={"grad": xp})
    assert torch.equal(xp, want["grad"]) and torch.equal(got["loss"], want["loss"])
    assert (xp.as_strided((4, pad), (v + pad, 1), lead + v) == 7).all()
    xp.copy_(x)
    ops.distill_backward(xp, tp, ip, got["lse"], out={"grad": xp})
    oo.close(f32(xp), host(want["grad"]), 1e-5 * np.abs(host(want["grad"])) + 1e-7, kind)


def test_distill_broadcast_rows_share_a_teacher():
    g = np.random.default_rng(5)
    x = rand(g, 4, 300)
    t, idx = teacher(g, 1, 300, 6)
    check_distill(x, t.expand(4, -1), idx.expand(4, -1))
    check_distill(x[:1].expand(4, -1), t.expand(4, -1), idx.expand(4, -1))


def test_distill_repeated_places_add_up():
    g = np.random.default_rng(6)
    x = rand(g, 3, 50)
    idx = torch.tensor([[4, 4, 4, 9], [1, 2, 1, 2], [49, 0, 49, 49]], dtype=torch.int32, device="cuda")
    check_distill(x, rand(g, 3, 4), idx)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("v", [37, 5000])
def test_distill_empty_and_masked_rows(kind, v):
    """Rows without a teacher's entry, masks of -inf and of the type's lowest value, whole rows of either,
    a teacher that gives -inf, and indexes that are left out."""
    g = np.random.default_rng(7)
    low = torch.finfo(TYPES[kind]).min
    x = rand(g, 8, v, kind=kind)
    t, idx = teacher(g, 8, v, 5)
    idx[0] = -1
    t[0] = float("nan")                      # whatever stands at entries left out
    x[1, 3:] = -INF
    idx[1] = torch.tensor([0, 1, 2, -1, -7], dtype=torch.int32)
    x[2] = -INF
    x[3, 1:] = low
    idx[3] = torch.tensor([0, -1, -1, -1, -1], dtype=torch.int32)
    x[4] = low
    t[5] = -INF
    t[6, 2:] = -INF
    idx[7, 0] = -2147483648
    check_distill(x, t, idx, kind=kind)
    step = ops.distill_step(x, t, idx)
    for r in (0, 2, 5):
        assert step["loss"][r] == 0 and (step["grad"][r] == 0).all()
    assert step["lse"][2] == -INF


def test_distill_infinities_and_nan_stay_in_their_rows():
    g = np.random.default_rng(8)
    x = rand(g, 5, 3000)
    t, idx = teacher(g, 5, 3000, 5)
    idx[:, 0] = 17
    x[0, 17] = -INF          # the teacher wants what the student excludes
    x[1, 2999] = float("nan")
    x[2, 5] = INF
    t[3, 1] = float("nan")
    step = ops.distill_step(x, t, idx)
    assert step["loss"][0] == INF and torch.isfinite(step["grad"][0]).all()
    for r in (1, 2, 3):
        assert torch.isnan(step["loss"][r])
    assert torch.isnan(step["grad"][1]).all() and torch.isnan(step["grad"][3]).all()
    check_distill(x[4:], t[4:], idx[4:])
    x[1, 0] = float("nan")   # first in its row
    assert torch.isnan(ops.distill_forward(x, t, idx)["loss"][1])


def test_distill_flags_places_past_the_vocabulary():
    g = np.random.default_rng(9)
    x = rand(g, 4, 40)
    t, idx = teacher(g, 4, 40, 3, wide=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = ops.distill_step(x, t, idx, status=status)
    assert status.item() == 0
    far = idx.clone()
    far[2, 1], far[3, 0] = 40, 1 << 40
    got = ops.distill_step(x, t, far, status=status)
    assert status.item() == capi.PER_DEVFLAG_BAD_INDEX
    far[2, 1] = far[3, 0] = -1
    want = ops.distill_step(x, t, far)
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["grad"], want["grad"])
    assert torch.equal(a["loss"][:2], got["loss"][:2])


def test_distill_rows_far_apart():
    """Row offsets past 2^31 elements."""
    g = np.random.default_rng(10)
    v = 1000
    stride = (1 << 31) + 24
    store = torch.empty(stride + v, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((2, v), (stride, 1))
    x.copy_(rand(g, 2, v, kind="bf16"))
    t, idx = teacher(g, 2, v, 4)
    want = ops.distill_step(x.contiguous(), t, idx)
    got = ops.distill_step(x, t, idx, out={"grad": x})
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(x, want["grad"])


def test_distill_runs_alike_twice_and_in_a_graph():
    g = np.random.default_rng(11)
    x = rand(g, 40, 30011, kind="bf16", scale=2.0)
    t, idx = teacher(g, 40, 30011, 64)
    first = ops.distill_step(x, t, idx)
    out = {k: torch.empty_like(z) for k, z in first.items()}
    again = ops.distill_step(x, t, idx, out=out)
    for k in first:
        assert torch.equal(first[k], again[k])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ops.distill_step(x, t, idx, out=out)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = ops.distill_step(x, t, idx)
    for k in want:
        assert torch.equal(want[k], out[k])


def test_distill_loss_in_autograd():
    g = np.random.default_rng(12)
    x = rand(g, 6, 500).requires_grad_()
    t, idx = teacher(g, 6, 500, 7)
    w = rand(g, 6).abs()
    loss = ops.distill_loss(x, t, idx, 2.0)
    (loss * w).sum().backward()
    want = oo.distill(host(x), host(t), host(idx), 2.0, host(w))
    oo.close(f32(loss), want["loss"], want["bloss"])
    oo.close(f32(x.grad), want["grad"], want["bgrad"])


def test_distill_refusals_of_the_binding():
    x, t, i = torch.zeros(4, 10, device="cuda"), torch.zeros(4, 3, device="cuda"), torch.zeros(4, 3, device="cuda").int()
    with pytest.raises(TypeError):
        ops.distill_forward(x.double(), t, i)
    with pytest.raises(TypeError):
        ops.distill_forward(x, t, i.float())
    with pytest.raises(ValueError):
        ops.distill_forward(x, t[:3], i)
    with pytest.raises(ValueError):
        ops.distill_forward(x.t(), t, i)
    with pytest.raises(ValueError):
        ops.distill_forward(x, t, i[:, :2])
    with pytest.raises(ValueError):
        ops.distill_step(x, t, i, row_scale=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        ops.distill_step(x, t, i, out={"grad": torch.zeros(4, 9, device="cuda")})
    with pytest.raises(TypeError):
        ops.distill_backward(x, t, i, None)
    with pytest.raises(ops.PerError):
        ops.distill_forward(x, t, i, temperature=0.0)
    got = ops.distill_step(x[:0], t[:0], i[:0])
    assert got["grad"].shape == (0, 10)


# -- verification ------------------------------------------------------------------------------

def probs(g, b, d, v, kind="f32", noise=0.6):
    x = g.normal(size=(b, d + 1, v)) * 2
    y = x[:, :d] + noise * g.normal(size=(b, d, v))
    soft = lambda z: torch.softmax(torch.from_numpy(z).cuda(), -1).to(TYPES[kind])
    p, q = soft(x), soft(y) if d else torch.empty(b, 0, v, dtype=TYPES[kind], device="cuda")
    tok = torch.multinomial(q.float().reshape(-1, v), 1).reshape(b, d) if d else torch.zeros(b, 0, device="cuda").long()
    u = torch.from_numpy(g.random((b, d)).astype(np.float32)).cuda()
    us = torch.from_numpy(g.random(b).astype(np.float32)).cuda()
    return p, q, tok, u, us


def check_verify(p, q, tok, u, us, lens=None, **kw):
    want = oo.verify(f32(p), None if q is None else f32(q), host(tok), f32(u), f32(us), None if lens is None else host(lens))
    got = ops.verify_draft(p, q, tok, u, us, draft_lens=lens, **kw)
    np.testing.assert_array_equal(got["accepted"].cpu().numpy(), want["accepted"])
    np.testing.assert_array_equal(got["tokens"].cpu().numpy(), want["tokens"])
    # one division of binary32: at most an ulp
    np.testing.assert_allclose(got["accept_p"].cpu().numpy(), want["accept_p"], rtol=2.0 ** -23, atol=0)
    return got


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("b, d, v", [(1, 0, 1), (1, 1, 1), (3, 2, 2), (1, 4, 31), (17, 3, 1000), (5, 8, 4097), (2, 33, 515),
                                     (3, 5, 20011), (2, 2, 65536), (1, 3, 131075), (1, 1, 262144)])
def test_verify(kind, b, d, v):
    g = np.random.default_rng(b + d + v)
    torch.manual_seed(v)
    p, q, tok, u, us = probs(g, b, d, v, kind)
    check_verify(p, q, tok, u, us)
    check_verify(p, None, tok, u, us)
    if d:
        lens = torch.from_numpy(g.integers(-1, d + 2, size=b).astype(np.int32)).cuda()
        check_verify(p, q, tok.int(), u, us, lens)
        check_verify(p, None, tok, u, us, lens)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_verify_many_sequences(kind):
    g = np.random.default_rng(20)
    torch.manual_seed(1)
    p, q, tok, u, us = probs(g, 700, 4, 301, kind, noise=1.0)
    got = check_verify(p, q, tok, u, us)
    seen = got["accepted"].cpu().numpy()
    assert set(seen) == set(range(5))


@pytest.mark.parametrize("us", [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan"), 2.0 ** -40, 0.5])
@pytest.mark.parametrize("v", [5, 10007])
def test_verify_ends_of_the_draw(us, v):
    g = np.random.default_rng(21)
    torch.manual_seed(2)
    p, q, tok, u, _ = probs(g, 3, 2, v)
    u[0] = 1.0
    u[1] = 0.0
    u[2, 0] = float("nan")
    check_verify(p, q, tok, u, torch.full((3,), us, device="cuda"))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("v", [6, 9001])
def test_verify_rows_that_leave_nothing(kind, v):
    """A residual of nothing falls back to the target's row; a target that holds nothing gives -1; NaN,
    negative and infinite masses; masses at the row's ends."""
    dt = TYPES[kind]
    z = lambda *s: torch.zeros(*s, dtype=dt, device="cuda")
    p, q = z(6, 2, v), z(6, 1, v)
    tok = torch.zeros(6, 1, dtype=torch.int64, device="cuda")
    p[0, 0, 2], q[0, 0, 2] = 0.5, 0.5            # refused token 0, residual of nothing: the target's row
    p[1, 0, v - 1], q[1, 0, 0] = 0.25, 1.0       # all of the residual at the last place
    # sequence 2: nothing anywhere
    p[3, 0, 1], p[3, 0, 3], q[3, 0, 0] = float("nan"), INF, 0.5
    p[4, 0, 0], q[4, 0, 0], p[4, 1, 4] = 1.0, 0.5, 1.0   # accepted; then one certain place
    p[5, 0, 1], p[5, 0, 5], q[5, 0, 0] = -1.0, 2.0 ** -14, 1.0
    u = torch.full((6, 1), 0.75, device="cuda")
    us = torch.full((6,), 0.3, device="cuda")
    got = check_verify(p, q, tok, u, us)
    assert got["tokens"][:, 0].tolist() == [2, v - 1, -1, 3, 0, 5] and got["tokens"][4, 1] == 4
    check_verify(p, None, tok, u, us)


def test_verify_tokens_outside_the_vocabulary():
    g = np.random.default_rng(22)
    torch.manual_seed(3)
    p, q, tok, u, us = probs(g, 4, 3, 50)
    u[:] = 0.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_verify(p, q, tok, u, us, status=status)
    assert status.item() == 0
    tok[1, 1], tok[2, 0], tok[3, 2] = 50, -1, 1 << 40
    got = check_verify(p, q, tok, u, us, status=status)
    assert status.item() == capi.PER_DEVFLAG_BAD_INDEX
    assert got["accepted"].tolist() == [3, 1, 0, 2]
    check_verify(p, None, tok, u, us)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad, lead", [(1, 0), (3, 1), (8, 8), (5, 3)])
def test_verify_strides(kind, pad, lead):
    g = np.random.default_rng(23)
    torch.manual_seed(4)
    p, q, tok, u, us = probs(g, 5, 3, 1030, kind)
    want = check_verify(p, q, tok, u, us)
    wide = torch.zeros(5, 7, dtype=tok.dtype, device="cuda")
    wide[:, 2:5] = tok
    got = ops.verify_draft(padded(p, pad, lead), padded(q, pad + 2, lead), wide[:, 2:5], padded(u, 2), us)
    for k in want:
        assert torch.equal(got[k], want[k])
    # positions outermost
    pt = p.transpose(0, 1).contiguous().transpose(0, 1)
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    got = ops.verify_draft(pt, qt, tok, u, us)
    for k in want:
        assert torch.equal(got[k], want[k])


def test_verify_refusals_of_the_binding():
    p, q = torch.zeros(2, 4, 9, device="cuda"), torch.zeros(2, 3, 9, device="cuda")
    t, u, s = torch.zeros(2, 3, device="cuda").int(), torch.zeros(2, 3, device="cuda"), torch.zeros(2, device="cuda")
    ops.verify_draft(p, q, t, u, s)
    with pytest.raises(TypeError):
        ops.verify_draft(p, q.half(), t, u, s)
    with pytest.raises(ValueError):
        ops.verify_draft(p, q[:, :2], t, u, s)
    with pytest.raises(TypeError):
        ops.verify_draft(p, q, t.float(), u, s)
    with pytest.raises(ValueError):
        ops.verify_draft(p, q, t, u[:, :2], s)
    with pytest.raises(TypeError):
        ops.verify_draft(p, q, t, u, None)
    with pytest.raises(TypeError):
        ops.verify_draft(p, q, t, u, s, draft_lens=s)
    assert ops.verify_draft(p[:0], q[:0], t[:0], u[:0], s[:0])["tokens"].shape == (0, 4)


# -- the recurrence ----------------------------------------------------------------------------

def scan_inputs(g, b, t, c, kind="f32", sigmoid=False, p=0.05):
    a = rand(g, b, t, c, kind=kind, scale=1.5, shift=2.0)
    if not sigmoid:
        a = torch.sigmoid(a.float()).to(TYPES[kind])
    resets = torch.from_numpy((g.random((b, t)) < p).astype(np.uint8)).cuda()
    return a, rand(g, b, t, c, kind=kind), rand(g, b, c), resets


def check_scan(a, x, h0, resets, sigmoid, reverse, kind, gh=None, gl=None, back=True):
    gate = ops.GATE_SIGMOID if sigmoid else ops.GATE_DECAY
    hn = lambda z: None if z is None else host(z)
    want = oo.scan(host(a), host(x), hn(h0), hn(resets), sigmoid, reverse)
    got = ops.scan_forward(a, x, h0=h0, resets=resets, gate=gate, reverse=reverse)
    oo.close(f32(got["h"]), want["h"], want["bh"], kind)
    oo.close(f32(got["last"]), want["last"], want["blast"])
    if not back:
        return got
    wb = oo.scan_backward(host(a), host(x), host(got["h"]), host(gh), hn(h0), hn(resets), hn(gl), sigmoid, reverse)
    gb = ops.scan_backward(a, x, got["h"], gh, h0=h0, resets=resets, grad_last=gl, gate=gate, reverse=reverse)
    oo.close(f32(gb["grad_a"]), wb["grad_a"], wb["bgrad_a"], kind)
    oo.close(f32(gb["grad_x"]), wb["grad_x"], wb["bgrad_x"], kind)
    oo.close(f32(gb["grad_h0"]), wb["grad_h0"], wb["bgrad_h0"])
    return {**got, **gb}


SHAPES = [(1, 1, 1), (2, 1, 64), (3, 2, 5), (1, 7, 33), (2, 64, 64), (1, 255, 8), (2, 257, 72), (1, 1000, 130), (3, 129, 1),
          (1, 4100, 16), (2, 2049, 40), (1, 30000, 8), (5, 300, 256)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("b, t, c", SHAPES)
def test_scan(kind, sigmoid, b, t, c):
    g = np.random.default_rng(b + t + c)
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, sigmoid)
    gh, gl = rand(g, b, t, c, kind=kind), rand(g, b, c)
    check_scan(a, x, h0, resets, sigmoid, False, kind, gh, gl)
    check_scan(a, x, None, None, sigmoid, False, kind, gh, None)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("b, t, c", [(1, 1, 3), (2, 66, 64), (1, 341, 1023), (3, 1025, 8), (1, 5000, 24)])
def test_scan_backwards_in_time(kind, sigmoid, b, t, c):
    g = np.random.default_rng(30)
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, sigmoid)
    check_scan(a, x, h0, resets, sigmoid, True, kind, rand(g, b, t, c, kind=kind), rand(g, b, c))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scan_wide(kind):
    """Enough channels to fill the GPU without splitting time."""
    g = np.random.default_rng(31)
    a, x, h0, resets = scan_inputs(g, 9, 70, 4096, kind, True)
    check_scan(a, x, h0, resets, True, False, kind, rand(g, 9, 70, 4096, kind=kind), None)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad, lead, c", [(1, 0, 40), (8, 8, 40), (3, 1, 40), (40, 0, 40), (0, 1, 64), (16, 4, 64)])
def test_scan_strides(kind, pad, lead, c):
    """Rows inside wider rows (gate and input halves of one projection), starts off 16 bytes, time
    outermost."""
    g = np.random.default_rng(32)
    b, t = 2, 150
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, True)
    gh = rand(g, b, t, c, kind=kind)
    want = check_scan(a, x, h0, resets, True, False, kind, gh, None)
    sig = ops.GATE_SIGMOID
    out = {"h": padded(torch.zeros_like(a), pad, lead)}
    got = ops.scan_forward(padded(a, pad, lead), padded(x, pad + 1, lead), h0, resets, sig, out=out)
    # against the definition: the unstrided call's own output is rounded, and may round the other way
    ref = oo.scan(host(a), host(x), host(h0), host(resets), True)
    oo.close(f32(got["h"]), ref["h"], ref["bh"], kind)
    rest = out["h"].as_strided((b * t - 1, pad), (c + pad, 1), lead + c)
    assert (rest == 7).all(), "written between the rows"
    tm = lambda z: z.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros(b, t, 3, dtype=torch.uint8, device="cuda")
    wide[..., 1] = resets
    back = ops.scan_backward(tm(a), tm(x), tm(want["h"]), tm(gh), h0, wide[..., 1], gate=sig,
                             out={"grad_a": tm(torch.zeros_like(a))})
    ref = oo.scan_backward(host(a), host(x), host(want["h"]), host(gh), host(h0), host(resets), None, True)
    for k in ("grad_a", "grad_x"):
        oo.close(f32(back[k]), ref[k], ref["b" + k], kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("b, t, c", [(1, 40, 16), (2, 700, 24), (1, 6000, 64)])
def test_scan_masked_places_may_hold_anything(kind, b, t, c):
    """What a reset or a weight of 0 drops: infinities, NaN, the type's lowest values."""
    g = np.random.default_rng(33)
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, False, p=0.02)
    gh = rand(g, b, t, c, kind=kind)
    cut = t // 2
    x[:, cut - 1] = float("nan")              # the state before an episode's start
    x[:, cut // 2, : c // 2] = INF
    resets[:, cut] = 1
    h0[:] = torch.finfo(torch.float32).min
    resets[:, 0] = 1
    check_scan(a, x, h0, resets, False, False, kind, back=False)
    got = ops.scan_forward(a, x, h0=h0, resets=resets)
    assert torch.isfinite(got["h"][:, cut:].float()).all() and torch.isfinite(got["last"]).all()
    # the same through decays of exactly 0
    z = a.clone()
    z[:, cut] = 0
    z[:, 0] = 0
    check_scan(z, x, h0, None, False, False, kind, back=False)
    # gates: -inf drops the state, +inf the input
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, True)
    a[:, cut] = -INF
    x[:, cut - 1] = float("nan")
    check_scan(a, x, h0, None, True, False, kind, back=False)
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, True)
    a[:, 3:cut] = INF
    x[:, 3:cut] = float("nan")
    x[:, 5] = INF
    check_scan(a, x, h0, None, True, False, kind, gh, None)
    # backward: the stored state before a reset is not read
    a, x, h0, resets = scan_inputs(g, b, t, c, kind, False)
    h = ops.scan_forward(a, x, h0=h0, resets=resets)["h"]
    resets[:, cut] = 1
    resets[:, 0] = 1
    h[:, cut - 1] = float("nan")
    resets[:, cut - 1] = 1
    h0[:] = INF
    if cut >= 2:
        h[:, cut - 2] = -INF
    back = ops.scan_backward(a, x, h, gh, h0=h0, resets=resets)
    want = oo.scan_backward(host(a), host(x), host(h), host(gh), host(h0), host(resets))
    oo.close(f32(back["grad_a"]), want["grad_a"], want["bgrad_a"], kind)
    oo.close(f32(back["grad_h0"]), want["grad_h0"], want["bgrad_h0"])
    assert torch.isfinite(back["grad_a"].float()).all()


def test_scan_nothing_is_dropped_by_underflow():
    """An infinite state stays infinite through decays whose product underflows."""
    a = torch.full((1, 3000, 8), 0.5, device="cuda")
    x = torch.zeros(1, 3000, 8, device="cuda")
    h0 = torch.full((1, 8), INF, device="cuda")
    got = ops.scan_forward(a, x, h0=h0)
    assert torch.isinf(got["h"]).all() and torch.isinf(got["last"]).all()
    h0[:] = 1.0
    got = ops.scan_forward(a, x, h0=h0)
    want = oo.scan(host(a), host(x), host(h0))
    oo.close(f32(got["h"]), want["h"], want["bh"])


def test_scan_long_memories():
    """Decays near 1 over a long sequence: sums of many steps, split over time."""
    g = np.random.default_rng(34)
    a = torch.full((1, 50000, 32), 0.9999, device="cuda")
    x = rand(g, 1, 50000, 32)
    check_scan(a, x, None, None, False, False, "f32", rand(g, 1, 50000, 32), rand(g, 1, 32))
    a[:] = 1.0
    check_scan(a, x, None, None, False, False, "f32", rand(g, 1, 50000, 32), rand(g, 1, 32))


def test_scan_signed_decays():
    g = np.random.default_rng(35)
    a, x, h0, resets = scan_inputs(g, 2, 900, 48)
    a = a * torch.where(rand(g, 2, 900, 48) > 0, 1.0, -1.0)
    check_scan(a, x, h0, resets, False, False, "f32", rand(g, 2, 900, 48), rand(g, 2, 48))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("b, c", [(1, 1), (3, 37), (64, 2048), (130, 1000)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_scan_step(kind, b, c, sigmoid):
    g = np.random.default_rng(b + c)
    a, x, h0, resets = scan_inputs(g, b, 4, c, kind, sigmoid, p=0.3)
    gate = ops.GATE_SIGMOID if sigmoid else ops.GATE_DECAY
    state = h0.clone()
    want = oo.scan(host(a), host(x), host(h0), host(resets), sigmoid)
    for i in range(4):
        got = ops.scan_step(a[:, i], x[:, i], state, resets=resets[:, i], gate=gate, out={"state": state})
        oo.close(f32(got["h"]), want["h"][:, i], want["bh"][:, i], kind)
    oo.close(f32(state), want["last"], want["blast"])
    fresh = ops.scan_step(a[:, 0], x[:, 0], h0, gate=gate)
    assert fresh["state"].data_ptr() != h0.data_ptr()


def test_scan_lengths_of_zero():
    z = torch.zeros(2, 0, 5, device="cuda")
    h0 = torch.arange(10.0, device="cuda").reshape(2, 5)
    got = ops.scan_forward(z, z, h0=h0)
    assert got["h"].shape == (2, 0, 5) and torch.equal(got["last"], h0)
    assert (ops.scan_forward(z, z)["last"] == 0).all()
    back = ops.scan_backward(z, z, z, z, h0=h0, grad_last=h0)
    assert torch.equal(back["grad_h0"], h0)
    assert ops.scan_forward(z[:0], z[:0])["last"].shape == (0, 5)


def test_scan_steps_far_apart():
    """Step offsets past 2^31 elements."""
    g = np.random.default_rng(36)
    a, x, h0, _ = scan_inputs(g, 1, 3, 16, "bf16", True)
    stride = (1 << 30) + 8
    store = torch.empty(2 * stride + 16, dtype=torch.bfloat16, device="cuda")
    far = store.as_strided((1, 3, 16), (0, stride, 1))
    far.copy_(a)
    want = ops.scan_forward(a, x, h0=h0, gate=ops.GATE_SIGMOID)
    got = ops.scan_forward(far, x, h0=h0, gate=ops.GATE_SIGMOID)
    assert torch.equal(got["h"], want["h"])


def test_scan_last_in_the_place_of_h0():
    g = np.random.default_rng(37)
    a, x, h0, resets = scan_inputs(g, 2, 9000, 64)
    want = ops.scan_forward(a, x, h0=h0, resets=resets)
    state = h0.clone()
    got = ops.scan_forward(a, x, h0=state, resets=resets, out={"last": state})
    assert torch.equal(got["h"], want["h"]) and torch.equal(state, want["last"])


def test_gated_scan_in_autograd():
    g = np.random.default_rng(38)
    a, x, h0, resets = scan_inputs(g, 2, 200, 24, "f32", True)
    gh, gl = rand(g, 2, 200, 24), rand(g, 2, 24)
    for z in (a, x, h0):
        z.requires_grad_()
    h, last = ops.gated_scan(a, x, h0, resets, ops.GATE_SIGMOID)
    ((h * gh).sum() + (last * gl).sum()).backward()
    want = oo.scan_backward(host(a), host(x), host(h), host(gh), host(h0), host(resets), host(gl), True)
    oo.close(f32(a.grad), want["grad_a"], want["bgrad_a"])
    oo.close(f32(x.grad), want["grad_x"], want["bgrad_x"])
    oo.close(f32(h0.grad), want["grad_h0"], want["bgrad_h0"])
    a.grad = None
    h, _ = ops.gated_scan(a, x, None, None, ops.GATE_SIGMOID)
    h.sum().backward()                      # an expanded gradient
    assert torch.isfinite(a.grad).all()


def test_scan_refusals_of_the_binding():
    a, h0 = torch.zeros(2, 5, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
    with pytest.raises(TypeError):
        ops.scan_forward(a, a.half())
    with pytest.raises(ValueError):
        ops.scan_forward(a, a[:, :4])
    with pytest.raises(TypeError):
        ops.scan_forward(a, a, h0=h0.half())
    with pytest.raises(ValueError):
        ops.scan_forward(a, a, h0=torch.zeros(8, 2, device="cuda").t())
    with pytest.raises(TypeError):
        ops.scan_forward(a, a, resets=torch.zeros(2, 5, device="cuda"))
    with pytest.raises(ValueError):
        ops.scan_forward(a, a, gate=7)
    with pytest.raises(ValueError):
        ops.scan_forward(a.transpose(1, 2), a.transpose(1, 2))
    with pytest.raises(ops.PerError):
        ops.scan_backward(a, None, a, a, gate=ops.GATE_SIGMOID)
    with pytest.raises(ops.PerError):
        ops.scan_forward(a, a, out={"h": torch.zeros(1, 1, 8, device="cuda").expand(2, 5, 8)})


# -- streams -----------------------------------------------------------------------------------

def test_operators_on_another_stream():
    """Work on a given stream is ordered there, and its outputs belong to it."""
    g = np.random.default_rng(40)
    x = rand(g, 64, 50000)
    t, idx = teacher(g, 64, 50000, 8)
    a, v, h0, resets = scan_inputs(g, 2, 400, 64)
    want, ws = ops.distill_step(x, t, idx), ops.scan_forward(a, v, h0=h0, resets=resets)
    p, q, tok, u, us = probs(g, 3, 2, 900)
    wv = ops.verify_draft(p, q, tok, u, us)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.distill_step(x, t, idx, stream=s)
    gs = ops.scan_forward(a, v, h0=h0, resets=resets, stream=s)
    gv = ops.verify_draft(p, q, tok, u, us, stream=s)
    s.synchronize()
    for w, o in ((want, got), (ws, gs), (wv, gv)):
        for k in w:
            assert torch.equal(w[k], o[k])
    with torch.cuda.stream(s):
        again = ops.distill_step(x, t, idx)
    s.synchronize()
    assert torch.equal(again["grad"], want["grad"])


def test_operators_in_a_graph():
    g = np.random.default_rng(41)
    a, x, h0, resets = scan_inputs(g, 2, 5000, 64, "bf16", True)
    p, q, tok, u, us = probs(g, 8, 3, 4000)
    state = h0.clone()
    sig = ops.GATE_SIGMOID
    so, vo = ops.scan_forward(a, x, h0=state, resets=resets, gate=sig), ops.verify_draft(p, q, tok, u, us)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ops.scan_forward(a, x, h0=state, resets=resets, gate=sig, out=so)
        ops.verify_draft(p, q, tok, u, us, out=vo)
    x.neg_()
    us.copy_(1 - us)
    graph.replay()
    torch.cuda.synchronize()
    want = ops.scan_forward(a, x, h0=h0, resets=resets, gate=sig)
    assert torch.equal(so["h"], want["h"])
    check_verify(p, q, tok, u, us)
    assert torch.equal(vo["tokens"], ops.verify_draft(p, q, tok, u, us)["tokens"])
