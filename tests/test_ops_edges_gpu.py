"""The operators where finite inputs overflow on the way, where waits run out, on other streams, and under
torch.autograd beyond the first derivative.  Bounds come from tests/ops_oracle.py or are derived beside
each test; U is half an ulp of binary32, relative."""
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


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    capi.load()


def host(t):
    return t.detach().to(torch.float64 if t.dtype.is_floating_point else torch.int64).cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def rand(g, *shape, kind="f32"):
    return torch.from_numpy(g.normal(size=shape).astype(np.float32)).cuda().to(TYPES[kind])


# -- sums that overflow before a reset ---------------------------------------------------------

# first large step, second, reset: on both sides of a lane's 8 (or 16) steps, the reset one group of lanes later or more
OVERFLOWS = [(7, 8, 18), (3, 12, 20), (7, 8, 24), (0, 15, 31), (15, 16, 33), (15, 16, 36), (14, 47, 50), (7, 24, 31), (31, 32, 42)]


def overflow_case(g, b, t, c, kind, decay):
    """Sequence r holds a pattern at the front, in the middle or at the end; and the place from which each sequence
    counts from 0 again."""
    a = torch.full((b, t, c), decay, device="cuda").to(TYPES[kind])
    x = rand(g, b, t, c, kind=kind)
    resets = torch.zeros(b, t, dtype=torch.uint8, device="cuda")
    low = torch.finfo(TYPES[kind]).min
    at = []
    for r in range(b):
        first, then, reset = OVERFLOWS[r % len(OVERFLOWS)]
        base = [0, t // 128 * 64, (t - 51) // 64 * 64][(r + r // len(OVERFLOWS)) % 3]
        x[r, base + first] = low
        x[r, base + then] = low
        resets[r, base + reset] = 1
        at.append(base + reset)
    return a, x, resets, at


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [1.0, 0.99, 0.75, 2.0 ** -13])
@pytest.mark.parametrize("b, t, c", [(27, 64, 8), (27, 200, 16), (27, 3000, 16), (54, 128, 1024), (3, 9000, 33)])
def test_scan_a_reset_drops_a_state_that_overflowed(kind, decay, b, t, c):
    """Finite inputs whose sum is infinite, and a reset after them: what follows counts from 0."""
    g = np.random.default_rng(50)
    a, x, resets, at = overflow_case(g, b, t, c, kind, decay)
    for reverse in (False, True):
        turn = (lambda z: z.flip(1)) if reverse else (lambda z: z)
        got = ops.scan_forward(turn(a), turn(x), resets=turn(resets), reverse=reverse)
        h = turn(got["h"])
        for r in range(b):
            part = slice(at[r], None)
            want = oo.scan(host(a[r:r + 1, part]), host(x[r:r + 1, part]), None, host(resets[r:r + 1, part]))
            oo.close(f32(h[r:r + 1, part]), want["h"], want["bh"], kind)
            oo.close(f32(got["last"][r:r + 1]), want["last"], want["blast"])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("b, t, c", [(27, 64, 8), (27, 200, 16), (27, 3000, 16), (54, 128, 1024), (3, 9000, 33)])
def test_scan_a_reset_drops_a_gradient_that_overflowed(kind, sigmoid, b, t, c):
    g = np.random.default_rng(51)
    a, gh, resets, at = overflow_case(g, b, t, c, kind, 20.0 if sigmoid else 1.0)   # (a gate of 20: a weight next to 1)
    # the gradient runs from the last step on
    a, gh, resets = a.flip(1), gh.flip(1), resets.flip(1)
    x, h = rand(g, b, t, c, kind=kind), rand(g, b, t, c, kind=kind)
    if not sigmoid:
        x = None
    h0 = rand(g, b, c)
    gate = ops.GATE_SIGMOID if sigmoid else ops.GATE_DECAY
    for reverse in (False, True):
        turn = (lambda z: None if z is None else z.flip(1)) if reverse else (lambda z: z)
        got = ops.scan_backward(turn(a), turn(x), turn(h), turn(gh), h0=h0, resets=turn(resets), gate=gate, reverse=reverse)
        for r in range(b):
            part = slice(None, t - 1 - at[r])      # before the reset
            cut = lambda z: None if z is None else host(z[r:r + 1, part])
            want = oo.scan_backward(cut(a), cut(x), cut(h), cut(gh), host(h0[r:r + 1]), cut(resets), None, sigmoid)
            for k in ("grad_a", "grad_x"):
                oo.close(f32(turn(got[k])[r:r + 1, part]), want[k], want["b" + k], kind)
            oo.close(f32(got["grad_h0"][r:r + 1]), want["grad_h0"], want["bgrad_h0"])


def test_scan_an_infinite_sum_outlasts_underflow():
    """16 steps that join to an infinite state, then 16 whose weights' product underflows: no 0 times it."""
    a = torch.ones(2, 96, 8, device="cuda")
    x = torch.zeros_like(a)
    a[:, 16:32] = 1e-5
    x[:, 3] = x[:, 12] = torch.finfo(torch.float32).max
    h = ops.scan_forward(a, x)["h"]
    assert torch.isfinite(h[:, :12]).all() and (h[:, 12:16] == float("inf")).all() and not torch.isnan(h).any()


# -- waits that run out ------------------------------------------------------------------------

def _scan_c(direction, a, x, h, gh, outs, status, **kw):
    """The C call of a pass over contiguous [B, T, C] arrays."""
    import ctypes
    b, t, c = a.shape
    st = (ctypes.c_int64 * 2)(t * c, c)
    sh = capi.per_scan_shape(steps=t, batch=b, channels=c, type=capi.PER_TYPE_F32, d_status=status.data_ptr(), **kw)
    for n in ("a", "x", "h", "gh", "ga", "gx"):
        setattr(sh, "stride_" + n, st)
    stream = torch.cuda.current_stream().cuda_stream
    if direction == "forward":
        s = capi.per_scan_forward(ctypes.byref(sh), a.data_ptr(), x.data_ptr(), None, None, outs[0].data_ptr(),
                                  outs[1].data_ptr(), stream)
    else:
        s = capi.per_scan_backward(ctypes.byref(sh), a.data_ptr(), None, h.data_ptr(), None, None, gh.data_ptr(), None,
                                   outs[0].data_ptr(), outs[2].data_ptr(), outs[1].data_ptr(), stream)
    assert s == capi.PER_OK


@pytest.mark.parametrize("direction", ["forward", "backward"])
@pytest.mark.parametrize("withhold", [1, 2])
@pytest.mark.parametrize("t", [700, 20000])
def test_scan_a_wait_that_runs_out_is_reported(direction, withhold, t):
    """One part of a sequence that is split over CTAs tells the others nothing: the call ends, the status says so, and
    no state looks valid; the next call is right again."""
    g = np.random.default_rng(55)
    a, x, gh = torch.sigmoid(rand(g, 1, t, 16)), rand(g, 1, t, 16), rand(g, 1, t, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = lambda: [torch.zeros_like(a), torch.zeros(1, 16, device="cuda"), torch.zeros_like(a)]
    h = ops.scan_forward(a, x, status=status)["h"]
    want, bad, got = new(), new(), new()
    _scan_c(direction, a, x, h, gh, want, status)
    assert status.item() == 0
    _scan_c(direction, a, x, h, gh, bad, status, wait_limit_ms=20, withhold=withhold)
    torch.cuda.synchronize()
    assert status.item() == capi.PER_DEVFLAG_TIMEOUT
    assert torch.isnan(bad[0]).all() and torch.isnan(bad[1]).all()
    status.zero_()
    _scan_c(direction, a, x, h, gh, got, status, wait_limit_ms=20)
    assert status.item() == 0
    for i in range(3):
        assert torch.equal(got[i], want[i])


def test_scan_status_of_the_binding():
    g = np.random.default_rng(56)
    a, x = torch.sigmoid(rand(g, 1, 5000, 16)), rand(g, 1, 5000, 16)
    status = torch.full((1,), 8, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = ops.scan_forward(a, x, status=status, stream=s)["h"]
    ops.scan_backward(a, x, h, x, status=status, stream=s)
    s.synchronize()
    assert status.item() == 8                 # bits are set, never cleared
    with pytest.raises(TypeError):
        ops.scan_forward(a, x, status=torch.zeros(1, device="cuda"))


# -- torch.autograd ----------------------------------------------------------------------------

def test_second_derivatives_are_refused():
    """The gradients are constants to autograd: differentiating them again must not pass silently."""
    g = np.random.default_rng(60)
    x = rand(g, 3, 50).requires_grad_()
    t, idx = x.detach().topk(4, dim=1)
    grad, = torch.autograd.grad(ops.distill_loss(x, t, idx).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (grad.square().sum() + x.square().sum()).backward()
    a, v = rand(g, 2, 40, 8).requires_grad_(), rand(g, 2, 40, 8).requires_grad_()
    for gate in (ops.GATE_DECAY, ops.GATE_SIGMOID):
        h, last = ops.gated_scan(a, v, gate=gate)
        grad, = torch.autograd.grad(h.square().sum() + last.sum(), v, create_graph=True)
        with pytest.raises(RuntimeError):
            (grad.square().sum() + v.square().sum()).backward()


def test_a_graph_of_the_backward_pass_that_is_not_used_is_no_error():
    g = np.random.default_rng(63)
    a, v = rand(g, 2, 40, 8).requires_grad_(), rand(g, 2, 40, 8).requires_grad_()
    want = torch.autograd.grad(ops.gated_scan(a, v)[0].sum(), (a, v))
    got = torch.autograd.grad(ops.gated_scan(a, v)[0].sum(), (a, v), create_graph=True)
    for w, o in zip(want, got):
        assert torch.equal(w, o)
    # a path that does not lead through the operator's gradient stays differentiable
    x = rand(g, 3, 50).requires_grad_()
    t, idx = x.detach().topk(4, dim=1)
    z, = torch.autograd.grad(ops.distill_loss(x.detach() * 2, t, idx).sum() + x.square().sum(), x, create_graph=True)
    z.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))


# -- other streams -----------------------------------------------------------------------------

def _cases(g):
    x = rand(g, 32, 40000)
    t, idx = x.topk(4, dim=1)
    a, v, h0 = torch.sigmoid(rand(g, 2, 3000, 256)), rand(g, 2, 3000, 256), rand(g, 2, 256)
    p = torch.softmax(rand(g, 2000, 3, 64), -1)
    tok, u, us = torch.zeros(2000, 2, device="cuda").int(), torch.rand(2000, 2, device="cuda"), torch.rand(2000, device="cuda")
    lse = ops.distill_forward(x, t, idx)["lse"]
    h = ops.scan_forward(a, v)["h"]
    status = dict(status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return {"distill_forward": ((x, t, idx), status), "distill_backward": ((x, t, idx, lse), status),
            "distill_step": ((x, t, idx), status), "verify_draft": ((p, p[:, :2].contiguous(), tok, u, us), status),
            "scan_forward": ((a, v), status), "scan_step": ((v[:, 0], v[:, 0], h0), {}), "scan_backward": ((a, v, h, v), status)}


@pytest.mark.parametrize("name", ["distill_forward", "distill_backward", "distill_step", "verify_draft", "scan_forward", "scan_step",
                                  "scan_backward"])
def test_outputs_given_to_another_stream_are_held(name):
    """The caller drops its own outputs and the status while the other stream has yet to write them: their memory is
    not given out again before it has."""
    args, kw = _cases(np.random.default_rng(70))[name]
    call = getattr(ops, name)
    want = call(*args, **kw)
    out = {k: torch.empty_like(z) for k, z in want.items()}
    kw = {k: z.clone() for k, z in kw.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)             # about 0.1 s
    call(*args, **kw, out=out, stream=s)
    mine = [*out.values(), *kw.values()]
    held = {z.data_ptr(): z.untyped_storage().nbytes() for z in mine}
    sizes = [z.shape for z in mine]
    dtypes = [z.dtype for z in mine]
    del out, mine, kw
    again = [torch.empty(z, dtype=d, device="cuda") for z, d in zip(sizes, dtypes) for _ in range(4)]
    assert not s.query(), "the other stream has already passed the call"
    for z in again:
        for at, n in held.items():
            assert z.data_ptr() + z.untyped_storage().nbytes() <= at or z.data_ptr() >= at + n, "memory given out again"
    s.synchronize()


# -- what binary32 keeps -----------------------------------------------------------------------

@pytest.mark.parametrize("t", [2, 64, 4096])
def test_scan_gates_keep_their_digits(t):
    """f and 1 - f of large gates, each read off a state, for one thread a channel and for tiles.  e = exp(-a) to
    4 U (a power of 2 to 2^-22) and its last product (U), at most once in f as in 1 - f = e f; 1 + e rounded (U), its
    reciprocal to 1 ulp (2 U) and e f rounded (U): 9 U."""
    c = 512
    a = torch.zeros(1, t, c, device="cuda")
    a[0, 0::2] = 80.0                                # a new episode: the state is the input's weight times x
    a[0, 1::2] = torch.linspace(-80, 80, c, device="cuda")
    x = torch.zeros_like(a)
    resets = torch.zeros(1, t, dtype=torch.uint8, device="cuda")
    resets[0, 0::2] = 1
    # 1 - f: a reset, then x = 1
    ones = torch.ones_like(a)
    v = ops.scan_forward(a.flip(1), ones, resets=torch.ones_like(resets), gate=ops.GATE_SIGMOID)["h"]
    e = np.exp(-host(a.flip(1)))
    np.testing.assert_allclose(host(v), e / (1 + e), rtol=9 * oo.U, atol=0)
    # f: a state of 1 (a gate of -80 takes x whole), then x = 0
    a[0, 0::2] = -80.0
    x[0, 0::2] = 1.0
    h = ops.scan_forward(a, x, resets=resets, gate=ops.GATE_SIGMOID)["h"]
    assert (h[0, 0::2] == 1).all()
    f = 1 / (1 + np.exp(-host(a[0, 1::2])))
    np.testing.assert_allclose(host(h[0, 1::2]), f, rtol=9 * oo.U, atol=0)
    # the gradient of x: 1 - f (a reset at each step, so that g = gh)
    back = ops.scan_backward(a, x, h, ones, resets=torch.ones_like(resets), gate=ops.GATE_SIGMOID)
    e = np.exp(-host(a))
    np.testing.assert_allclose(host(back["grad_x"]), e / (1 + e), rtol=9 * oo.U, atol=0)


@pytest.mark.parametrize("tau", [0.05, 0.25, 1.0, 3.0])
@pytest.mark.parametrize("lead", [0, 1])
def test_distill_probabilities_keep_their_digits(tau, lead):
    """The gradient of f32 logits away from the teacher's one entry is tau p, with the normaliser given.  Logits and
    normaliser are whole multiples of 2^-10, so their difference is exact.  The power of 2 is good to 2^-22 (4 U), its
    argument's rounding is made up for, and each product and sum that follows rounds once: 9 U."""
    g = np.random.default_rng(61)
    n, v = 4, 30011
    low = -60 * tau
    x = torch.from_numpy(np.round(g.uniform(low, 0, size=(n, v)) * 1024).astype(np.float32) / 1024).cuda()
    store = torch.zeros(n * v + lead, device="cuda")
    xs = store[lead:].view(n, v)
    xs.copy_(x)
    lse = torch.full((n,), 0.5, device="cuda")
    idx = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    got = ops.distill_backward(xs, torch.zeros(n, 1, device="cuda"), idx, lse, temperature=tau)["grad"]
    tau32 = float(np.float32(tau))
    want = tau32 * np.exp((host(x) - 0.5) / tau32)
    np.testing.assert_allclose(host(got)[:, 1:], want[:, 1:], rtol=9 * oo.U, atol=0)


@pytest.mark.parametrize("tau", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_distill_losses_do_not_lose_digits_to_a_common_offset(kind, tau):
    """The loss does not change with what all logits of a row share.  Everything is a whole multiple of 2^-10 (bf16
    students of 4), so differences from a row's largest are exact.  With y and z those of a teacher's entry and of the
    student there, over tau: q is good to (12 + K) U relative, log q = y - ln S to (2 |y| + 2 ln S + 8 + K) U,
    log p = z - ln s to (2 |z| + 2 ln s + 48) U (1009 terms in groups of about 32), their difference rounds once and so
    do the products and the K sums."""
    g = np.random.default_rng(62)
    n, v, k = 32, 1009, 8
    grid = lambda w, s: np.round(w * s) / s
    if kind == "f32":
        x = grid(g.normal(size=(n, v)) * tau, 1024) + 3000.0
        t = grid(g.normal(size=(n, k)) * tau, 1024) - 2000.0
    else:
        x = grid(g.normal(size=(n, v)) * 4 * tau, 0.25) + 600.0
        t = grid(g.normal(size=(n, k)) * tau, 1024) - 2000.0
    idx = np.stack([g.permutation(v)[:k] for _ in range(n)])
    dev = lambda z, kd="f32": torch.from_numpy(np.asarray(z, np.float32)).cuda().to(TYPES[kd])
    xs, ts = dev(x, kind), dev(t)
    assert (host(xs) == x).all() and (host(ts) == t).all()
    at = torch.from_numpy(idx).int().cuda()
    got = [ops.distill_forward(xs, ts, at, temperature=tau)["loss"], ops.distill_step(xs, ts, at, temperature=tau)["loss"]]
    y = (t - t.max(1, keepdims=True)) / tau
    z = (x - x.max(1, keepdims=True)) / tau
    S, s = np.exp(y).sum(1, keepdims=True), np.exp(z).sum(1, keepdims=True)
    z = np.take_along_axis(z, idx, 1)
    q, lq, lp = np.exp(y) / S, y - np.log(S), z - np.log(s)
    want = tau * tau * (q * (lq - lp)).sum(1)
    d = np.abs(lq - lp)
    off = q * ((13 + k) * d + 2 * np.abs(y) + 2 * np.log(S) + 2 * np.abs(z) + 2 * np.log(s) + 56 + k)
    bound = oo.U * (tau * tau * off.sum(1) + (k + 4) * np.abs(want))
    for loss in got:
        assert (np.abs(host(loss) - want) <= bound).all()


# -- what a gradient does not need -------------------------------------------------------------

@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("t, c", [(1, 5), (300, 40), (9000, 24)])
def test_gated_scan_gradients_of_one_output_or_input_alone(sigmoid, kind, t, c):
    """They are those of the whole call with zeros in the other's place."""
    g = np.random.default_rng(80)
    gate = ops.GATE_SIGMOID if sigmoid else ops.GATE_DECAY
    a = rand(g, 2, t, c, kind=kind)
    a = (a if sigmoid else torch.sigmoid(a)).requires_grad_()
    x, h0, gl = rand(g, 2, t, c, kind=kind).requires_grad_(), rand(g, 2, c).requires_grad_(), rand(g, 2, c)
    h, last = ops.gated_scan(a, x, h0, gate=gate)
    zero = torch.zeros_like(h)
    want = ops.scan_backward(a.detach(), x.detach(), h.detach(), zero, h0=h0.detach(), grad_last=gl, gate=gate)
    for wrt, names in (((a, x, h0), ("grad_a", "grad_x", "grad_h0")), ((x,), ("grad_x",)), ((a,), ("grad_a",)), ((h0,), ("grad_h0",))):
        z = [y.detach().requires_grad_(any(y is w for w in wrt)) for y in (a, x, h0)]
        _, last = ops.gated_scan(*z, gate=gate)
        got = torch.autograd.grad(last, [y for y in z if y.requires_grad], gl)
        for o, n in zip(got, names):
            assert torch.equal(o, want[n])
    h, last = ops.gated_scan(a, x, h0, gate=gate)
    got = torch.autograd.grad(h, (a, x, h0), torch.ones_like(h))
    want = ops.scan_backward(a.detach(), x.detach(), h.detach(), torch.ones_like(h), h0=h0.detach(), gate=gate)
    for o, n in zip(got, ("grad_a", "grad_x", "grad_h0")):
        assert torch.equal(o, want[n])
    for skip in (("grad_a",), ("grad_x", "grad_h0"), ("grad_a", "grad_x", "grad_h0")):
        got = ops.scan_backward(a.detach(), x.detach(), h.detach(), torch.ones_like(h), h0=h0.detach(), gate=gate, skip=skip)
        assert set(got) == set(want) - set(skip)
        for n in got:
            assert torch.equal(got[n], want[n])


def test_gated_scan_keeps_and_writes_only_what_is_needed():
    """A loss on the last state by x alone, with given decays: the backward pass allocates the gradient of x and
    little else, and x itself is not kept for it."""
    g = np.random.default_rng(81)
    a, x = torch.sigmoid(rand(g, 4, 2000, 256)), rand(g, 4, 2000, 256).requires_grad_()
    array = x.numel() * 4
    used = lambda: (torch.cuda.synchronize(), torch.cuda.memory_allocated())[1]
    before = used()
    _, last = ops.gated_scan(a, x * 1.0)              # (the product is dropped after the call)
    assert used() - before < 1.25 * array             # h
    loss = last.sum()
    before = used()
    torch.cuda.reset_peak_memory_stats()
    grad, = torch.autograd.grad(loss, x)
    # the operator's gradient, the product's behind it, and less than a quarter of an array besides
    assert torch.cuda.max_memory_allocated() - before < 2.25 * array
    want = ops.scan_backward(a, None, torch.zeros_like(a), torch.zeros_like(a), grad_last=torch.ones_like(last))
    assert torch.equal(grad, want["grad_x"])


# -- episodes ----------------------------------------------------------------------------------

def test_scan_resets_from_a_buffers_dones():
    """Forwards, the step after a done starts anew; backwards (returns) the done step itself does."""
    g = np.random.default_rng(90)
    b, t, c = 3, 200, 8
    a, x, h0 = rand(g, b, t, c), rand(g, b, t, c), rand(g, b, c)
    dones = torch.from_numpy((g.random((b, t)) < 0.05).astype(np.uint8)).cuda()
    starts = torch.zeros_like(dones)
    starts[:, 1:] = dones[:, :-1]
    got = ops.gated_scan(a, x, h0, resets=starts, gate=ops.GATE_SIGMOID)[0]
    gamma = torch.full((b, t, 1), 0.9, device="cuda")
    returns = ops.scan_forward(gamma, x[..., :1].contiguous(), resets=dones, reverse=True)["h"]
    for r in range(b):
        ends = [i + 1 for i in range(t) if dones[r, i]]
        for first, end in zip([0] + ends, ends + [t]):
            if first == end:
                continue
            part = (slice(r, r + 1), slice(first, end))
            want = oo.scan(host(a[part]), host(x[part]), host(h0[r:r + 1]) if first == 0 else None, None, True)
            oo.close(f32(got[part]), want["h"], want["bh"])
            want = oo.scan(host(gamma[part]), host(x[part][..., :1]), None, None, False, True)
            oo.close(f32(returns[part]), want["h"], want["bh"])


# -- strides where a sequence is split over CTAs -----------------------------------------------

def padded(t, pad, lead):
    """The same values with `pad` elements behind each row of the last axis and `lead` before the first."""
    rows, w = t.numel() // t.shape[-1], t.shape[-1] + pad
    store = torch.full((lead + rows * w,), 7.0, device=t.device).to(t.dtype)
    strides, s = [1], w
    for n in reversed(t.shape[:-1]):
        strides.insert(0, s)
        s *= n
    view = store.as_strided(t.shape, strides, lead)
    view.copy_(t)
    return view


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("b, c, pad, lead", [(1, 64, 8, 8), (1, 64, 1, 0), (1, 64, 0, 3), (2, 37, 3, 1)])
def test_scan_strides_of_long_sequences(kind, sigmoid, reverse, b, c, pad, lead):
    """Long sequences in rows inside wider rows and off 16 bytes, outputs too: nothing between the rows is written."""
    g = np.random.default_rng(95)
    t = 4500
    a, x, gh, h0, gl = (rand(g, b, t, c, kind=kind) * 1.5 + 2 if i == 0 else rand(g, b, t, c, kind=kind) if i < 3 else rand(g, b, c)
                        for i in range(5))
    a = a.to(TYPES[kind]) if sigmoid else torch.sigmoid(a.float()).to(TYPES[kind])
    resets = torch.from_numpy((g.random((b, t)) < 0.01).astype(np.uint8)).cuda()
    gate = ops.GATE_SIGMOID if sigmoid else ops.GATE_DECAY
    kw = dict(gate=gate, reverse=reverse)
    got = ops.scan_forward(padded(a, pad, lead), padded(x, pad + 1, lead), h0, resets,
                           out={"h": padded(torch.zeros_like(a), pad, lead)}, **kw)
    want = oo.scan(host(a), host(x), host(h0), host(resets), sigmoid, reverse)
    oo.close(f32(got["h"]), want["h"], want["bh"], kind)
    oo.close(f32(got["last"]), want["last"], want["blast"])
    back = ops.scan_backward(padded(a, pad, lead), padded(x, pad + 1, lead), got["h"], padded(gh, pad, lead + 1), h0, resets, gl,
                             out={k: padded(torch.zeros_like(a), pad, lead) for k in ("grad_a", "grad_x")}, **kw)
    ref = oo.scan_backward(host(a), host(x), host(got["h"]), host(gh), host(h0), host(resets), host(gl), sigmoid, reverse)
    for k in ("grad_a", "grad_x"):
        oo.close(f32(back[k]), ref[k], ref["b" + k], kind)
    oo.close(f32(back["grad_h0"]), ref["grad_h0"], ref["bgrad_h0"])
    if pad:
        for z in (got["h"], back["grad_a"], back["grad_x"]):
            between = z.as_strided((b * t - 1, pad), (c + pad, 1), lead + c)
            assert (between == 7).all(), "written between the rows"


# -- closed gates next to resets ---------------------------------------------------------------

def shut_case(g, b, t, c, kind, closed):
    """Gates of -inf or -120 (the state is dropped) before a reset in the same lane's steps, and after one."""
    a, x, h0 = rand(g, b, t, c, kind=kind), rand(g, b, t, c, kind=kind), rand(g, b, c)
    resets = torch.zeros(b, t, dtype=torch.uint8, device="cuda")
    for i in range(2, t - 3, 5):
        a[:, i, i % c::7] = closed
        resets[:, i + 1 + i // 5 % 2] = 1
    return a, x, h0, resets


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("closed", [-float("inf"), -120.0])
@pytest.mark.parametrize("b, t, c", [(2, 64, 16), (1, 3000, 40), (64, 100, 1024)])
def test_scan_closed_gates_before_resets(kind, closed, b, t, c):
    g = np.random.default_rng(100)
    a, x, h0, resets = shut_case(g, b, t, c, kind, closed)
    want = oo.scan(host(a), host(x), host(h0), host(resets), True)
    got = ops.scan_forward(a, x, h0, resets, ops.GATE_SIGMOID)
    oo.close(f32(got["h"]), want["h"], want["bh"], kind)
    oo.close(f32(got["last"]), want["last"], want["blast"])
    gh = rand(g, b, t, c, kind=kind)
    back = ops.scan_backward(a, x, got["h"], gh, h0, resets, gate=ops.GATE_SIGMOID)
    ref = oo.scan_backward(host(a), host(x), host(got["h"]), host(gh), host(h0), host(resets), None, True)
    # (slopes below 2^-126 count as 0: they are e^-120 here, and 0)
    for k in ("grad_a", "grad_x"):
        oo.close(f32(back[k]), ref[k], ref["b" + k] + 1e-37, kind)
    oo.close(f32(back["grad_h0"]), ref["grad_h0"], ref["bgrad_h0"])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("held", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("b, t, c", [(2, 64, 16), (1, 3000, 40), (64, 100, 1024)])
def test_scan_dropped_inputs_before_resets(kind, held, b, t, c):
    """A gate of +inf drops its step's input, whatever that holds, with a reset later in the same lane's steps too."""
    g = np.random.default_rng(101)
    a, x, h0, resets = shut_case(g, b, t, c, kind, float("inf"))
    x = torch.where(torch.isinf(a), torch.full_like(x, held), x)
    want = oo.scan(host(a), host(x), host(h0), host(resets), True)
    got = ops.scan_forward(a, x, h0, resets, ops.GATE_SIGMOID)
    assert np.isfinite(want["h"]).all()
    oo.close(f32(got["h"]), want["h"], want["bh"], kind)
    oo.close(f32(got["last"]), want["last"], want["blast"])
    gh = rand(g, b, t, c, kind=kind)
    back = ops.scan_backward(a, x, got["h"], gh, h0, resets, gate=ops.GATE_SIGMOID)
    ref = oo.scan_backward(host(a), host(x), host(got["h"]), host(gh), host(h0), host(resets), None, True)
    for k in ("grad_a", "grad_x"):
        oo.close(f32(back[k]), ref[k], ref["b" + k], kind)
    oo.close(f32(back["grad_h0"]), ref["grad_h0"], ref["bgrad_h0"])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("t", [1, 64, 4096])
def test_scan_lowest_inputs_do_not_overflow(kind, t):
    """1 - f is at most 1: the type's lowest value times it is finite."""
    c = 1024
    low = torch.finfo(TYPES[kind]).min
    a = torch.linspace(-85, -0.5, t * c, device="cuda").view(1, t, c).to(TYPES[kind])
    x = torch.full_like(a, low)
    ones = torch.ones(1, t, dtype=torch.uint8, device="cuda")
    got = ops.scan_forward(a, x, resets=ones, gate=ops.GATE_SIGMOID)
    assert torch.isfinite(got["h"].float()).all() and torch.isfinite(got["last"]).all()
    back = ops.scan_backward(a, x, torch.zeros_like(a), x, resets=ones, gate=ops.GATE_SIGMOID)
    assert torch.isfinite(back["grad_x"].float()).all()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tau", [1.0, 0.3])
@pytest.mark.parametrize("v", [4, 5000, 140001])
def test_distill_rows_masked_by_the_lowest_value(kind, tau, v):
    """A row of lowest values alone has nothing to learn from, as one of -inf; one value above the mask takes all; binary16's
    lowest is a number like others.  Rows between stay as they are."""
    g = np.random.default_rng(110)
    low = torch.finfo(TYPES[kind]).min
    x = rand(g, 6, v, kind=kind)
    t, idx = rand(g, 6, 3), torch.from_numpy(np.stack([g.permutation(v)[:3] for _ in range(6)])).cuda()
    x[1] = low
    x[3] = low
    x[3, ::2] = -float("inf")
    x[4] = low
    x[4, 1] = 2.0
    idx[4] = torch.tensor([1, -1, -1])
    step = ops.distill_step(x, t, idx, temperature=tau)
    fwd = ops.distill_forward(x, t, idx, temperature=tau)
    back = ops.distill_backward(x, t, idx, fwd["lse"], temperature=tau)
    if kind != "f16":
        for r in (1, 3):
            for z in (step["loss"], fwd["loss"], step["grad"], back["grad"]):
                assert (z[r] == 0).all()
    rows = [0, 2, 4, 5] + ([1] if kind == "f16" else [])
    tau32 = float(np.float32(tau))
    want = oo.distill(host(x)[rows], host(t)[rows], host(idx)[rows], tau32)
    for got in (step, fwd):
        oo.close(f32(got["loss"])[rows], want["loss"], want["bloss"])
    for got in (step, back):
        oo.close(f32(got["grad"])[rows], want["grad"], want["bgrad"], kind)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("b, t, c", [(2, 96, 8), (1, 5000, 24), (40, 300, 256)])
def test_scan_infinite_states_keep_their_sign(kind, b, t, c):
    """Through decays of either sign, whose products underflow: the sign of the state is that of the product."""
    g = np.random.default_rng(120)
    a = (0.5 * torch.where(rand(g, b, t, c) > 0, 1.0, -1.0)).to(TYPES[kind])
    x, h0 = rand(g, b, t, c, kind=kind), torch.full((b, c), float("inf"), device="cuda")
    want = torch.cumprod(torch.sign(a.double()), 1) * float("inf")
    got = ops.scan_forward(a, x, h0=h0)
    assert torch.equal(got["h"].double(), want) and torch.equal(got["last"].double(), want[:, -1])
    back = ops.scan_backward(a, None, torch.zeros_like(a), x, grad_last=h0)
    ends = torch.cumprod(torch.sign(a.double()).flip(1), 1).flip(1) * float("inf")       # of w_t ... w_{T-1}
    assert torch.equal(back["grad_h0"].double(), ends[:, 0])
    assert torch.equal(back["grad_x"][:, :-1].double(), ends[:, 1:]) and torch.isinf(back["grad_x"][:, -1]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [0.1, 0.5])
def test_distill_losses_of_lowest_logits_are_finite(kind, tau):
    """The teacher wants what the student masks by its type's lowest value: tau times that is finite, and so is the
    loss (U is taken eight times: the difference, q, its sum and the products)."""
    g = np.random.default_rng(130)
    low = torch.finfo(TYPES[kind]).min
    x = rand(g, 200, 64, kind=kind)
    x[:, 5] = low
    t, idx = rand(g, 200, 3), torch.full((200, 3), 5, dtype=torch.int32, device="cuda")
    want = -float(np.float32(tau)) * low * np.ones(200)
    for call in (ops.distill_forward, ops.distill_step):
        got = call(x, t, idx, temperature=tau)["loss"]
        np.testing.assert_allclose(host(got), want, rtol=8 * oo.U, atol=0)
