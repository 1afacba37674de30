"""The learner's and the actor's operators beside the replay buffer: what is timed and compared.

A replay learner takes a weighted batch, computes a loss per row and writes the losses back as
priorities; the actor that fills the buffer drafts tokens and has them verified.  Three operators:

  distill  loss of a student's logits against a teacher's top logits, its gradient, or both in one
           pass with the rows' importance weights (`rl_infra_gb300.ops.distill_*`)
  verify   drafted tokens against the target's probabilities, from given random numbers
           (`ops.verify_draft`)
  scan     a gated linear recurrence over time, its gradient and its single step (`ops.scan_*`)

`own` chooses between the plain forms below (elementary torch operations in 32 bits, rounded once
at the end) and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
PAD = 16       # one teacher row in PAD is shorter than the others, one in 4 * PAD is empty


# -- the cases --------------------------------------------------------------------------------

def listed():
    return [
        # the priorities of a small replayed batch refreshed: a short odd vocabulary, latency
        dict(name="distill_refresh", op="distill", part="forward", n=32, v=1009, k=8, dtype="f32", tau=1.0),
        # a learner's batch of the DQN workload's size over an odd vocabulary (rows start unaligned)
        dict(name="distill_step_odd", op="distill", part="step", n=1024, v=32001, k=20, dtype="bf16", tau=2.0),
        # the gradient alone, from the saved normalisers, as an autograd backward runs it
        dict(name="distill_backward", op="distill", part="backward", n=512, v=65536, k=64, dtype="f16", tau=1.0),
        # the largest learner step: 8192 replayed positions over a vocabulary of 2^17
        dict(name="distill_step_large", op="distill", part="step", n=8192, v=131072, k=64, dtype="bf16", tau=1.0),
        # one sequence served alone: latency
        dict(name="verify_one", op="verify", b=1, d=4, v=32768, dtype="f32", point=False),
        # a serving batch over an odd vocabulary, in 16 bits
        dict(name="verify_batch", op="verify", b=64, d=7, v=50021, dtype="bf16", point=False),
        # actors of a large rollout
        dict(name="verify_large", op="verify", b=512, d=8, v=131072, dtype="f32", point=False),
        # one token for each of a batch of sequences: latency
        dict(name="scan_step", op="scan", part="step", b=64, t=1, c=2048, dtype="bf16", gate="sigmoid", reverse=False),
        # discounted returns of replayed trajectories, backwards in time (time-major, odd batch)
        dict(name="scan_returns", op="scan", part="forward", b=1, t=341, c=1023, dtype="f32", gate="decay", reverse=True),
        # one long sequence
        dict(name="scan_long", op="scan", part="forward", b=1, t=65537, c=1024, dtype="bf16", gate="sigmoid", reverse=False),
        # the gradient over a batch of replayed sequences with episode ends in them
        dict(name="scan_backward", op="scan", part="backward", b=16, t=2048, c=2048, dtype="bf16", gate="sigmoid", reverse=False),
        # the largest: both passes of a recurrent trunk, given decays, 32 bits
        dict(name="scan_train_large", op="scan", part="train", b=8, t=16384, c=1024, dtype="f32", gate="decay", reverse=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["distill", "distill", "verify", "scan", "scan"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    while True:
        if op == "distill":
            case = dict(op=op, part=rng.choice(["forward", "step", "backward"]), n=_log(rng, 1, 8192),
                        v=_log(rng, 500, 131072), k=_log(rng, 1, 256), dtype=dtype,
                        tau=rng.choice([1.0, 1.0, 2.0, 0.7]))
        elif op == "verify":
            case = dict(op=op, b=_log(rng, 1, 512), d=rng.randint(1, 8), v=_log(rng, 500, 131072), dtype=dtype,
                        point=rng.random() < 0.25)
        else:
            part = rng.choice(["forward", "backward", "train", "step"])
            case = dict(op=op, part=part, b=_log(rng, 1, 64), t=1 if part == "step" else _log(rng, 2, 65536),
                        c=_log(rng, 16, 4096), dtype=dtype, gate=rng.choice(["sigmoid", "decay"]),
                        reverse=part != "step" and rng.random() < 0.25)
            if rng.random() < 0.5:
                case["c"] = max(64, case["c"] // 64 * 64)
        most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
        if work(case)["bytes"] <= most:
            return case


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "distill":
        cells, small = case["n"] * case["v"], case["n"] * (case["k"] * 8 + 8)
        passes = {"forward": 1, "backward": 2, "step": 2}[case["part"]]
        return {"bytes": cells * e * passes + small, "flops": cells * (4 if case["part"] == "forward" else 8)}
    if case["op"] == "verify":
        # a sequence needs the row it stops at, and the draft's row there when it was refused;
        # about one draft in four is refused
        refused = 1.0 - 0.75 ** case["d"]
        rows = case["b"] * (1.0 + (0.0 if case["point"] else refused))
        return {"bytes": int(rows * case["v"] * e) + case["b"] * case["d"] * 16, "flops": int(rows * case["v"] * 3)}
    cells, edge = case["b"] * case["t"] * case["c"], case["b"] * case["c"]
    resets = case["b"] * case["t"]
    fwd = {"bytes": cells * 3 * e + edge * 8 + resets, "flops": cells * 4}
    bwd = {"bytes": cells * (6 if case["gate"] == "sigmoid" else 5) * e + edge * 8 + resets, "flops": cells * 8}
    if case["part"] in ("forward", "step"):
        return fwd
    if case["part"] == "backward":
        return bwd
    # both passes: the forward's output is written once and read once by the gradient
    return {"bytes": fwd["bytes"] + bwd["bytes"], "flops": fwd["flops"] + bwd["flops"]}


# -- the inputs -------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_distill(case, g):
    n, v, k, dt = case["n"], case["v"], min(case["k"], case["v"]), DTYPES[case["dtype"]]
    x = torch.empty(n, v, dtype=dt, device="cuda")
    top = torch.empty(n, k, device="cuda")
    idx = torch.empty(n, k, dtype=torch.int64, device="cuda")
    part = max(1, (1 << 27) // v)
    for r in range(0, n, part):      # the teacher agrees with the student up to noise
        m = min(part, n - r)
        x[r:r + m] = (2.0 * _randn(g, m, v)).to(dt)
        t = 0.8 * x[r:r + m].float() + 1.5 * _randn(g, m, v)
        top[r:r + m], idx[r:r + m] = t.topk(k, dim=1)
    idx = idx.to(torch.int32)
    row = torch.arange(n, device="cuda")
    keep = torch.where(row % PAD == PAD - 1, k // 2 + (k == 1), k)
    keep = torch.where(row % (4 * PAD) == 4 * PAD - 2, 0, keep)
    idx = torch.where(torch.arange(k, device="cuda") < keep[:, None], idx, -1)
    # importance weights of a prioritized batch, over the batch's size
    scale = torch.rand(n, generator=g, device="cuda").clamp_(0.05).pow_(0.4) / n
    if case["dtype"] == "f16":       # 16-bit gradients with a narrow exponent are trained with a loss scale
        scale *= 4096.0
    state = dict(case=case, x=x, top=top, idx=idx, scale=scale)
    if case["part"] == "backward":
        m = torch.empty(n, device="cuda")
        for r in range(0, n, part):
            m[r:r + part] = case["tau"] * torch.logsumexp(x[r:r + part].float() / case["tau"], dim=1)
        state["lse"] = m
    return state


def _prepare_verify(case, g):
    b, d, v, dt = case["b"], case["d"], case["v"], DTYPES[case["dtype"]]
    p = torch.empty(b, d + 1, v, dtype=dt, device="cuda")
    q = None if case["point"] else torch.empty(b, d, v, dtype=dt, device="cuda")
    tokens = torch.empty(b, d, dtype=torch.int64, device="cuda")
    for r in range(b):               # the draft's distribution is the target's with noise
        x = 3.0 * _randn(g, d + 1, v)
        p[r] = torch.softmax(x, dim=1).to(dt)
        w = torch.softmax(x[:d] + 0.6 * _randn(g, d, v), dim=1)
        if q is None:
            tokens[r] = w.argmax(dim=1)
        else:
            q[r] = w.to(dt)
            tokens[r] = torch.multinomial(q[r].float(), 1, generator=g).squeeze(1)
    lens = torch.full((b,), d, dtype=torch.int32, device="cuda")
    lens[3::8] = d // 2              # some sequences drafted fewer
    return dict(case=case, p=p, q=q, tokens=tokens.to(torch.int32), lens=lens,
                u=torch.rand(b, d, generator=g, device="cuda"), us=torch.rand(b, generator=g, device="cuda"))


def _prepare_scan(case, g):
    b, t, c, dt = case["b"], case["t"], case["c"], DTYPES[case["dtype"]]
    gate = case["gate"]
    z = _randn(g, b, t, c).mul_(1.5).add_(2.0)
    a = (z if gate == "sigmoid" else torch.sigmoid_(z)).to(dt)
    x = _randn(g, b, t, c).to(dt)
    h0 = _randn(g, b, c)
    resets = (torch.rand(b, t, generator=g, device="cuda") < 1.0 / 256).to(torch.uint8)
    state = dict(case=case, a=a, x=x, h0=h0, resets=resets)
    if case["part"] in ("backward", "train"):
        state["gh"] = _randn(g, b, t, c).to(dt)
        state["gl"] = _randn(g, b, c)
    if case["part"] == "backward":   # the forward pass's output, which the gradient reads
        state["h"] = _plain_scan(a, x, h0, resets, gate, case["reverse"])["h"]
    return state


def prepare(case, seed):
    g = _gen(seed)
    return {"distill": _prepare_distill, "verify": _prepare_verify, "scan": _prepare_scan}[case["op"]](case, g)


# -- the plain forms --------------------------------------------------------------------------

def _plain_distill(x, top, idx, tau, scale, lse, grad):
    valid = idx >= 0
    at = idx.clamp_min(0).long()
    some = valid.any(1)
    t = torch.where(valid, top, -math.inf)
    t = t - torch.where(some, t.max(1).values, 0.0)[:, None]
    q = torch.exp(t / tau)
    mass = q.sum(1).clamp_min(1e-30)
    q = q / mass[:, None]
    logq = torch.where(valid, t / tau - torch.log(mass)[:, None], 0.0)
    xf = x.float()
    out = {}
    if lse is None:
        m = xf.max(1).values
        lse = m + tau * torch.log(torch.exp((xf - m[:, None]) / tau).sum(1))
        logp = (xf.gather(1, at) - lse[:, None]) / tau
        out["loss"] = tau * tau * torch.where(valid, q * (logq - logp), 0.0).sum(1)
        out["lse"] = lse
    if grad:
        p = torch.exp((xf - lse[:, None]) / tau)
        p = p * some[:, None]
        p = p.scatter_add(1, at, torch.where(valid, -q, 0.0))
        out["grad"] = (p * (tau * scale)[:, None]).to(x.dtype)
    return out


def _plain_verify(p, q, tokens, lens, u, us):
    b, d = tokens.shape
    at = tokens.long()[..., None]
    pt = p[:, :d].gather(2, at)[..., 0].float()
    qt = torch.ones_like(pt) if q is None else q.gather(2, at)[..., 0].float()
    within = torch.arange(d, device=p.device) < lens[:, None]
    n = ((u * qt < pt) & within).long().cumprod(1).sum(1)
    row = torch.arange(b, device=p.device)
    r = p[row, n].float()
    refused = n < lens
    stop = n.clamp_max(d - 1)
    if q is None:
        point = torch.zeros_like(r).scatter(1, at[row, stop], 1.0)
        r = torch.where(refused[:, None], r * (1.0 - point), r)
    else:
        r = r - torch.where(refused[:, None], q[row, stop].float(), 0.0)
    units = (r.clamp(0.0, 1.0) * 2.0 ** 40).long()
    # no mass left: the target's own row
    sums = torch.where((units > 0).any(1, keepdim=True), units,
                       (p[row, n].float().clamp(0.0, 1.0) * 2.0 ** 40).long()).cumsum(1)
    total = sums[:, -1]
    w = (us * 2.0 ** 31).long()
    mark = w * (total >> 31) + ((w * (total & 0x7fffffff)) >> 31)
    drawn = (sums <= mark[:, None]).sum(1)
    place = torch.arange(d + 1, device=p.device)
    out = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(place < n[:, None], out, torch.where(place == n[:, None], drawn[:, None].int(), -1))
    ratio = torch.where(pt < qt, pt / qt, 1.0)
    return {"accepted": n.int(), "tokens": out.int(), "accept_p": torch.where(within, ratio, 0.0)}


def _doubling(a, x):
    """h_t = a_t h_{t-1} + x_t along dim 1 (h_{-1} = 0), by doubling the stretch each step."""
    d, t = 1, x.shape[1]
    while d < t:
        x = torch.cat([x[:, :d], x[:, d:] + a[:, d:] * x[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return x


def _weights(a, x, resets, gate):
    if gate == "sigmoid":
        f, v = torch.sigmoid(a.float()), torch.sigmoid(-a.float()) * x.float()
    else:
        f, v = a.float(), x.float()
    return torch.where(resets[..., None] != 0, 0.0, f), f, v


def _plain_states(a, x, h0, resets, gate, reverse):
    w, f, v = _weights(a, x, resets, gate)
    if reverse:
        w, v = w.flip(1), v.flip(1)
    v = torch.cat([v[:, :1] + w[:, :1] * h0[:, None], v[:, 1:]], 1)
    return _doubling(w, v)


def _plain_scan(a, x, h0, resets, gate, reverse):
    h = _plain_states(a, x, h0, resets, gate, reverse)
    last = h[:, -1].clone()
    return {"h": (h.flip(1) if reverse else h).to(a.dtype), "last": last}


def _plain_scan_backward(a, x, h, h0, resets, gh, gl, gate, reverse):
    """`h`: in time's direction of the pass (flipped where reverse), 32 bits."""
    w, f, v = _weights(a, x, resets, gate)
    keep, g, xf = (resets == 0)[..., None].float(), gh.float(), x.float()
    if reverse:
        w, f, keep, g, xf = w.flip(1), f.flip(1), keep.flip(1), g.flip(1), xf.flip(1)
    g = torch.cat([g[:, :-1], g[:, -1:] + gl[:, None]], 1)
    later = torch.cat([w[:, 1:], torch.zeros_like(w[:, :1])], 1)
    g = _doubling(later.flip(1), g.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1) * keep
    if gate == "sigmoid":
        ga, gx = g * (before - xf) * f * (1.0 - f), g * (1.0 - f)
    else:
        ga, gx = g * before, g
    gh0 = w[:, 0] * g[:, 0]
    if reverse:
        ga, gx = ga.flip(1), gx.flip(1)
    return {"grad_a": ga.to(a.dtype), "grad_x": gx.to(x.dtype), "grad_h0": gh0}


def _plain(s):
    case = s["case"]
    if case["op"] == "distill":
        return _plain_distill(s["x"], s["top"], s["idx"], case["tau"], s["scale"], s.get("lse"),
                              case["part"] != "forward")
    if case["op"] == "verify":
        return _plain_verify(s["p"], s["q"], s["tokens"], s["lens"], s["u"], s["us"])
    gate, reverse, part = case["gate"], case["reverse"], case["part"]
    a, x, h0, resets = s["a"], s["x"], s["h0"], s["resets"]
    if part in ("forward", "step"):
        return _plain_scan(a, x, h0, resets, gate, reverse)
    if part == "backward":
        h = s["h"].float()
        return _plain_scan_backward(a, x, h.flip(1) if reverse else h, h0, resets, s["gh"], s["gl"], gate, reverse)
    h = _plain_states(a, x, h0, resets, gate, reverse)
    back = _plain_scan_backward(a, x, h, h0, resets, s["gh"], s["gl"], gate, reverse)
    return {"h": (h.flip(1) if reverse else h).to(a.dtype), "last": h[:, -1].clone(), **back}


# -- the library's calls ----------------------------------------------------------------------

def _own(s):
    from rl_infra_gb300 import ops
    case = s["case"]
    if case["op"] == "distill":
        part, tau = case["part"], case["tau"]
        if part == "forward":
            return ops.distill_forward(s["x"], s["top"], s["idx"], temperature=tau)
        if part == "step":
            return ops.distill_step(s["x"], s["top"], s["idx"], s["scale"], temperature=tau)
        return ops.distill_backward(s["x"], s["top"], s["idx"], s["lse"], s["scale"], temperature=tau)
    if case["op"] == "verify":
        return ops.verify_draft(s["p"], s["q"], s["tokens"], s["u"], s["us"], draft_lens=s["lens"])
    gate = ops.GATE_SIGMOID if case["gate"] == "sigmoid" else ops.GATE_DECAY
    part, reverse = case["part"], case["reverse"]
    a, x, h0, resets = s["a"], s["x"], s["h0"], s["resets"]
    if part == "step":
        got = ops.scan_step(a[:, 0], x[:, 0], h0, resets=resets[:, 0], gate=gate)
        return {"h": got["h"][:, None], "last": got["state"]}
    if part == "backward":
        return ops.scan_backward(a, x, s["h"], s["gh"], h0=h0, resets=resets, grad_last=s["gl"], gate=gate,
                                 reverse=reverse)
    got = ops.scan_forward(a, x, h0=h0, resets=resets, gate=gate, reverse=reverse)
    if part == "forward":
        return got
    back = ops.scan_backward(a, x, got["h"], s["gh"], h0=h0, resets=resets, grad_last=s["gl"], gate=gate,
                             reverse=reverse)
    return {**got, **back}


def run(state):
    return _own(state) if own else _plain(state)


# -- the definitions in 64 bits ---------------------------------------------------------------

def _exact_distill(s):
    case = s["case"]
    tau, n, part = case["tau"], case["n"], case["part"]
    want = {"forward": ("loss", "lse"), "backward": ("grad",), "step": ("loss", "lse", "grad")}[part]
    out = {"loss": torch.zeros(n, dtype=torch.float64, device="cuda"),
           "lse": torch.zeros(n, dtype=torch.float64, device="cuda")}
    # the gradient fits only rounded to 32 bits at the largest sizes; far finer than its own type
    grad = torch.empty(s["x"].shape, dtype=torch.float32 if s["x"].numel() > 1 << 28 else torch.float64,
                       device="cuda") if part != "forward" else None
    step = max(1, (1 << 25) // case["v"])
    for r in range(0, n, step):
        rows = slice(r, min(n, r + step))
        y = s["x"][rows].double() / tau
        idx, t = s["idx"][rows].long(), s["top"][rows].double() / tau
        ok = idx >= 0
        none = ~ok.any(1)
        teacher = torch.where(ok, t, -torch.inf).softmax(1).masked_fill(~ok, 0.0)
        if part == "backward":
            norm = s["lse"][rows].double() / tau
        else:
            norm = torch.logsumexp(y, 1)
        logp = y - norm[:, None]
        here = torch.where(ok, idx, 0)
        term = torch.where(teacher > 0, teacher * (torch.where(teacher > 0, teacher, 1.0).log() - logp.gather(1, here)), 0.0)
        out["loss"][rows] = tau ** 2 * term.sum(1)
        out["lse"][rows] = tau * norm
        if grad is not None:
            d = logp.exp()
            d[none] = 0.0
            d.scatter_add_(1, here, -teacher)
            grad[rows] = (d * (tau * s["scale"][rows].double())[:, None]).to(grad.dtype)
    out["grad"] = grad
    return {k: out[k] for k in want}


def _exact_verify(s):
    case = s["case"]
    d = case["d"]
    at = s["tokens"].long()
    rows = torch.arange(case["b"], device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    target = s["p"][rows[0], rows[1], at].double()
    draft = torch.ones_like(target) if s["q"] is None else s["q"][rows[0], rows[1], at].double()
    share = torch.where(draft > target, target / draft, torch.ones_like(target))
    share[rows[1].expand_as(share) >= s["lens"][:, None]] = 0.0
    return {"accepted": None, "tokens": None, "accept_p": share}     # the others are whole numbers


def _exact_scan(s):
    case = s["case"]
    b, t, c, part = case["b"], case["t"], case["c"], case["part"]
    if t * (1 if part in ("forward", "step") else 3) > 250000 or b * t * c > 1 << 28:
        return None
    order = range(t - 1, -1, -1) if case["reverse"] else range(t)
    gated = case["gate"] == "sigmoid"

    def at(i):
        f, v = s["a"][:, i].double(), s["x"][:, i].double()
        f = 1.0 / (1.0 + torch.exp(-f)) if gated else f
        return f, v, (s["resets"][:, i] == 0).double()[:, None]

    out = {}
    if part != "backward":
        all_h, h = torch.empty(b, t, c, dtype=torch.float64, device="cuda"), s["h0"].double()
        for i in order:
            f, v, keep = at(i)
            h = f * keep * h + ((1.0 - f) * v if gated else v)
            all_h[:, i] = h
        out["h"], out["last"] = all_h, h
    if part in ("backward", "train"):
        all_h = s["h"].double() if part == "backward" else all_h
        ga, gx = (torch.empty(b, t, c, dtype=torch.float64, device="cuda") for _ in range(2))
        carry = s["gl"].double()
        steps = list(order)
        for n in range(t - 1, -1, -1):
            i = steps[n]
            f, v, keep = at(i)
            before = keep * (all_h[:, steps[n - 1]] if n else s["h0"].double())
            g = s["gh"][:, i].double() + carry
            ga[:, i] = g * (before - v) * f * (1.0 - f) if gated else g * before
            gx[:, i] = g * (1.0 - f) if gated else g
            carry = f * keep * g
        out.update(grad_a=ga, grad_x=gx, grad_h0=carry)
    return out


def exact(case, seed):
    return {"distill": _exact_distill, "verify": _exact_verify, "scan": _exact_scan}[case["op"]](prepare(case, seed))
