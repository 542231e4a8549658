"""The operators of a recurrent layer body and of the end of its training step,
as measured cases: the layer norm ahead of the body's projection, the gated
linear recurrence that mixes its tokens (prompts, single tokens, gradients),
and the global norm of a list of gradients with their clipping.

``own`` selects what ``run`` does: the plain form (elementary torch
operations in 32 bits, rounded once at the end) or the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D_MODEL = 7168                      # hidden size of the stack workloads
EPS = 1e-5
CHUNK = 64                          # tokens between two states that a forward keeps for its backward
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed() -> list[dict]:
    return [
        # a decode batch of 64 tokens ahead of its projection: a call of a few microseconds
        dict(name="layer norm T64", op="ln", t=64, d=D_MODEL, dtype="bf16", bias=True, wide=False),
        # a long prompt at the stack's width
        dict(name="layer norm T16384", op="ln", t=16384, d=D_MODEL, dtype="bf16", bias=True, wide=False),
        # a small research model in 32 bits, its rows a slice of wider ones that start anywhere
        dict(name="layer norm odd fp32", op="ln", t=2047, d=1003, dtype="fp32", bias=False, wide=True),
        # one training step's gradients at the stack's width, gain and bias among them
        dict(name="layer norm backward T8192", op="ln_bwd", t=8192, d=D_MODEL, dtype="bf16", bias=True, wide=False),
        # the same of a small model of odd width
        dict(name="layer norm backward odd", op="ln_bwd", t=301, d=517, dtype="bf16", bias=True, wide=False),
        # one long prompt at the stack's width, with an output gate
        dict(name="gated recurrence T16384", op="gr", t=16384, seqs=1, c=D_MODEL, dtype="bf16", gate=True,
             initial=False),
        # a serving batch of ragged prompts that go on from earlier states, in 32 bits
        dict(name="gated recurrence ragged", op="gr", t=5003, seqs=37, c=1000, dtype="fp32", gate=False,
             initial=True),
        # forward and gradients of a packed training batch
        dict(name="gated recurrence training", op="gr_train", t=8192, seqs=5, c=4096, dtype="bf16", gate=True,
             initial=True),
        # one user's next token: a call of a few microseconds
        dict(name="gated recurrence step B1", op="gr_step", b=1, slots=8, c=D_MODEL, dtype="bf16", gate=True),
        # the next token of 64 users
        dict(name="gated recurrence step B64", op="gr_step", b=64, slots=80, c=D_MODEL, dtype="bf16", gate=True),
        # the pseudo-queries' gradients of a 93-layer stack, a tensor each: many small tensors
        dict(name="clip 94 pseudo-queries", op="clip", kind="even", tensors=94, total=94 * D_MODEL, dtype="fp32",
             clips=True),
        # the gradients of four layers' bodies: wide projections in 16 bits beside gains and biases in 32
        dict(name="clip 4 layers", op="clip", kind="layers", tensors=4 * 6, total=4 * (4 * D_MODEL * D_MODEL + 6 * D_MODEL),
             dtype="mixed", clips=True),
    ]


def _log(rng: random.Random, lo: int, hi: int, odd: float = 0.4, mult: int = 64) -> int:
    """A size spread over the logarithm of lo..hi: at random, or (1 - odd) a multiple of `mult` where it fits."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and x > mult:
        x = x // mult * mult
    return max(lo, min(hi, x))


def draw(rng: random.Random) -> dict:
    op = rng.choice(["ln", "ln", "ln_bwd", "ln_bwd", "gr", "gr", "gr_train", "gr_train", "gr_step", "clip", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("ln", "ln_bwd"):
        return dict(op=op, t=_log(rng, 1, 8192), d=_log(rng, 16, D_MODEL), dtype=dtype, bias=rng.random() < 0.7,
                    wide=rng.random() < 0.3)
    if op == "clip":
        kind = rng.choice(["even", "uneven", "uneven"])
        tensors = _log(rng, 1, 600, mult=8)
        return dict(op=op, kind=kind, tensors=tensors, total=tensors * _log(rng, 1, 200_000_000 // tensors, mult=512),
                    dtype=rng.choice(["bf16", "fp32", "mixed"]), clips=rng.random() < 0.7)
    c = _log(rng, 16, D_MODEL)
    gate = rng.random() < 0.6
    if op == "gr_step":
        b = _log(rng, 1, 128, mult=8)
        return dict(op=op, b=b, slots=b + rng.randint(0, 16), c=c, dtype=dtype, gate=gate)
    t = _log(rng, 1, 8192 if op == "gr" else 4096)
    return dict(op=op, t=t, seqs=min(t, _log(rng, 1, 48, mult=32)), c=c, dtype=dtype, gate=gate,
                initial=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --

def _lengths(total: int, seqs: int, seed: int) -> list[int]:
    """Sequence lengths of a ragged batch: random cuts, each sequence at least one token."""
    rng = random.Random(seed)
    cuts = sorted(rng.sample(range(1, total), seqs - 1)) if seqs > 1 else []
    ends = cuts + [total]
    return [e - s for s, e in zip([0] + cuts, ends)]


def _tensors(case: dict) -> list[tuple[int, str]]:
    """Elements and type of every tensor of a list of gradients (of the case alone)."""
    n, total, dtype = case["tensors"], case["total"], case["dtype"]
    if case["kind"] == "layers":
        d = D_MODEL
        layer = [(3 * d * d, "bf16"), (d * d, "bf16"), (3 * d, "fp32"), (d, "fp32"), (d, "fp32"), (d, "fp32")]
        return layer * (n // len(layer))
    if case["kind"] == "even":
        sizes = [total // n] * n
    else:  # a few large tensors and many small ones, of any length
        rng = random.Random(1000003 * n + total)
        parts = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(n)]
        sizes = [max(1, int(total * p / sum(parts))) for p in parts]
    return [(m, ("bf16", "fp32")[i % 2] if dtype == "mixed" else dtype) for i, m in enumerate(sizes)]


def prepare(case: dict, seed: int) -> dict:
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    if op == "clip":
        rng = random.Random(int(seed))
        sizes = _tensors(case)
        # gradients of layers differ by orders of magnitude
        scales = [10.0 ** rng.uniform(-4.0, -1.0) for _ in sizes]
        # the tensors of a type lie one behind the other in one buffer, as a program that keeps its gradients has them
        s["flat"] = {t: torch.empty(sum(m for m, u in sizes if u == t), device=dev, dtype=_DT[t])
                     for t in sorted({t for _, t in sizes})}
        s["flat_outs"] = {t: torch.empty_like(x) for t, x in s["flat"].items()}
        s["grads"], s["outs"], at = [], [], dict.fromkeys(s["flat"], 0)
        for (m, t), k in zip(sizes, scales):
            part = slice(at[t], at[t] + m)
            at[t] += m
            s["flat"][t][part] = normal(m, scale=k)
            s["grads"].append(s["flat"][t][part])
            s["outs"].append(s["flat_outs"][t][part])
        s["norm"] = torch.empty(1, device=dev, dtype=torch.float32)
        s["max_norm"] = (0.3 if case["clips"] else 3.0) * math.sqrt(sum(m * k * k for (m, _), k in zip(sizes, scales)))
        return s
    dt = _DT[case["dtype"]]
    if op in ("ln", "ln_bwd"):
        t, d = case["t"], case["d"]
        # rows whose mean is not small beside their spread, as a residual stream's are
        rows = normal(t, d + (5 if case["wide"] else 0)) + normal(t, 1, scale=2.0)
        s["x"] = rows.to(dt)[:, 3:3 + d] if case["wide"] else rows.to(dt)
        s["gain"] = 1.0 + normal(d, scale=0.1)
        s["bias"] = normal(d, scale=0.1) if case["bias"] else None
        s["out"] = torch.empty((t, d), device=dev, dtype=dt)
        if op == "ln_bwd":
            s["grad_out"] = normal(t, d, dtype=dt)
            s["grad_gain"] = torch.empty(d, device=dev, dtype=torch.float32)
            s["grad_bias"] = torch.empty(d, device=dev, dtype=torch.float32) if case["bias"] else None
        return s
    c, gate = case["c"], case["gate"]
    n = case["b"] if op == "gr_step" else case["t"]
    # x, the forget gate and the output gate are slices of one projection's rows; memories of a token to some hundreds
    rows = normal(n, (3 if gate else 2) * c)
    rows[:, c:2 * c].mul_(2.0).add_(2.0)
    rows = rows.to(dt)
    s["x"], s["forget"], s["gate"] = rows[:, :c], rows[:, c:2 * c], rows[:, 2 * c:] if gate else None
    s["out"] = torch.empty((n, c), device=dev, dtype=dt)
    if op == "gr_step":
        s["state"] = normal(case["slots"], c)
        s["slots"] = torch.randperm(case["slots"], generator=g, device=dev)[:n].to(torch.int32)
        return s
    lens = _lengths(n, case["seqs"], int(seed))
    s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    s["initial"] = normal(case["seqs"], c) if case["initial"] else None
    s["final"] = torch.empty((case["seqs"], c), device=dev, dtype=torch.float32)
    if op == "gr_train":
        s["grad_out"] = normal(n, c, dtype=dt)
        s["grad_final"] = normal(case["seqs"], c) if case["initial"] else None
        s["grad_initial"] = torch.empty((case["seqs"], c), device=dev, dtype=torch.float32) if case["initial"] else None
        # the gradients of the projection's rows, side by side as its backward reads them
        grads = torch.empty((n, (3 if gate else 2) * c), device=dev, dtype=dt)
        s["grads"] = (grads[:, :c], grads[:, c:2 * c], grads[:, 2 * c:] if gate else None)
        s["chunk_states"] = torch.empty((-(-n // CHUNK), c), device=dev, dtype=torch.float32)
    return s


# ------------------------------------------------------------ the operators --

def _run_own(s: dict):
    import depth_wise_attention_block_gb300 as A

    c = s["case"]
    op = c["op"]
    if op == "ln":
        A.attnres_layer_norm(s["x"], s["out"], gain=s["gain"], bias=s["bias"], eps=EPS)
        return s["out"]
    if op == "ln_bwd":
        if "workspace" not in s:  # kept with the buffers: made by the first pass
            s["workspace"] = torch.empty(max(256, A.attnres_layer_norm_backward_workspace_size(c["t"], c["d"])),
                                         device="cuda", dtype=torch.uint8)
        A.attnres_layer_norm_backward(s["x"], s["grad_out"], s["out"], gain=s["gain"], grad_gain=s["grad_gain"],
                                      grad_bias=s["grad_bias"], eps=EPS, workspace=s["workspace"])
        return s["out"], s["grad_gain"], s["grad_bias"]
    if op == "clip":
        if "workspace" not in s:
            s["workspace"] = torch.empty(max(256, A.attnres_grad_clip_workspace_size()), device="cuda", dtype=torch.uint8)
        A.attnres_grad_clip(s["grads"], s["max_norm"], s["norm"], outs=s["outs"], workspace=s["workspace"])
        return s["flat_outs"], s["norm"]
    if op == "gr_step":
        A.attnres_gated_recurrence_step(s["x"], s["forget"], s["state"], s["out"], gate=s["gate"], slots=s["slots"])
        return s["out"], s["state"]
    A.attnres_gated_recurrence(s["x"], s["forget"], s["out"], gate=s["gate"], cu_seqlens=s["cu"],
                               initial_state=s["initial"], final_state=s["final"], chunk_states=s.get("chunk_states"))
    if op == "gr":
        return s["out"], s["final"]
    gx, gf, gg = s["grads"]
    A.attnres_gated_recurrence_backward(s["x"], s["forget"], s["chunk_states"], s["grad_out"], gx, gf, gg,
                                        gate=s["gate"], cu_seqlens=s["cu"], initial_state=s["initial"],
                                        grad_final_state=s["grad_final"], grad_initial_state=s["grad_initial"])
    return s["out"], s["final"], s["grads"], s["grad_initial"]


def _scan(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """h_t = a_t h_{t-1} + b_t over the first dimension, by spans that double."""
    k = 1
    while k < a.shape[0]:
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _sigmoids(z: torch.Tensor):
    """1 / (1 + e^-z) and what it lacks to one, neither by a difference."""
    return 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))


def run(s: dict):
    if own:
        return _run_own(s)
    c = s["case"]
    op = c["op"]
    if op == "clip":
        total = sum(x.float().square().sum(dtype=torch.float64) for x in s["grads"])  # long sums
        norm = torch.sqrt(total).float().reshape(1)
        factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
        for x, out in zip(s["grads"], s["outs"]):
            out.copy_(x.float() * factor)
        return s["flat_outs"], norm
    dt = _DT[c["dtype"]]
    if op in ("ln", "ln_bwd"):
        x = s["x"].float()
        x = x - x.mean(-1, keepdim=True)
        rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        hat = x * rstd
        if op == "ln":
            y = hat * s["gain"]
            return (y if s["bias"] is None else y + s["bias"]).to(dt)
        dy = s["grad_out"].float()
        n = dy * s["gain"]
        dx = (n - n.mean(-1, keepdim=True) - hat * (n * hat).mean(-1, keepdim=True)) * rstd
        return dx.to(dt), (dy * hat).sum(0), None if s["bias"] is None else dy.sum(0)
    x = s["x"].float()
    a, rest = _sigmoids(s["forget"].float())
    b = rest * x
    if s["gate"] is not None:
        z = s["gate"].float()
        sig, unsig = _sigmoids(z)
        silu, slope = z * sig, sig * (1 + z * unsig)
    if op == "gr_step":
        at = s["slots"].long()
        h = a * s["state"][at] + b
        s["state"][at] = h
        return (h if s["gate"] is None else h * silu).to(dt), s["state"]
    cu = s["cu"].long()
    first, last = cu[:-1], cu[1:] - 1
    zero = torch.zeros((), device=x.device)
    begin = torch.zeros((c["seqs"], c["c"]), device=x.device) if s["initial"] is None else s["initial"]
    keep = a.clone()
    keep[first] = zero
    b[first] += a[first] * begin
    h = _scan(keep, b)
    out = (h if s["gate"] is None else h * silu).to(dt)
    if op == "gr":
        return out, h[last]
    dy = s["grad_out"].float()
    dh = dy if s["gate"] is None else dy * silu
    dh = dh.clone()
    if s["grad_final"] is not None:
        dh[last] += s["grad_final"]
    before = torch.cat([h[:1], h[:-1]])
    before[first] = begin
    pull = torch.cat([a[1:], a[:1]])
    pull[last] = zero
    dh = _scan(pull.flip(0), dh.flip(0)).flip(0)
    grads = ((rest * dh).to(dt), (dh * (before - x) * a * rest).to(dt),
             None if s["gate"] is None else (dy * h * slope).to(dt))
    return out, h[last], grads, None if s["initial"] is None else a[first] * dh[first]


# -------------------------------------------------------------------- work --

def work(case: dict) -> dict:
    op = case["op"]
    if op == "clip":
        sizes = _tensors(case)
        return {"bytes": sum(2 * m * (2 if t == "bf16" else 4) for m, t in sizes), "flops": sum(3 * m for m, _ in sizes)}
    es = 2 if case["dtype"] == "bf16" else 4
    if op in ("ln", "ln_bwd"):
        t, d = case["t"], case["d"]
        vectors = 4 * d * ((2 if case["bias"] else 1) if op == "ln" else (3 if case["bias"] else 2))
        return {"bytes": es * t * d * (2 if op == "ln" else 3) + vectors, "flops": t * d * (8 if op == "ln" else 17)}
    c, gates = case["c"], 1 if case["gate"] else 0
    if op == "gr_step":
        return {"bytes": case["b"] * c * (8 + es * (3 + gates)), "flops": case["b"] * c * (9 + 6 * gates)}
    t, states = case["t"], 4 * case["seqs"] * c
    if op == "gr":
        return {"bytes": es * t * c * (3 + gates) + states * (2 if case["initial"] else 1), "flops": t * c * (9 + 6 * gates)}
    return {"bytes": es * t * c * (6 + 2 * gates) + states * (4 if case["initial"] else 1),
            "flops": t * c * (20 + 20 * gates)}


# -------------------------------------------- the definitions, in 64 bits --

def exact(case: dict, seed: int):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.nn.functional
    if op == "clip":
        parts = torch.stack([torch.linalg.vector_norm(x, dtype=torch.float64) for x in s["grads"]])
        norm = torch.linalg.vector_norm(parts)
        factor = min(1.0, s["max_norm"] / float(norm))
        return {t: x.double() * factor for t, x in s["flat"].items()}, norm.reshape(1)
    if op in ("ln", "ln_bwd"):
        x, gain = s["x"].double().requires_grad_(), s["gain"].double().requires_grad_()
        bias = None if s["bias"] is None else s["bias"].double().requires_grad_()
        y = f.layer_norm(x, (case["d"],), gain, bias, EPS)
        if op == "ln":
            return y.detach()
        got = torch.autograd.grad(y, (x, gain) if bias is None else (x, gain, bias), s["grad_out"].double())
        return (*got, None) if bias is None else got
    x, z = s["x"].double(), s["forget"].double()
    a, rest = torch.sigmoid(z), torch.sigmoid(-z)
    gate = None if s["gate"] is None else s["gate"].double()
    silu = torch.ones_like(x) if gate is None else f.silu(gate)
    if op == "gr_step":
        out, state = torch.empty_like(x), s["state"].double()
        for row, slot in enumerate(s["slots"].tolist()):
            state[slot] = a[row] * state[slot] + rest[row] * x[row]
            out[row] = state[slot] * silu[row]
        return out, state
    # the recurrence itself, a token at a time
    cu = s["cu"].tolist()
    start = {t: i for i, t in enumerate(cu[:-1])}
    t_all, n = case["t"], case["seqs"]
    h, before = torch.empty_like(x), torch.empty_like(x)
    final = torch.empty((n, case["c"]), device=x.device, dtype=torch.float64)
    add = rest * x
    state = None
    for t in range(t_all):
        if t in start:
            state = torch.zeros_like(x[0]) if s["initial"] is None else s["initial"][start[t]].double()
        before[t] = state
        state = torch.addcmul(add[t], a[t], state, out=h[t])
    for i in range(n):
        final[i] = h[cu[i + 1] - 1]
    out = h * silu
    if op == "gr":
        return out, final
    dy = s["grad_out"].double()
    dh = dy * silu
    grad_initial = None if s["initial"] is None else torch.empty_like(final)
    ends = {cu[i + 1] - 1: i for i in range(n)}
    arriving = None
    for t in range(t_all - 1, -1, -1):
        if t in ends:
            arriving = torch.zeros_like(x[0]) if s["grad_final"] is None else s["grad_final"][ends[t]].double()
        dh[t] += arriving
        arriving = a[t] * dh[t]
        if t in start and grad_initial is not None:
            grad_initial[start[t]] = arriving
    slope = None
    if gate is not None:
        sig = torch.sigmoid(gate)
        slope = sig + gate * sig * torch.sigmoid(-gate)
    return out, final, (rest * dh, dh * (before - x) * a * rest, None if gate is None else dy * h * slope), grad_initial
