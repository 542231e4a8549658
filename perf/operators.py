"""The operators of a layer body that runs between two depth aggregations,
as measured cases: the projection with its fused epilogue, the head norms
with the position rotation, and the linear attention with a decay per head
(prompts, single tokens, gradients).

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
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 64                         # tokens per chunk of the plain scan


# ------------------------------------------------------------------- cases --

def listed() -> list[dict]:
    return [
        # a decode batch of 64 tokens through the fused q, k, v projection
        dict(name="linear decode T64", op="linear", m=64, n=3 * D_MODEL, k=D_MODEL, dtype="bf16", act="none",
             bias=False, residual=False),
        # a prompt of 2048 tokens through a gated-style projection back into the residual stream
        dict(name="linear prefill T2048", op="linear", m=2048, n=D_MODEL, k=D_MODEL, dtype="bf16", act="silu",
             bias=True, residual=True),
        # odd sizes in 32 bits (small research models, odd vocabularies)
        dict(name="linear odd fp32", op="linear", m=301, n=1003, k=517, dtype="fp32", act="gelu", bias=True,
             residual=True),
        # one training step's gradients of an up-projection
        dict(name="linear backward", op="linear_bwd", m=2048, n=D_MODEL, k=2048, dtype="bf16", act="gelu_tanh",
             bias=True, residual=False),
        # the heads of a decode batch: a call of a few microseconds
        dict(name="qk norm rope T64", op="qk", t=64, hq=56, hk=8, d=128, rot=128, interleaved=False, gain=True,
             dtype="bf16"),
        # the heads of a long prompt
        dict(name="qk norm rope T16384", op="qk", t=16384, hq=56, hk=56, d=128, rot=128, interleaved=True, gain=True,
             dtype="bf16"),
        # training in 32 bits with a partly rotated head and grouped key heads
        dict(name="qk norm rope backward", op="qk_bwd", t=2047, hq=24, hk=6, d=96, rot=64, interleaved=False,
             gain=True, dtype="fp32"),
        # one long prompt at the stack's width
        dict(name="linear attention T16384", op="la", t=16384, seqs=1, h=56, dk=128, dv=128, dtype="bf16",
             initial=False),
        # a serving batch of ragged prompts that go on from earlier states, in 32 bits
        dict(name="linear attention ragged", op="la", t=5003, seqs=37, h=16, dk=64, dv=96, dtype="fp32",
             initial=True),
        # gradients of a packed training batch
        dict(name="linear attention backward", op="la_bwd", t=8192, seqs=5, h=32, dk=128, dv=128, dtype="bf16",
             initial=True),
        # one user's next token: a call of a few microseconds
        dict(name="linear attention step B1", op="la_step", b=1, slots=8, h=56, dk=128, dv=128, dtype="bf16"),
        # the next token of 64 users
        dict(name="linear attention step B64", op="la_step", b=64, slots=80, h=56, dk=128, dv=128, dtype="bf16"),
    ]


def _log(rng: random.Random, lo: int, hi: int, odd: float = 0.4, mult: int = 64) -> int:
    """A size spread over the logarithm of lo..hi: at random, or (1 - odd) a multiple of `mult` where it fits."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and x > mult:
        x = x // mult * mult
    return max(lo, min(hi, x))


def draw(rng: random.Random) -> dict:
    op = rng.choice(["linear", "linear", "linear_bwd", "qk", "qk_bwd", "la", "la", "la_bwd", "la_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("linear", "linear_bwd"):
        return dict(op=op, m=_log(rng, 1, 2048), n=_log(rng, 16, D_MODEL), k=_log(rng, 16, 2048 if op == "linear_bwd" else D_MODEL),
                    dtype=dtype, act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.5, residual=op == "linear" and rng.random() < 0.5)
    if op in ("qk", "qk_bwd"):
        d = rng.choice([64, 96, 128, 128, 192, 256, 2 * rng.randint(8, 100)])
        hk = rng.choice([1, 2, 4, 8])
        return dict(op=op, t=_log(rng, 1, 8192), hq=hk * rng.choice([1, 2, 4]), hk=hk, d=d,
                    rot=rng.choice([d, d, d // 4 * 2, 0]), interleaved=rng.random() < 0.5, gain=rng.random() < 0.8,
                    dtype=dtype)
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (96, 96),
                         (rng.randint(8, 160), rng.randint(8, 160))])
    if op == "la_step":
        b = _log(rng, 1, 128, mult=8)
        return dict(op=op, b=b, slots=b + rng.randint(0, 16), h=rng.choice([4, 8, 16, 32, 56]), dk=dk, dv=dv,
                    dtype=dtype)
    t = _log(rng, 1, 8192)
    return dict(op=op, t=t, seqs=min(t, _log(rng, 1, 24, mult=32)), h=rng.choice([1, 2, 4, 8, 16, 24]), dk=dk, dv=dv,
                dtype=dtype, initial=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --

def _lengths(total: int, seqs: int, seed: int) -> list[int]:
    """Sequence lengths of a ragged batch: random cuts, each sequence at least one token."""
    rng = random.Random(seed)
    cuts = sorted(rng.sample(range(1, total), seqs - 1)) if seqs > 1 else []
    ends = cuts + [total]
    return [e - s for s, e in zip([0] + cuts, ends)]


def _slopes(h: int, dev) -> torch.Tensor:
    """Log-decays of the heads, a geometric series from fast to slow forgetting."""
    return -torch.exp2(-8.0 * torch.arange(1, h + 1, device=dev, dtype=torch.float32) / h)


def prepare(case: dict, seed: int) -> dict:
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    s = {"case": dict(case)}
    if op in ("linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = normal(m, k)
        s["w"] = normal(n, k, scale=1.0 / math.sqrt(k))
        s["bias"] = normal(n, scale=0.1, dtype=torch.float32) if case["bias"] else None
        if op == "linear":
            s["residual"] = normal(m, n) if case["residual"] else None
            s["out"] = torch.empty((m, n), device=dev, dtype=dt)
        else:
            s["grad_out"] = normal(m, n)
            s["grads"] = (torch.empty_like(s["x"]), torch.empty_like(s["w"]),
                          torch.empty(n, device=dev, dtype=torch.float32))
        return s
    if op in ("qk", "qk_bwd"):
        t, hq, hk, d, rot = case["t"], case["hq"], case["hk"], case["d"], case["rot"]
        # q and k are slices of one projection's rows (q, k and v side by side)
        rows = normal(t, (hq + 2 * hk) * d)
        s["q"] = rows[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = rows[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        start = torch.randint(0, 1 << 17, (1,), generator=g, device=dev)
        s["positions"] = start + torch.arange(t, device=dev)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / max(rot, 1))).float()
        s["gains"] = tuple(1.0 + normal(d, scale=0.1, dtype=torch.float32) for _ in range(2)) if case["gain"] \
            else (None, None)
        s["outs"] = tuple(torch.empty((t, h, d), device=dev, dtype=dt) for h in (hq, hk))
        if op == "qk_bwd":
            s["grad_outs"] = (normal(t, hq, d), normal(t, hk, d))
            s["grad_gains"] = tuple(torch.empty(d, device=dev, dtype=torch.float32) for _ in range(2)) \
                if case["gain"] else (None, None)
        return s
    h, dk, dv = case["h"], case["dk"], case["dv"]
    s["log_decay"] = _slopes(h, dev)
    if op == "la_step":
        b, slots = case["b"], case["slots"]
        rows = normal(b, h * (2 * dk + dv))
        s["q"], s["k"] = (rows[:, i * h * dk:(i + 1) * h * dk].unflatten(1, (h, dk)) for i in range(2))
        s["v"] = rows[:, 2 * h * dk:].unflatten(1, (h, dv))
        s["state"] = normal(slots, h, dk, dv, dtype=torch.float32)
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:b].to(torch.int32)
        s["out"] = torch.empty((b, h, dv), device=dev, dtype=dt)
        return s
    t, seqs = case["t"], case["seqs"]
    lens = _lengths(t, seqs, seed)
    s["max_len"] = max(lens)
    s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    rows = normal(t, h * (2 * dk + dv))
    s["q"], s["k"] = (rows[:, i * h * dk:(i + 1) * h * dk].unflatten(1, (h, dk)) for i in range(2))
    s["v"] = rows[:, 2 * h * dk:].unflatten(1, (h, dv))
    s["initial"] = normal(seqs, h, dk, dv, dtype=torch.float32) if case["initial"] else None
    if op == "la":
        s["out"] = torch.empty((t, h, dv), device=dev, dtype=dt)
        s["final"] = torch.empty((seqs, h, dk, dv), device=dev, dtype=torch.float32)
    else:
        s["grad_out"] = normal(t, h, dv)
        s["grad_final"] = normal(seqs, h, dk, dv, dtype=torch.float32) if case["initial"] else None
        s["grads"] = tuple(torch.empty((t, h, w), device=dev, dtype=dt) for w in (dk, dk, dv))
        s["grad_initial"] = torch.empty((seqs, h, dk, dv), device=dev, dtype=torch.float32) \
            if case["initial"] else None
    return s


# ------------------------------------------------------------ the operators --

def _kept(s: dict, size) -> torch.Tensor:
    """The workspace that a program keeps with its buffers: made by the first pass."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(256, size()), device="cuda", dtype=torch.uint8)
    return s["workspace"]


def _run_own(s: dict):
    import depth_wise_attention_block_gb300 as A

    c = s["case"]
    op, dt = c["op"], _DT[c["dtype"]]
    if op == "linear":
        ws = _kept(s, lambda: A.attnres_linear_workspace_size(c["m"], c["n"], c["k"], dt))
        A.attnres_linear(s["x"], s["w"], s["out"], bias=s["bias"], residual=s["residual"], activation=c["act"],
                         workspace=ws)
        return s["out"]
    if op == "linear_bwd":
        ws = _kept(s, lambda: A.attnres_linear_backward_workspace_size(c["m"], c["n"], c["k"], dt, c["act"]))
        gx, gw, gb = s["grads"]
        A.attnres_linear_backward(s["x"], s["w"], s["grad_out"], grad_x=gx, grad_w=gw, grad_bias=gb, bias=s["bias"],
                                  activation=c["act"], workspace=ws)
        return s["grads"]
    if op == "qk":
        A.attnres_qk_norm_rope(s["q"], s["k"], s["outs"][0], s["outs"][1], q_gain=s["gains"][0], k_gain=s["gains"][1],
                               positions=s["positions"], inv_freq=s["inv_freq"], interleaved=c["interleaved"], eps=EPS)
        return s["outs"]
    if op == "qk_bwd":
        ws = _kept(s, lambda: A.attnres_qk_norm_rope_backward_workspace_size(c["t"], c["hq"], c["hk"], c["d"]))
        A.attnres_qk_norm_rope_backward(s["q"], s["k"], s["grad_outs"][0], s["grad_outs"][1], s["outs"][0],
                                        s["outs"][1], q_gain=s["gains"][0], k_gain=s["gains"][1],
                                        grad_q_gain=s["grad_gains"][0], grad_k_gain=s["grad_gains"][1],
                                        positions=s["positions"], inv_freq=s["inv_freq"],
                                        interleaved=c["interleaved"], eps=EPS, workspace=ws)
        return s["outs"], s["grad_gains"]
    if op == "la":
        ws = _kept(s, lambda: A.attnres_linear_attention_workspace_size(c["t"], c["h"], c["dk"], c["dv"], dt, c["seqs"]))
        A.attnres_linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["out"], cu_seqlens=s["cu"],
                                   initial_state=s["initial"], final_state=s["final"], workspace=ws)
        return s["out"], s["final"]
    if op == "la_bwd":
        ws = _kept(s, lambda: A.attnres_linear_attention_backward_workspace_size(c["t"], c["h"], c["dk"], c["dv"], dt,
                                                                                 c["seqs"]))
        gq, gk, gv = s["grads"]
        A.attnres_linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["grad_out"], gq, gk, gv,
                                            cu_seqlens=s["cu"], initial_state=s["initial"],
                                            grad_final_state=s["grad_final"], grad_initial_state=s["grad_initial"],
                                            workspace=ws)
        return s["grads"], s["grad_initial"]
    A.attnres_linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["out"], slots=s["slots"])
    return s["out"], s["state"]


def _act(z: torch.Tensor, kind: str) -> torch.Tensor:
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z: torch.Tensor, kind: str) -> torch.Tensor:
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _turn(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, rot: int, interleaved: bool) -> torch.Tensor:
    """The first `rot` channels' pairs turned by (cos, sin) [t, 1, rot / 2]."""
    if rot == 0:
        return x
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _angles(s: dict, dtype: torch.dtype):
    """cos and sin [t, 1, rot / 2], the angles of far positions taken in 64 bits."""
    ang = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def _pack(x: torch.Tensor, rows: torch.Tensor, valid: torch.Tensor) -> torch.Tensor:
    """[t, h, d] rows of a ragged batch as [seqs, h, len, d], zero behind each end."""
    return (x[rows].float() * valid[..., None, None]).transpose(1, 2)


def _scan(a, b, c, g, start, lens):
    """out_i = a_i S_i with S_i = e^g S_{i-1} + b_i c_i^T, and each sequence's last S.

    a, b [n, h, l, da], c [n, h, l, dc], g [h], start [n, h, da, dc] or None, lens [n]; l a multiple of the chunk.
    Chunks: within one by a decayed triangle of products, across them by the chunks' own sums.
    """
    n, h, l, da = a.shape
    dc, m = c.shape[-1], l // _CHUNK
    i = torch.arange(_CHUNK, device=a.device)
    j = torch.arange(m, device=a.device)
    g4 = g.view(1, h, 1, 1, 1)
    ca, cb, cc = a.view(n, h, m, _CHUNK, da), b.view(n, h, m, _CHUNK, da), c.view(n, h, m, _CHUNK, dc)
    ago = (i[:, None] - i[None, :])
    within = torch.where(ago >= 0, torch.exp(g4 * ago.clamp(min=0)), torch.zeros((), device=a.device))
    out = (ca @ cb.transpose(-1, -2) * within) @ cc
    sums = ((cb * torch.exp(g4 * (_CHUNK - 1 - i)[:, None])).transpose(-1, -2) @ cc).view(n, h, m, da * dc)
    gap = j[:, None] - 1 - j[None, :]
    g3 = g.view(1, h, 1, 1)
    across = torch.where(gap >= 0, torch.exp(g3 * (_CHUNK * gap.clamp(min=0))), torch.zeros((), device=a.device))
    before = across @ sums
    if start is not None:
        before = before + torch.exp(g3 * (_CHUNK * j[:, None])) * start.reshape(n, h, 1, da * dc)
    out = out + torch.exp(g4 * (i[:, None] + 1)) * (ca @ before.view(n, h, m, da, dc))
    left = lens.view(n, 1, 1) - 1 - torch.arange(l, device=a.device)
    weight = torch.where(left >= 0, torch.exp(g.view(1, h, 1) * left.clamp(min=0)), torch.zeros((), device=a.device))
    last = (b * weight[..., None]).transpose(-1, -2) @ c
    if start is not None:
        last = last + torch.exp(g.view(1, h, 1, 1) * lens.view(n, 1, 1, 1)) * start
    return out.view(n, h, l, dc), last


def _ragged(s: dict):
    """Where each sequence's padded places lie among the rows, forward and from the end, and back."""
    cu = s["cu"].long()
    lens, t = cu[1:] - cu[:-1], s["q"].shape[0]
    at = torch.arange(-(-s["max_len"] // _CHUNK) * _CHUNK, device=cu.device)
    valid = at < lens[:, None]
    ahead = (cu[:-1, None] + at).clamp(max=t - 1)
    back = (cu[1:, None] - 1 - at).clamp(min=0)
    row = torch.arange(t, device=cu.device)
    seq = torch.searchsorted(cu[1:], row, right=True)
    return lens, valid, ahead, back, seq, row - cu[seq], cu[seq + 1] - 1 - row


def run(s: dict):
    if own:
        return _run_own(s)
    c = s["case"]
    op, dt = c["op"], _DT[c["dtype"]]
    if op in ("linear", "linear_bwd"):
        x, w = s["x"].float(), s["w"].float()
        if op == "linear" or c["act"] != "none":
            z = x @ w.t()
            if s["bias"] is not None:
                z = z + s["bias"]
        if op == "linear":
            y = _act(z, c["act"])
            if s["residual"] is not None:
                y = y + s["residual"].float()
            return y.to(dt)
        dz = s["grad_out"].float()
        if c["act"] != "none":
            dz = dz * _act_slope(z, c["act"])
        return (dz @ w).to(dt), (dz.t() @ x).to(dt), dz.sum(0)
    if op in ("qk", "qk_bwd"):
        cos, sin = _angles(s, torch.float32)
        heads, gains = [], []
        for n in range(2):
            x, gain = (s["q"], s["k"])[n].float(), s["gains"][n]
            rho = torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            hat = x / rho
            if op == "qk":
                heads.append(_turn(hat if gain is None else hat * gain, cos, sin, c["rot"], c["interleaved"]).to(dt))
                continue
            dy = _turn(s["grad_outs"][n].float(), cos, -sin, c["rot"], c["interleaved"])
            dn = dy if gain is None else dy * gain
            heads.append(((dn - hat * (dn * hat).mean(-1, keepdim=True)) / rho).to(dt))
            gains.append(None if gain is None else (dy * hat).sum((0, 1)))
        return tuple(heads) if op == "qk" else (tuple(heads), tuple(gains))
    g = s["log_decay"]
    scale = c["dk"] ** -0.5
    if op == "la_step":
        at = s["slots"].long()
        new = torch.exp(g)[:, None, None] * s["state"][at] + s["k"].float()[..., None] * s["v"].float()[:, :, None, :]
        s["state"][at] = new
        out = scale * (s["q"].float()[:, :, None, :] @ new)[:, :, 0]
        return out.to(dt), s["state"]
    lens, valid, ahead, back, seq, at, from_end = _ragged(s)
    if op == "la":
        q, k, v = (_pack(s[n], ahead, valid) for n in "qkv")
        out, last = _scan(q, k, v, g, s["initial"], lens)
        return (scale * out[seq, :, at]).to(dt), last
    v, k, do = (_pack(x, ahead, valid) for x in (s["v"], s["k"], s["grad_out"]))
    dq, _ = _scan(do, v, k, g, None if s["initial"] is None else s["initial"].transpose(-1, -2), lens)
    q, k, v, do = (_pack(x, back, valid) for x in (s["q"], s["k"], s["v"], s["grad_out"]))
    arriving = None if s["grad_final"] is None else s["grad_final"] / (scale * torch.exp(g)[:, None, None])
    dk, _ = _scan(v, do, q, g, None if arriving is None else arriving.transpose(-1, -2), lens)
    dv, first = _scan(k, q, do, g, arriving, lens)
    grads = (scale * dq[seq, :, at]).to(dt), (scale * dk[seq, :, from_end]).to(dt), (scale * dv[seq, :, from_end]).to(dt)
    return grads, None if s["initial"] is None else scale * torch.exp(g)[:, None, None] * first


# -------------------------------------------------------------------- work --

def work(case: dict) -> dict:
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    op = c["op"]
    if op == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": es * (m * k + n * k + m * n * (2 if c["residual"] else 1)) + (4 * n if c["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "linear_bwd":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": es * (2 * m * k + 2 * n * k + m * n) + 8 * n,
                "flops": (4 if c["act"] == "none" else 6) * m * n * k}
    if op in ("qk", "qk_bwd"):
        x = c["t"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": es * x * (2 if op == "qk" else 3) + 8 * c["t"], "flops": (10 if op == "qk" else 20) * x}
    h, dk, dv = c["h"], c["dk"], c["dv"]
    if op == "la_step":
        return {"bytes": c["b"] * h * (8 * dk * dv + es * (2 * dk + 2 * dv)), "flops": 6 * c["b"] * h * dk * dv}
    t, st = c["t"], 4 * c["seqs"] * h * dk * dv
    if op == "la":
        return {"bytes": es * t * h * (2 * dk + 2 * dv) + st * (2 if c["initial"] else 1), "flops": 4 * t * h * dk * dv}
    return {"bytes": es * t * h * (4 * dk + 3 * dv) + st * (3 if c["initial"] else 0), "flops": 10 * t * h * dk * dv}


# -------------------------------------------- the definitions, in 64 bits --

def _exact_heads(x, gain, positions, inv_freq, interleaved):
    """One head tensor normed and rotated through complex numbers."""
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if gain is not None:
        y = y * gain
    r = 2 * inv_freq.numel()
    if r == 0:
        return y
    pairs = y[..., :r].unflatten(-1, (r // 2, 2)) if interleaved else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous())
    ang = positions.double()[:, None] * inv_freq.double()
    z = z * torch.polar(torch.ones_like(ang), ang)[:, None]
    z = torch.view_as_real(z)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., r:]], -1)


def _exact_act(z, kind):
    f = torch.nn.functional
    return {"none": lambda: z, "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh"), "silu": lambda: f.silu(z)}[kind]()


def exact(case: dict, seed: int):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
        b = (torch.zeros(case["n"], device=x.device) if s["bias"] is None else s["bias"]).double().requires_grad_()
        y = _exact_act(torch.addmm(b, x, w.t()), case["act"])
        if op == "linear":
            return (y if s["residual"] is None else y + s["residual"].double()).detach()
        return torch.autograd.grad(y, (x, w, b), s["grad_out"].double())
    if op in ("qk", "qk_bwd"):
        outs, gains = [], []
        for x, gain, n in ((s["q"], s["gains"][0], 0), (s["k"], s["gains"][1], 1)):
            if op == "qk":
                outs.append(_exact_heads(x.double(), None if gain is None else gain.double(), s["positions"],
                                         s["inv_freq"], case["interleaved"]))
                continue
            x, gain = x.double().requires_grad_(), None if gain is None else gain.double().requires_grad_()
            y = _exact_heads(x, gain, s["positions"], s["inv_freq"], case["interleaved"])
            got = torch.autograd.grad(y, (x,) if gain is None else (x, gain), s["grad_outs"][n].double())
            outs.append(got[0])
            gains.append(None if gain is None else got[1])
        return tuple(outs) if op == "qk" else (tuple(outs), tuple(gains))
    decay = torch.exp(s["log_decay"].double())[:, None, None]
    scale = 1.0 / math.sqrt(case["dk"])
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if op == "la_step":
        out, state = torch.empty_like(v), s["state"].double()
        for row, slot in enumerate(s["slots"].tolist()):
            state[slot] = decay * state[slot] + torch.einsum("hk,hv->hkv", k[row], v[row])
            out[row] = scale * torch.einsum("hk,hkv->hv", q[row], state[slot])
        return out, state
    # the recurrence itself, token by token over all sequences at once; a row behind a sequence's end is not taken
    cu = s["cu"].tolist()
    n, longest = len(cu) - 1, s["max_len"]
    lens = s["cu"][1:].long() - s["cu"][:-1].long()
    first = s["cu"][:-1].long()
    zero = torch.zeros((n, case["h"], case["dk"], case["dv"]), device=q.device, dtype=torch.float64)
    S = zero.clone() if s["initial"] is None else s["initial"].double()
    out, dq = torch.empty_like(v), torch.empty_like(q)
    do = s["grad_out"].double() if op == "la_bwd" else None
    order = torch.argsort(lens, descending=True)
    first, lens, S = first[order], lens[order], S[order]
    alive = [int(x) for x in (lens[None, :] > torch.arange(longest, device=q.device)[:, None]).sum(1).tolist()]
    for i in range(longest):
        m = alive[i]
        r = first[:m] + i
        S[:m] = decay * S[:m] + k[r][..., :, None] * v[r][..., None, :]
        if op == "la":
            out[r] = scale * (q[r][..., None, :] @ S[:m])[..., 0, :]
        else:
            dq[r] = scale * (S[:m] @ do[r][..., :, None])[..., 0]
    back = torch.argsort(order)
    if op == "la":
        return out, S[back]
    # gradients: the state's gradient runs from each sequence's end to its start
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    R = zero.clone() if s["grad_final"] is None else s["grad_final"].double()[order]
    for i in range(longest):
        m = alive[i]
        r = first[:m] + lens[:m] - 1 - i
        R[:m] = R[:m] + scale * q[r][..., :, None] * do[r][..., None, :]
        dk[r] = (R[:m] @ v[r][..., :, None])[..., 0]
        dv[r] = (k[r][..., None, :] @ R[:m])[..., 0, :]
        R[:m] = decay * R[:m]
    return (dq, dk, dv), R[back] if case["initial"] else None
