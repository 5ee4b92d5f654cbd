"""Cases for timing and checking the operators between the layers.

What a training step computes at the boundary of a layer: the residual stream
with the norms before and after a block, its gate and scales, forward and
backward; activations kept for the backward pass in 8 bits; and the weight
gradient of a linear layer from such a checkpoint, written into a block's G.

A case is a dict of plain values. ``run`` computes an operator's plain form in
elementary fp32 torch operations, or, with ``own`` set, makes the library's
calls. ``exact`` gives the same outputs from the definition in 64 bits.
"""

from __future__ import annotations

import math

import torch

own = False  # False: the plain forms; True: the library's calls

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-5
BLOCK = 32                       # values of a checkpoint that share a scale
TOP = {"i8": 127.0, "e4m3": 448.0}  # the largest magnitude of a stored value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # eight tokens of a short fine-tuning step through a pre-norm layer boundary: latency is all
        dict(name="norm_few", op="norm", n=8, hidden=2048, dtype="bf16", wdtype="bf16", post=False, gate_rows=0, alpha=1.0,
             beta=1.0, fmt="", pad=0),
        # TinyLlama, a sequence: norms on both sides of the block, a gate per channel
        dict(name="norm_seq", op="norm", n=4096, hidden=2048, dtype="bf16", wdtype="bf16", post=True, gate_rows=1, alpha=1.0,
             beta=0.5, fmt="", pad=0),
        # LLaMA-7B, a micro-batch of eight sequences, the stream checkpointed on its way and restored as the backward does
        dict(name="norm_checkpointed", op="norm", n=16384, hidden=4096, dtype="bf16", wdtype="bf16", post=True, gate_rows=1,
             alpha=1.0, beta=0.25, fmt="i8", pad=0),
        # backward of a short odd batch in the plain pre-norm form
        dict(name="norm_grad_few", op="norm_grad", n=37, hidden=2048, dtype="bf16", wdtype="f32", post=False, gate_rows=0,
             alpha=1.0, beta=1.0, fmt="", pad=0, accumulate=False),
        # backward of four samples with a gate each, from the activations themselves
        dict(name="norm_grad_samples", op="norm_grad", n=4096, hidden=4096, dtype="bf16", wdtype="bf16", post=True,
             gate_rows=4, alpha=1.0, beta=1.0, fmt="", pad=0, accumulate=False),
        # Llama-70B hidden size, an odd batch, from 8-bit checkpoints, weight gradients added to a further micro-batch's
        dict(name="norm_grad_checkpointed", op="norm_grad", n=16381, hidden=8192, dtype="bf16", wdtype="bf16", post=True,
             gate_rows=1, alpha=1.0, beta=0.25, fmt="i8", pad=0, accumulate=True),
        # fp32 activations of an odd width, a gate per token
        dict(name="norm_grad_odd", op="norm_grad", n=1023, hidden=4095, dtype="f32", wdtype="f32", post=True, gate_rows=1023,
             alpha=0.7, beta=0.3, fmt="", pad=0, accumulate=False),
        # a few tokens kept and restored
        dict(name="checkpoint_few", op="checkpoint", n=16, hidden=2048, dtype="bf16", fmt="e4m3", pad=0),
        # a whole batch's activations of one layer
        dict(name="checkpoint_batch", op="checkpoint", n=65521, hidden=4096, dtype="bf16", fmt="i8", pad=0),
        # TinyLlama's K projection: few rows of weights, a long sum over the tokens, its input normed again
        dict(name="wgrad_kv", op="wgrad", n=4096, out=256, hidden=2048, fmt="i8", norm=True, wdtype="bf16", accumulate=False),
        # LLaMA-7B's up projection over a micro-batch
        dict(name="wgrad_up", op="wgrad", n=8192, out=11008, hidden=4096, fmt="e4m3", norm=False, wdtype="bf16",
             accumulate=True),
        # odd sizes, an fp32 gradient
        dict(name="wgrad_odd", op="wgrad", n=1021, out=5631, hidden=2047, fmt="i8", norm=False, wdtype="f32", accumulate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A hidden size: usually a multiple of 8, one in four any number."""
    h = _log(rng, lo, hi)
    return h if rng.random() < 0.25 else max(8, h // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "checkpoint", "wgrad", "wgrad"])
    if op == "wgrad":
        c = dict(op=op, n=_log(rng, 1, 16384), out=_width(rng, 16, 11008), hidden=_width(rng, 16, 8192),
                 fmt=rng.choice(["i8", "e4m3"]), norm=rng.random() < 0.4, wdtype="bf16", accumulate=rng.random() < 0.4)
        while c["n"] * c["out"] * c["hidden"] > 8192 * 11008 * 4096:
            c["n"] = max(1, c["n"] // 2)
        if not c["norm"] and rng.random() < 0.3:
            c["wdtype"] = "f32"
        return c
    c = dict(op=op, n=_log(rng, 1, 32768), hidden=_width(rng, 32, 12288), dtype=rng.choice(["bf16", "bf16", "f32"]),
             pad=rng.choice([0, 0, 8, 3]))
    most = 65521 * 4096 if op == "checkpoint" else 16384 * 4096 if op == "norm" else 16381 * 8192
    if c["dtype"] == "f32":
        most //= 2
    while c["n"] * c["hidden"] > most:
        c["n"] = max(1, c["n"] // 2)
    if op == "checkpoint":
        return dict(c, fmt=rng.choice(["i8", "e4m3"]))
    post = rng.random() < 0.6
    rows = rng.choice([0, 1, 1, 2, c["n"]])
    if rows == 2 and c["n"] % 2:
        c["n"] = max(2, c["n"] - 1)
    c |= dict(wdtype=rng.choice(["bf16", "f32"]), post=post, gate_rows=min(rows, c["n"]), alpha=rng.choice([1.0, 1.0, 0.7]),
              beta=rng.choice([1.0, 0.25]), fmt=rng.choice(["", "i8", "e4m3"]))
    if op == "norm_grad":
        c["accumulate"] = rng.random() < 0.4
    return c


# ---------------------------------------------------------------------------
# checkpoints in torch: the plain form, and the inputs of the backward cases
# ---------------------------------------------------------------------------
def _blocks(x):
    """rows x blocks x 32, the last block filled with zeros."""
    n, h = x.shape
    full = -(-h // BLOCK) * BLOCK
    if full != h:
        x = torch.cat([x, x.new_zeros(n, full - h)], dim=1)
    return x.view(n, full // BLOCK, BLOCK)


def _pack(x, fmt):
    """(values, scale bytes): per block the smallest power of two with |x| <= top * 2^k, values rounded to nearest even."""
    b = _blocks(x.float())
    most = b.abs().amax(dim=2)
    _, e = torch.frexp(most / TOP[fmt])       # a power of two: exact unless subnormal, which the inputs are not
    k = e - 1
    k = torch.where(torch.ldexp(torch.full_like(most, TOP[fmt]), k) < most, k + 1, k)
    k = torch.where(most > 0, k, torch.full_like(k, -127)).clamp_(-127, 127)
    q = torch.ldexp(torch.ldexp(b, (-k // 2).unsqueeze(2)), (-k - (-k // 2)).unsqueeze(2))
    q = torch.round(q).to(torch.int8) if fmt == "i8" else q.to(torch.float8_e4m3fn)
    return q.view(x.shape[0], -1)[:, :x.shape[1]], (k + 127).to(torch.uint8)


def _unpack(q, scales):
    b = _blocks(q.float())
    k = scales.int() - 127
    v = torch.ldexp(torch.ldexp(b, (k // 2).unsqueeze(2)), (k - k // 2).unsqueeze(2))
    return v.view(q.shape[0], -1)[:, :q.shape[1]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _padded(t, pad):
    """The same values in rows `pad` elements further apart."""
    if not pad:
        return t
    return torch.empty(t.shape[0], t.shape[1] + pad, device="cuda", dtype=t.dtype)[:, :t.shape[1]].copy_(t)


def _stream_like(g, n, h, std, dtype):
    """Activations: tokens of different sizes, a few channels far larger than the others."""
    x = torch.randn(n, h, generator=g, device="cuda")
    x.mul_(torch.exp(0.3 * torch.randn(n, 1, generator=g, device="cuda")) * std)
    c = torch.randint(0, h, (max(1, h // 512),), generator=g, device="cuda")
    x[:, c] *= 20.0
    return x.to(dtype)


def _grad_like(g, n, h, dtype):
    x = torch.randn(n, h, generator=g, device="cuda").mul_(1e-3)
    x[torch.rand(n, generator=g, device="cuda") < 0.05] = 0.0  # tokens without a loss
    return x.to(dtype)


def _checkpoint_buffers(n, h):
    return (torch.empty(n, -(-h // 16) * 16, device="cuda", dtype=torch.uint8)[:, :h],
            torch.empty(n, -(-h // BLOCK), device="cuda", dtype=torch.uint8))


def _checkpoint_of(x, fmt):
    q, scales = _pack(x, fmt)
    data, s = _checkpoint_buffers(*x.shape)
    data.copy_(q.view(torch.uint8))
    s.copy_(scales)
    return data, s, fmt


def _values(c):
    data, scales, fmt = c
    q = data.contiguous().view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn)
    return _unpack(q, scales)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    n, h = case["n"], case["hidden"]
    s = dict(case)
    if op == "wgrad":
        w = DTYPES[case["wdtype"]]
        s["dy"] = _grad_like(g, n, case["out"], BF16)
        s["c"] = _checkpoint_of(_stream_like(g, n, h, 1.0, BF16), case["fmt"])
        s["weight"] = (1.0 + 0.1 * torch.randn(1, h, generator=g, device="cuda")).to(BF16) if case["norm"] else None
        s["dw"] = (torch.randn(case["out"], h, generator=g, device="cuda") * 1e-3 * math.sqrt(n)).to(w)
    else:
        t, pad = DTYPES[case["dtype"]], case["pad"]

        def buffer():
            return torch.empty(n, h + pad, device="cuda", dtype=t)[:, :h]

        if op == "checkpoint":
            s["x"] = _padded(_stream_like(g, n, h, 1.0, t), pad)
            s["c"] = (*_checkpoint_buffers(n, h), case["fmt"])
            s["out"] = buffer()
        else:
            w, rows = DTYPES[case["wdtype"]], case["gate_rows"]
            y = _stream_like(g, n, h, 0.5, t)
            x = _stream_like(g, n, h, 1.0, t)
            s["w_pre"] = (1.0 + 0.1 * torch.randn(1, h, generator=g, device="cuda")).to(w)
            s["w_post"] = (1.0 + 0.1 * torch.randn(1, h, generator=g, device="cuda")).to(w) if case["post"] else None
            s["gate"] = (0.5 + 0.1 * torch.randn(rows, h, generator=g, device="cuda")).to(w) if rows else None
            if op == "norm":
                s["x"], s["y"] = _padded(x, pad), _padded(y, pad)
                s["h"], s["z"] = buffer(), buffer()
                if case["fmt"]:
                    s["c"] = (*_checkpoint_buffers(n, h), case["fmt"])
                    s["out"] = buffer()
            else:
                s["dh"], s["dz"] = (_padded(_grad_like(g, n, h, t), pad) for _ in range(2))
                s["h"] = _checkpoint_of(x, case["fmt"]) if case["fmt"] else _padded(x, pad)
                s["y"] = _checkpoint_of(y, case["fmt"]) if case["fmt"] else _padded(y, pad)
                s["dx"], s["dy"] = buffer(), buffer()
                # what another micro-batch left there
                for k, like in (("dgate", s["gate"]), ("dw_post", s["w_post"]), ("dw_pre", s["w_pre"])):
                    s[k] = None if like is None else (torch.randn(like.shape, generator=g, device="cuda") * 1e-3).to(w)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program that uses the library keeps: the scratch memory."""
    from optimizer_update_gb300 import lst
    size = 0
    if s["op"] == "norm_grad":
        size = lst.lst_residual_norm_grad_workspace_bytes(s["n"], s["hidden"], s["gate_rows"])
    elif s["op"] == "wgrad":
        size = lst.lst_checkpoint_wgrad_workspace_bytes(lst.matrix(s["dy"]), lst.checkpoint(*s["c"]), lst.matrix(s["dw"]))
    s["ws"] = torch.empty(max(1, size), device="cuda", dtype=torch.uint8)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _per_token(gate, n):
    """Gate rows, each for n / rows tokens."""
    return gate.float().repeat_interleave(n // gate.shape[0], dim=0) if gate.shape[0] not in (1, n) else gate.float()


def _rho(x):
    return torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS)


def _plain_checkpoint(s):
    return _unpack(*_pack(s["x"], s["fmt"])).to(s["out"].dtype)


def _plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    if s["post"]:
        y = y * _rho(y) * s["w_post"].float()
    if s["gate"] is not None:
        y = y * _per_token(s["gate"], s["n"])
    h = s["alpha"] * x + s["beta"] * y
    z = h * _rho(h) * s["w_pre"].float()
    out = {"h": h.to(s["h"].dtype), "z": z.to(s["z"].dtype)}
    if s["fmt"]:
        out["restored"] = _unpack(*_pack(out["h"], s["fmt"])).to(s["out"].dtype)
    return out


def _plain_norm_grad(s):
    n = s["n"]
    h, y = (_values(s[k]) if s["fmt"] else s[k].float() for k in ("h", "y"))
    dz, w = s["dz"].float(), s["w_pre"].float()
    rho = _rho(h)
    d = dz * w
    d = s["dh"].float() + rho * (d - h * rho.square() * (d * h).mean(dim=1, keepdim=True))
    sums = {"dw_pre": (dz * h * rho).sum(dim=0, keepdim=True)}
    out = {"dx": (s["alpha"] * d).to(s["dx"].dtype)}
    e = s["beta"] * d
    tau = _rho(y) if s["post"] else None
    u = y * tau * s["w_post"].float() if s["post"] else y
    if s["gate"] is not None:
        rows = s["gate"].shape[0]
        sums["dgate"] = (e * u).view(rows, n // rows, -1).sum(dim=1)
        e = e * _per_token(s["gate"], n)
    if s["post"]:
        sums["dw_post"] = (e * y * tau).sum(dim=0, keepdim=True)
        e = e * s["w_post"].float()
        e = tau * (e - y * tau.square() * (e * y).mean(dim=1, keepdim=True))
    out["dy"] = e.to(s["dy"].dtype)
    return out | {k: s[k].copy_(s[k].float() + v if s["accumulate"] else v) for k, v in sums.items()}


def _plain_wgrad(s):
    x = _values(s["c"])
    if s["norm"]:
        x = x * _rho(x) * s["weight"].float()
    dw = s["dy"].float().T @ x
    return s["dw"].copy_(s["dw"].float() + dw if s["accumulate"] else dw)


_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "checkpoint": _plain_checkpoint, "wgrad": _plain_wgrad}


def _own_checkpoint(s):
    from optimizer_update_gb300 import lst
    c = lst.checkpoint(*s["c"])
    lst.lst_checkpoint_save(lst.matrix(s["x"]), c, _stream())
    lst.lst_checkpoint_restore(c, lst.matrix(s["out"]), _stream())
    return s["out"]


def _matrix(t):
    from optimizer_update_gb300 import lst
    return None if t is None else lst.matrix(t)


def _own_norm(s):
    from optimizer_update_gb300 import lst
    c = lst.checkpoint(*s["c"]) if s["fmt"] else None
    lst.lst_residual_norm(lst.matrix(s["x"]), lst.matrix(s["y"]), _matrix(s["gate"]), _matrix(s["w_post"]),
                          lst.matrix(s["w_pre"]), lst.residual_params(s["alpha"], s["beta"], EPS), lst.matrix(s["h"]),
                          lst.matrix(s["z"]), c, None, _stream())
    out = {"h": s["h"], "z": s["z"]}
    if s["fmt"]:
        lst.lst_checkpoint_restore(c, lst.matrix(s["out"]), _stream())
        out["restored"] = s["out"]
    return out


def _own_norm_grad(s):
    from optimizer_update_gb300 import lst
    h, y = (lst.checkpoint(*s[k]) if s["fmt"] else lst.matrix(s[k]) for k in ("h", "y"))
    lst.lst_residual_norm_grad(lst.matrix(s["dh"]), lst.matrix(s["dz"]), h, y, _matrix(s["gate"]), _matrix(s["w_post"]),
                               lst.matrix(s["w_pre"]), lst.residual_params(s["alpha"], s["beta"], EPS), lst.matrix(s["dx"]),
                               lst.matrix(s["dy"]), _matrix(s["dgate"]), _matrix(s["dw_post"]), lst.matrix(s["dw_pre"]),
                               s["accumulate"], s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return {k: s[k] for k in ("dx", "dy", "dgate", "dw_post", "dw_pre") if s[k] is not None}


def _own_wgrad(s):
    from optimizer_update_gb300 import lst
    lst.lst_checkpoint_wgrad(lst.matrix(s["dy"]), lst.checkpoint(*s["c"]), _matrix(s["weight"]), EPS, lst.matrix(s["dw"]),
                             s["accumulate"], s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return s["dw"]


_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "checkpoint": _own_checkpoint, "wgrad": _own_wgrad}


def _stream():
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, n, h = case["op"], case["n"], case["hidden"]
    kept = n * (h + -(-h // BLOCK))  # a checkpoint
    if op == "wgrad":
        size = {"bf16": 2, "f32": 4}[case["wdtype"]]
        return {"bytes": 2 * n * case["out"] + kept + size * case["out"] * h * (2 if case["accumulate"] else 1),
                "flops": 2 * n * case["out"] * h}
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    if op == "checkpoint":
        return {"bytes": 2 * n * h * size + kept, "flops": 4 * n * h}
    rows = case["gate_rows"] + 1 + case["post"]
    vectors = rows * h * {"bf16": 2, "f32": 4}[case["wdtype"]]
    if op == "norm":
        return {"bytes": 4 * n * h * size + vectors + (kept + n * h * size if case["fmt"] else 0), "flops": 12 * n * h}
    return {"bytes": 4 * n * h * size + 2 * (kept if case["fmt"] else n * h * size) + (3 if case["accumulate"] else 2) * vectors,
            "flops": 30 * n * h}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_round(x, fmt):
    """What the checkpoint of x stands for, in 64 bits: the block's step is found by counting powers of two down from 2^128."""
    n, h = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -h % BLOCK)).unflatten(1, (-1, BLOCK))
    most = v.abs().max(dim=2, keepdim=True).values
    steps = torch.exp2(torch.arange(-127, 128, device=x.device, dtype=F64))
    scale = steps[torch.searchsorted(steps * TOP[fmt], most.clamp(max=TOP[fmt] * 2.0 ** 127))]
    if fmt == "i8":
        r = torch.round(v / scale)
    else:  # 3 bits behind the leading one, and steps of 2^-9 below 2^-6
        a = v / scale
        step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
        r = torch.round(a / step) * step
    return (r * scale).flatten(1)[:, :h]


def _exact_norm(x, w):
    return torch.nn.functional.normalize(x, dim=1, eps=0.0) * w * (x.shape[1] ** 0.5) * (
        x.square().mean(1, keepdim=True) / (x.square().mean(1, keepdim=True) + EPS)).sqrt()


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, n = case["op"], case["n"]
    if op == "checkpoint":
        return _exact_round(s["x"], case["fmt"])
    if op == "wgrad":
        x = _exact_values(s["c"])
        if case["norm"]:
            x = _exact_norm(x, s["weight"].double())
        dw = torch.einsum("to,ti->oi", s["dy"].double(), x)
        return dw + s["dw"].double() if case["accumulate"] else dw
    wide = {k: None if s[k] is None else s[k].double() for k in ("gate", "w_post", "w_pre")}

    def branch(y, gate, w_post):
        u = _exact_norm(y, w_post) if w_post is not None else y
        if gate is not None:
            u = (u.unflatten(0, (gate.shape[0], -1)) * gate.unsqueeze(1)).flatten(0, 1)
        return case["beta"] * u

    if op == "norm":
        h = torch.add(branch(s["y"].double(), wide["gate"], wide["w_post"]), s["x"].double(), alpha=case["alpha"])
        out = {"h": h, "z": _exact_norm(h, wide["w_pre"])}
        if case["fmt"]:
            out["restored"] = _exact_round(h.to(s["h"].dtype), case["fmt"])
        return out
    h, y = (_exact_values(s[k]) if case["fmt"] else s[k].double() for k in ("h", "y"))
    h.requires_grad_()
    y.requires_grad_()
    for v in wide.values():
        if v is not None:
            v.requires_grad_()
    through, dw_pre = torch.autograd.grad(_exact_norm(h, wide["w_pre"]), (h, wide["w_pre"]), s["dz"].double())
    d = through + s["dh"].double()
    names = ["dy"] + ["dgate"] * (wide["gate"] is not None) + ["dw_post"] * (wide["w_post"] is not None)
    leaves = [v for v in (y, wide["gate"], wide["w_post"]) if v is not None]
    out = dict(zip(names, torch.autograd.grad(branch(y, wide["gate"], wide["w_post"]), leaves, d)))
    out |= {"dx": case["alpha"] * d, "dw_pre": dw_pre}
    if case["accumulate"]:
        for k in ("dgate", "dw_post", "dw_pre"):
            if k in out:
                out[k] = out[k] + s[k].double()
    return out


def _exact_values(c):
    data, scales, fmt = c
    q = (data.contiguous().view(torch.int8) if fmt == "i8" else data.contiguous().view(torch.float8_e4m3fn)).double()
    step = torch.exp2(scales.double() - 127.0)
    return q * step.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]
