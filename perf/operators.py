"""Cases for timing and checking the training operators around the packed blocks.

The operators are those a training step needs next to the optimizer update of
a packed block: the embedding lookup and its gradient (the embedding block),
the softmax cross entropy of a large vocabulary and its gradients (the LM-head
block), Newton-Schulz orthogonalisation and the Muon step made of it (the
matrices of the decoder blocks).

A case is a dict of plain values. ``run`` computes an operator's plain form in
elementary fp32 torch operations, or, with ``own`` set, makes the library's
calls. ``exact`` gives the same outputs from the definition in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False  # False: the plain forms; True: the library's calls

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
INDEX = {32: torch.int32, 64: torch.int64}
IGNORE = -100          # target of a token that has no loss (padding, prompt)
NS = (3.4445, -4.7750, 2.0315)  # coefficients of the quintic Newton-Schulz step
NS_STEPS = 5
NS_EPS = 1e-7

# One decoder layer of the framework's TinyLlama-1.1B and LLaMA-7B workloads.
TINYLLAMA = dict(hidden=2048, kv=256, ffn=5632)
LLAMA7B = dict(hidden=4096, kv=4096, ffn=11008)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the next token of eight sequences being decoded: latency is all
        dict(name="embed_decode", op="embed", n=8, hidden=2048, vocab=32000, dtype="bf16", index=64, scale=1.0),
        # a training batch of 16 sequences of 4096 tokens, scaled by sqrt(hidden)
        dict(name="embed_batch", op="embed", n=65536, hidden=4096, vocab=32000, dtype="bf16", index=64, scale=64.0),
        # TinyLlama's embedding gradient of one sequence, written over the block's G segment
        dict(name="embed_grad_seq", op="embed_grad", n=4096, hidden=2048, vocab=32000, dtype="bf16", index=64, scale=1.0,
             accumulate=False),
        # a large batch added to an odd-sized fp32 gradient (a further micro-batch)
        dict(name="embed_grad_batch", op="embed_grad", n=65521, hidden=4095, vocab=32003, dtype="f32", index=32,
             scale=1.0, accumulate=True),
        # scoring the last 16 tokens of an answer: reading the head's weight is the work
        dict(name="xent_score", op="xent", n=16, hidden=2048, vocab=32000, index=64, grad=False),
        # evaluation loss over a long batch of the LLaMA-7B shape
        dict(name="xent_eval", op="xent", n=8192, hidden=4096, vocab=32000, index=64, grad=False),
        # training loss of a short sequence, an odd number of tokens (TinyLlama head)
        dict(name="xent_train_seq", op="xent", n=1023, hidden=2048, vocab=32000, index=64, grad=True),
        # training loss over a vocabulary of 128 Ki entries
        dict(name="xent_train_vocab", op="xent", n=4096, hidden=4096, vocab=131072, index=64, grad=True),
        # one K projection of TinyLlama
        dict(name="ns_kv", op="ns", count=1, rows=256, cols=2048, dtype="bf16", pad=0),
        # one up projection of LLaMA-7B: tall, as the weights are stored
        dict(name="ns_ffn", op="ns", count=1, rows=11008, cols=4096, dtype="bf16", pad=0),
        # one TinyLlama decoder layer, 16 B/param mixed layout: 7 matrices by Muon, 2 norms by AdamW
        dict(name="muon_tinyllama", op="muon", fmt="L16M", blocks=1, **TINYLLAMA),
        # one LLaMA-7B decoder layer, 12 B/param layout
        dict(name="muon_llama7b", op="muon", fmt="L12", blocks=1, **LLAMA7B),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A hidden size: usually a multiple of 8, one in four any number."""
    h = _log(rng, lo, hi)
    return h if rng.random() < 0.25 else max(8, h // 8 * 8)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "xent", "xent", "ns", "ns", "muon"])
    if op in ("embed", "embed_grad"):
        c = dict(op=op, n=_log(rng, 1, 65536), hidden=_width(rng, 64, 8192), vocab=_log(rng, 1000, 131072),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), index=rng.choice([32, 64]), scale=rng.choice([1.0, 0.5, 45.25]))
        while c["n"] * c["hidden"] > 65536 * 4096 or c["vocab"] * c["hidden"] > 1 << 29:
            c["hidden"] = max(64, c["hidden"] // 2)
        if op == "embed_grad":
            c["accumulate"] = rng.random() < 0.4
        return c
    if op == "xent":
        n, h, v = _log(rng, 1, 8192), _width(rng, 64, 4096), _log(rng, 500, 131072)
        while n * v > 1 << 29:
            n = max(1, n // 2)
        return dict(op=op, n=n, hidden=h, vocab=v, index=rng.choice([32, 64]), grad=rng.random() < 0.7)
    if op == "ns":
        r, c = _log(rng, 16, 8192), _log(rng, 16, 8192)
        while min(r, c) ** 2 * max(r, c) > 4096 * 4096 * 11008:
            r, c = max(16, r // 2), max(16, c // 2)
        count = rng.choice([1, 1, 2, 3, 8])
        while count > 1 and count * min(r, c) ** 2 * max(r, c) > 4096 * 4096 * 11008:
            count -= 1
        return dict(op=op, count=count, rows=r, cols=c, dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 3]))
    h = max(64, _log(rng, 64, 2048) // 16 * 16)
    return dict(op="muon", fmt=rng.choice(["L12", "L16M", "L16F"]), blocks=rng.choice([1, 1, 2]), hidden=h,
                kv=max(16, h // rng.choice([1, 4, 8])), ffn=int(h * rng.uniform(2.5, 3.5)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).mul_(std).to(dtype)


ZIPF = 10.0  # token t has probability proportional to ln((t + 11) / (t + 10)), about 1 / (t + 10)


def _tokens(g, n, vocab, index):
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = ZIPF * (((vocab + ZIPF) / ZIPF) ** u - 1.0)
    return t.floor().clamp_(0, vocab - 1).to(INDEX[index])


def _distinct(n, vocab):
    """Expected number of different tokens among n drawn by _tokens."""
    t = np.arange(vocab, dtype=np.float64)
    p = np.log((t + ZIPF + 1) / (t + ZIPF)) / math.log((vocab + ZIPF) / ZIPF)
    return float((-np.expm1(n * np.log1p(-p))).sum())


def _momentum_like(g, rows, cols, std):
    """A gradient-like matrix: a few strong directions over noise."""
    k = max(1, min(32, min(rows, cols) // 4))
    d = torch.arange(1, k + 1, device="cuda", dtype=F32) ** -0.5
    low = (torch.randn(rows, k, generator=g, device="cuda") * d) @ torch.randn(k, cols, generator=g, device="cuda")
    x = low / 3.0 + 0.5 * torch.randn(rows, cols, generator=g, device="cuda")
    return x * std


def _layer_specs(case):
    """(name, shape, block) of the decoder layers of a Muon case: the framework's layer shapes."""
    h, kv, f = case["hidden"], case["kv"], case["ffn"]
    out = []
    for b in range(case["blocks"]):
        out += [("q_proj", (h, h), b), ("k_proj", (kv, h), b), ("v_proj", (kv, h), b), ("o_proj", (h, h), b),
                ("gate_proj", (f, h), b), ("up_proj", (f, h), b), ("down_proj", (h, f), b),
                ("input_norm", (h,), b), ("post_attn_norm", (h,), b)]
    return out


SEGMENTS = {"L12": (("G", BF16), ("W", BF16), ("M", F32), ("V", F32)),
            "L16M": (("G", BF16), ("MASTER", F32), ("M", F32), ("V", F32), ("W", BF16)),
            "L16F": (("G", F32), ("W", F32), ("M", F32), ("V", F32))}


def _geometry(case):
    """Block layout as documented: tensors at multiples of 8 elements, segments of a multiple of 2048 elements.
    Returns ({(block, tensor): (offset, shape)}, padded elements per block)."""
    at, pos = {}, [0] * case["blocks"]
    for name, shape, b in _layer_specs(case):
        pos[b] = -(-pos[b] // 8) * 8
        at[b, name] = (pos[b], shape)
        pos[b] += math.prod(shape)
    return at, [-(-p // 2048) * 2048 for p in pos]


MUON = dict(lr=3e-5, momentum=0.95, weight_decay=0.01)  # a late-schedule rate
RMS_SCALE = 0.2  # update scaled by 0.2 sqrt(max(rows, cols)), the AdamW-matched size
ADAMW = dict(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=10)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "embed":
        s["table"] = _normal(g, (case["vocab"], case["hidden"]), 0.02, DTYPES[case["dtype"]])
        s["tokens"] = _tokens(g, case["n"], case["vocab"], case["index"])
        s["out"] = torch.empty(case["n"], case["hidden"], device="cuda", dtype=DTYPES[case["dtype"]])
    elif op == "embed_grad":
        s["dout"] = _normal(g, (case["n"], case["hidden"]), 1e-3, DTYPES[case["dtype"]])
        s["tokens"] = _tokens(g, case["n"], case["vocab"], case["index"])
        s["grad"] = _normal(g, (case["vocab"], case["hidden"]), 1e-3, DTYPES[case["dtype"]])
    elif op == "xent":
        n, h, v = case["n"], case["hidden"], case["vocab"]
        s["w"] = _normal(g, (v, h), 0.02, BF16)
        t = _tokens(g, n, v, 64)
        x = torch.randn(n, h, generator=g, device="cuda")
        # the model half knows its targets: their logits are raised by 0 to 8
        lift = torch.rand(n, 1, generator=g, device="cuda") * 8.0
        wt = s["w"][t].float()
        s["x"] = (x + lift * wt / wt.square().sum(1, keepdim=True)).to(BF16)
        out = torch.rand(n, generator=g, device="cuda") < 0.05
        out[0] = False
        s["targets"] = torch.where(out, torch.full_like(t, IGNORE), t).to(INDEX[case["index"]])
        s["loss"], s["lse"] = (torch.empty(n, device="cuda", dtype=F32) for _ in range(2))
        if case["grad"]:
            s["mean"] = torch.empty(1, device="cuda", dtype=F32)
            s["dx"] = torch.empty(n, h, device="cuda", dtype=BF16)
            s["dw"] = torch.empty(v, h, device="cuda", dtype=BF16)
    elif op == "ns":
        r, c, p = case["rows"], case["cols"], case["pad"]
        s["x"] = [torch.empty(r, c + p, device="cuda", dtype=DTYPES[case["dtype"]])[:, :c].copy_(_momentum_like(g, r, c, 1e-3))
                  for _ in range(case["count"])]
        s["out"] = [torch.empty(r, c, device="cuda", dtype=BF16) for _ in range(case["count"])]
    else:
        at, padded = _geometry(case)
        s["memory"], s["views"] = [], []
        for b in range(case["blocks"]):
            size = [padded[b] * torch.empty(0, dtype=d).element_size() for _, d in SEGMENTS[case["fmt"]]]
            buf = torch.zeros(sum(size), device="cuda", dtype=torch.uint8)
            ends = np.cumsum(size)
            s["memory"].append(buf)
            s["views"].append({f: buf[int(e) - z:int(e)].view(d) for (f, d), z, e in zip(SEGMENTS[case["fmt"]], size, ends)})
        for (b, name), (off, shape) in at.items():
            v, z = s["views"][b], math.prod(shape)
            w = torch.randn(z, generator=g, device="cuda") * 0.02
            for f in ("MASTER", "W"):
                if f in v:
                    v[f][off:off + z] = w
            for f, std in (("G", 1e-3), ("M", 1e-3)):
                x = _momentum_like(g, *shape, std) if len(shape) == 2 else torch.randn(z, generator=g, device="cuda") * std
                v[f][off:off + z] = x.reshape(-1)
            v["V"][off:off + z] = (torch.randn(z, generator=g, device="cuda") * 1e-3).square()
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program that uses the library keeps: the scratch memory and the layout handle."""
    from optimizer_update_gb300 import Layout, lst
    size = 0
    if s["op"] == "embed_grad":
        size = lst.lst_embed_grad_workspace_bytes(s["n"], s["hidden"], s["vocab"])
    elif s["op"] == "xent":
        size = lst.lst_xent_workspace_bytes(s["n"], s["hidden"], s["vocab"], s["grad"])
    elif s["op"] == "ns":
        size = lst.lst_orthogonalize_workspace_bytes(s["count"], s["rows"], s["cols"])
    elif s["op"] == "muon":
        s["layout"] = Layout(_layer_specs(s), s["fmt"])
        size = lst.lst_muon_workspace_bytes(s["layout"].handle)
    s["ws"] = torch.empty(max(1, size), device="cuda", dtype=torch.uint8)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _plain_embed(s):
    return (s["table"][s["tokens"]].float() * s["scale"]).to(s["out"].dtype)


def _plain_embed_grad(s):
    g = s["grad"].float() if s["accumulate"] else torch.zeros(s["grad"].shape, device="cuda", dtype=F32)
    g.index_add_(0, s["tokens"], s["dout"].float() * s["scale"])
    s["grad"].copy_(g)
    return s["grad"]


def _plain_xent(s):
    x, w, t = s["x"].float(), s["w"].float(), s["targets"].long()
    logits = x @ w.T
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    valid = t != IGNORE
    at = torch.where(valid, t, torch.zeros_like(t)).unsqueeze(1)
    loss = torch.where(valid, lse - logits.gather(1, at).squeeze(1), torch.zeros_like(lse))
    if not s["grad"]:
        return {"loss": loss, "lse": lse}
    count = valid.sum()
    mean = (loss.sum() / count).reshape(1)
    g = valid.float().unsqueeze(1) / count
    d = e.div_(total)
    d.scatter_add_(1, at, torch.full_like(lse, -1.0).unsqueeze(1))
    d.mul_(g)
    return {"loss": loss, "lse": lse, "mean": mean, "dx": (d @ w).to(BF16), "dw": (d.T @ x).to(BF16)}


def _plain_newton_schulz(u):
    a, b, c = NS
    x = u.T if u.shape[0] > u.shape[1] else u
    x = x / (x.square().sum().sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.T if u.shape[0] > u.shape[1] else x


def _plain_ns(s):
    return [_plain_newton_schulz(x.float()).to(BF16) for x in s["x"]]


def _plain_adamw(g, w, m, v):
    p = ADAMW
    m.copy_(p["beta1"] * m + (1 - p["beta1"]) * g)
    v.copy_(p["beta2"] * v + (1 - p["beta2"]) * g * g)
    u = (m / (1 - p["beta1"] ** p["step"])) / ((v / (1 - p["beta2"] ** p["step"])).sqrt() + p["eps"])
    return w * (1 - p["lr"] * p["weight_decay"]) - p["lr"] * u


def _plain_muon(s):
    p = MUON
    for (b, name), (off, shape) in _geometry(s)[0].items():
        x = {f: v[off:off + math.prod(shape)].view(shape) for f, v in s["views"][b].items()}
        weight = x["MASTER"] if "MASTER" in x else x["W"]
        g, w = x["G"].float(), weight.float()
        if len(shape) == 2:
            x["M"].copy_(p["momentum"] * x["M"] + g)
            o = _plain_newton_schulz(g + p["momentum"] * x["M"])
            w = w * (1 - p["lr"] * p["weight_decay"]) - p["lr"] * RMS_SCALE * math.sqrt(max(shape)) * o
        else:
            w = _plain_adamw(g, w, x["M"], x["V"])
        weight.copy_(w)
        if "MASTER" in x:
            x["W"].copy_(w)
    return [{f: v for f, v in views.items() if f != "G"} for views in s["views"]]


_plain = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "xent": _plain_xent, "ns": _plain_ns, "muon": _plain_muon}


def _own_embed(s):
    from optimizer_update_gb300 import lst
    lst.lst_embed(lst.matrix(s["table"]), lst.indices(s["tokens"]), lst.matrix(s["out"]), s["scale"], _stream())
    return s["out"]


def _own_embed_grad(s):
    from optimizer_update_gb300 import lst
    lst.lst_embed_grad(lst.matrix(s["dout"]), lst.indices(s["tokens"]), lst.matrix(s["grad"]), s["scale"],
                       s["accumulate"], s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return s["grad"]


def _own_xent(s):
    from optimizer_update_gb300 import lst
    x, w, t, ws = lst.matrix(s["x"]), lst.matrix(s["w"]), lst.indices(s["targets"]), s["ws"]
    if not s["grad"]:
        lst.lst_xent_loss(x, w, t, IGNORE, s["loss"].data_ptr(), s["lse"].data_ptr(), ws.data_ptr(), ws.numel(), _stream())
        return {"loss": s["loss"], "lse": s["lse"]}
    lst.lst_xent_grad(x, w, t, IGNORE, 1.0, s["loss"].data_ptr(), s["lse"].data_ptr(), s["mean"].data_ptr(),
                      lst.matrix(s["dx"]), lst.matrix(s["dw"]), False, ws.data_ptr(), ws.numel(), _stream())
    return {"loss": s["loss"], "lse": s["lse"], "mean": s["mean"], "dx": s["dx"], "dw": s["dw"]}


def _own_ns(s):
    from optimizer_update_gb300 import lst
    lst.lst_orthogonalize([lst.matrix(x) for x in s["x"]], [lst.matrix(o) for o in s["out"]], lst.ns_params(),
                          s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return s["out"]


def _own_muon(s):
    from optimizer_update_gb300 import lst
    lst.lst_muon_step(s["layout"].handle, [b.data_ptr() for b in s["memory"]],
                      lst.muon_hparams(rms_scale=RMS_SCALE, nesterov=True, **MUON), lst.adamw_hparams(**ADAMW), None,
                      s["ws"].data_ptr(), s["ws"].numel(), _stream())
    return [{f: v for f, v in views.items() if f != "G"} for views in s["views"]]


_own = {"embed": _own_embed, "embed_grad": _own_embed_grad, "xent": _own_xent, "ns": _own_ns, "muon": _own_muon}


def _stream():
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _ns_flops(rows, cols):
    """Five quintic steps on m x n, m <= n, symmetric products counted once: either X X^T, its square and the product
    with X in every step, or the Gram matrix carried over two steps (steps 1-2 and 4-5) and X formed three times."""
    m, n = min(rows, cols), max(rows, cols)
    return min(15 * m * m * n + 5 * m ** 3, 9 * m * m * n + 11 * m ** 3)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}.get(case.get("dtype"), 2)
    if op == "embed":
        rows = _distinct(case["n"], case["vocab"]) + case["n"]
        return {"bytes": rows * case["hidden"] * size + case["n"] * case["index"] / 8, "flops": case["n"] * case["hidden"]}
    if op == "embed_grad":
        seen = _distinct(case["n"], case["vocab"])
        rows = case["n"] + (2 * seen if case["accumulate"] else case["vocab"])
        return {"bytes": rows * case["hidden"] * size + case["n"] * case["index"] / 8, "flops": 2 * case["n"] * case["hidden"]}
    if op == "xent":
        n, h, v = case["n"], case["hidden"], case["vocab"]
        times = 2 if case["grad"] else 1  # dx, dw as large as x, w
        return {"bytes": 2 * h * (n + v) * times + n * (case["index"] / 8 + 8),
                "flops": (6 if case["grad"] else 2) * n * h * v}
    if op == "ns":
        z = case["rows"] * case["cols"] * case["count"]
        return {"bytes": z * (size + 2), "flops": case["count"] * _ns_flops(case["rows"], case["cols"])}
    each = {"L12": 2 + 2 * 2 + 2 * 4, "L16M": 2 + 2 * 4 + 2 * 4 + 2, "L16F": 4 + 2 * 4 + 2 * 4}[case["fmt"]]
    shapes = [shape for _, shape, _ in _layer_specs(case) if len(shape) == 2]
    return {"bytes": each * sum(r * c for r, c in shapes), "flops": sum(_ns_flops(r, c) for r, c in shapes)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_newton_schulz(u):
    """The five steps as one polynomial of the Gram matrix: X_5 = P_5 ... P_1 X_0, all P_k polynomials of X_0 X_0^T."""
    a, b, c = NS
    tall = u.shape[0] > u.shape[1]
    x = u.double() / (torch.linalg.matrix_norm(u.double()) + NS_EPS)
    gram = x.mT @ x if tall else x @ x.mT
    eye = torch.eye(gram.shape[0], device=gram.device, dtype=torch.float64)
    prod = eye
    for k in range(NS_STEPS):
        p = a * eye + gram @ (b * eye + c * gram)
        prod = p if k == 0 else p @ prod
        gram = p @ gram @ p
    return x @ prod if tall else prod @ x


def exact(case, seed):
    op = case["op"]
    global own
    was, own = own, False
    try:
        if op == "muon" and sum(4 * min(s) ** 2 * max(s) + 40 * min(s) ** 3 for _, s, _ in _layer_specs(case) if len(s) == 2) > 1.5e13:
            return None  # over 20 seconds in 64 bits
        s = prepare(case, seed)
    finally:
        own = was
    if op == "embed":
        return torch.index_select(s["table"], 0, s["tokens"]).double().mul_(case["scale"])
    if op == "embed_grad":
        t, order = torch.sort(s["tokens"].long(), stable=True)
        run_sum = torch.cumsum(s["dout"].double()[order], dim=0)
        last = torch.ones_like(t, dtype=torch.bool)
        last[:-1] = t[1:] != t[:-1]
        rows, ends = t[last], run_sum[last]
        sums = ends.clone()
        sums[1:] -= ends[:-1]
        out = s["grad"].double() if case["accumulate"] else torch.zeros(s["grad"].shape, device="cuda", dtype=torch.float64)
        out[rows] += sums * case["scale"]
        return out
    if op == "xent":
        x, w, t = s["x"].double(), s["w"].double(), s["targets"].long()
        z = torch.einsum("nh,vh->nv", x, w)
        lse = torch.logsumexp(z, dim=1)
        keep = torch.nonzero(t != IGNORE).squeeze(1)
        loss = torch.zeros_like(lse)
        loss[keep] = lse[keep] - z[keep, t[keep]]
        if not case["grad"]:
            return {"loss": loss, "lse": lse}
        p = torch.zeros_like(z)
        p[keep] = torch.exp(z[keep] - lse[keep, None])
        del z
        p[keep, t[keep]] -= 1.0
        p /= keep.numel()
        return {"loss": loss, "lse": lse, "mean": (loss.sum() / keep.numel()).reshape(1),
                "dx": torch.einsum("nv,vh->nh", p, w), "dw": torch.einsum("nv,nh->vh", p, x)}
    if op == "ns":
        return [_exact_newton_schulz(x) for x in s["x"]]
    out = [{f: v.double() for f, v in views.items()} for views in s["views"]]
    for (b, name), (off, shape) in _geometry(case)[0].items():
        x = {f: v[off:off + math.prod(shape)].view(shape) for f, v in out[b].items()}
        w = x["MASTER"] if "MASTER" in x else x["W"]
        if len(shape) == 2:
            x["M"].mul_(MUON["momentum"]).add_(x["G"])
            o = _exact_newton_schulz(x["G"] + MUON["momentum"] * x["M"])
            w.mul_(1 - MUON["lr"] * MUON["weight_decay"]).sub_(o, alpha=MUON["lr"] * RMS_SCALE * max(shape) ** 0.5)
        else:
            p = ADAMW
            x["M"].lerp_(x["G"], 1 - p["beta1"])
            x["V"].mul_(p["beta2"]).addcmul_(x["G"], x["G"], value=1 - p["beta2"])
            mh, vh = x["M"] / (1 - p["beta1"] ** p["step"]), x["V"] / (1 - p["beta2"] ** p["step"])
            w.mul_(1 - p["lr"] * p["weight_decay"]).sub_(p["lr"] * mh / (vh.sqrt() + p["eps"]))
        if "MASTER" in x:
            x["W"].copy_(w)
    return [{f: v for f, v in views.items() if f != "G"} for views in out]
