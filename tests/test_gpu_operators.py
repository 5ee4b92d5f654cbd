"""The training operators on the GPU against plain implementations in 64 bits.

Tolerances are error bounds, written out before the first run. u16 = 2^-8 and
uh = 2^-11 are the unit roundoffs of bf16 and fp16, u32 = 2^-24 that of fp32;
a sum of k products in fp32 is taken to be off by 2 k u32 times the sum of
their magnitudes (twice the textbook bound: tensor cores may truncate).
"""

from __future__ import annotations

import math
import os
import sys
import threading

import numpy as np
import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from optimizer_update_gb300 import Layout, lst  # noqa: E402

U16, UH, U32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100


def stream():
    return torch.cuda.current_stream().cuda_stream


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(DT[dtype])


def scratch(nbytes, fill=0xA5):
    return torch.full((max(1, nbytes),), fill, dtype=torch.uint8, device="cuda")  # contents on entry do not matter


def strided(t, pad, shift=0):
    """The same values with rows `pad` elements apart and `shift` elements into the storage."""
    r, c = t.shape
    buf = torch.full((r * (c + pad) + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


def within(got, exact, bound, what):
    got, exact = got.double(), exact.double()
    assert torch.isfinite(got).all(), what
    over = (got - exact).abs() - bound
    assert float(over.max()) <= 0.0, f"{what}: {float(over.max()):.3g} over its bound"


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,hidden,vocab,src,dst,index,scale,pad", [
    (1, 1, 1, "bf16", "bf16", torch.int64, 1.0, 0), (1, 2048, 32000, "bf16", "bf16", torch.int64, 1.0, 0),
    (37, 2048, 999, "bf16", "f32", torch.int32, 45.25, 0), (513, 77, 130, "f32", "bf16", torch.int64, 0.5, 3),
    (100, 4104, 50, "f32", "f32", torch.int32, -2.0, 8), (64, 15, 7, "bf16", "bf16", torch.int32, 3.0, 1),
    (5000, 256, 5, "bf16", "bf16", torch.int64, 1.5, 4)])
def test_embed(n, hidden, vocab, src, dst, index, scale, pad):
    g = gen(n + hidden)
    table = strided(randn(g, vocab, hidden, dtype=src), pad)
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(index)
    out = strided(torch.zeros(n, hidden, dtype=DT[dst], device="cuda"), pad)
    lst.lst_embed(lst.matrix(table), lst.indices(tokens), lst.matrix(out), scale, stream())
    # one fp32 product, rounded once: no tolerance
    assert torch.equal(out, (table.float()[tokens.long()] * scale).to(DT[dst]))


def test_embed_outside_tokens_and_canaries():
    table = randn(gen(0), 10, 24, dtype="bf16")
    tokens = torch.tensor([0, -1, 9, 10, 2 ** 40, -2 ** 40], device="cuda")
    buf = torch.full((6 + 2, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    lst.lst_embed(lst.matrix(table), lst.indices(tokens), lst.matrix(buf[1:7]), 1.0, stream())
    assert torch.equal(buf[[1, 3]], table[[0, 9]])
    assert torch.isnan(buf[[2, 4, 5, 6]]).all() and (buf[[0, 7]] == 7.0).all()


def test_embed_past_32_bits():
    """A table and a gradient of more than 2^31 elements: the last rows."""
    vocab, hidden = (1 << 20) + 77, 2056
    table = torch.empty(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    table[-3:] = randn(gen(1), 3, hidden, dtype="bf16")
    table[0] = 5.0
    tokens = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 1], device="cuda")
    out = torch.empty(4, hidden, dtype=torch.bfloat16, device="cuda")
    lst.lst_embed(lst.matrix(table), lst.indices(tokens), lst.matrix(out), 1.0, stream())
    assert torch.equal(out, table[tokens])
    ws = scratch(lst.lst_embed_grad_workspace_bytes(4, hidden, vocab))
    table.fill_(1.0)
    lst.lst_embed_grad(lst.matrix(out), lst.indices(tokens), lst.matrix(table), 1.0, False, ws.data_ptr(), ws.numel(),
                       stream())
    assert torch.equal(table[vocab - 3], out[2]) and torch.equal(table[0], out[1])
    assert torch.equal(table[vocab - 1], (out[0].float() + out[3].float()).bfloat16())
    assert not table[1:vocab - 3].any() and not table[vocab - 2].any()


def token_patterns(kind, n, vocab, g):
    if kind == "uniform":
        return torch.randint(0, vocab, (n,), generator=g, device="cuda")
    if kind == "one":           # every token the same: one run over all CTAs
        return torch.full((n,), vocab - 1, device="cuda")
    if kind == "two":           # long runs that end inside a CTA's positions
        return torch.where(torch.rand(n, generator=g, device="cuda") < 0.3, 0, vocab // 2)
    if kind == "distinct":
        return torch.randperm(vocab, generator=g, device="cuda")[:n]
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")  # "holes": a third outside the vocabulary
    t[::3] = torch.where(t[::3] % 2 == 0, -1, vocab + t[::3])
    return t


@pytest.mark.parametrize("n,hidden,vocab,kind,src,dst,accumulate,pad", [
    (1, 8, 1, "uniform", "bf16", "bf16", False, 0), (1, 2048, 32000, "uniform", "bf16", "bf16", False, 0),
    (31, 64, 40, "uniform", "f32", "f32", False, 0), (32, 64, 40, "one", "f32", "f32", True, 0),
    (33, 64, 40, "one", "f32", "f32", False, 0), (4096, 72, 100, "one", "bf16", "bf16", False, 0),
    (1000, 1032, 50, "two", "bf16", "f32", True, 8), (3000, 77, 1050, "uniform", "f32", "bf16", False, 3),
    (2000, 130, 2000, "distinct", "bf16", "bf16", True, 0), (999, 24, 300, "holes", "bf16", "bf16", False, 0),
    (999, 25, 300, "holes", "f32", "f32", True, 1), (20000, 136, 70000, "uniform", "bf16", "bf16", False, 0),
    (70001, 16, 1100000, "uniform", "f32", "f32", False, 0), (300, 4096, 17, "uniform", "bf16", "bf16", False, 0)])
def test_embed_grad(n, hidden, vocab, kind, src, dst, accumulate, pad):
    g = gen(n + vocab)
    dout = strided(randn(g, n, hidden, dtype=src), pad)
    tokens = token_patterns(kind, n, vocab, g).to(torch.int32 if n % 2 else torch.int64)
    before = randn(g, vocab, hidden, dtype=dst)
    scale = 0.75
    ws = scratch(lst.lst_embed_grad_workspace_bytes(n, hidden, vocab))

    def call():
        grad = strided(before, pad)
        lst.lst_embed_grad(lst.matrix(dout), lst.indices(tokens), lst.matrix(grad), scale, accumulate, ws.data_ptr(),
                           ws.numel(), stream())
        return grad

    grad = call()
    t = tokens.long()
    keep = (t >= 0) & (t < vocab)
    zeros = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda")
    exact = (before.double() if accumulate else zeros.clone()).index_add(0, t[keep], dout.double()[keep] * scale)
    mass = zeros.clone().index_add_(0, t[keep], dout.double()[keep].abs() * scale)
    if accumulate:
        mass += before.double().abs()
    count = torch.zeros(vocab, 1, dtype=torch.float64, device="cuda").index_add_(
        0, t[keep], torch.ones(int(keep.sum()), 1, dtype=torch.float64, device="cuda"))
    # count additions, the scale and the sum with what was there, then one rounding to the result's type
    bound = (count + 2) * U32 * mass + (U16 if dst == "bf16" else U32) * exact.abs() * (1 + 1e-6)
    within(grad, exact, bound, "grad")
    untouched = (count[:, 0] == 0)
    assert torch.equal(grad[untouched], before[untouched] if accumulate else torch.zeros_like(before[untouched]))
    assert torch.equal(call(), grad)  # the same order of additions on every run


@pytest.mark.parametrize("n", [16383, 16384, 40001])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_many_tokens(n, accumulate):
    """Around the number of tokens from which the sort takes more CTAs: 0.25-steps, sums exact in any order."""
    vocab, hidden = 5003, 24
    g = gen(n)
    t = (torch.rand(n, generator=g, device="cuda") ** 3 * (vocab + 1)).long().to(torch.int32)  # vocab itself is outside
    dout = (torch.randint(-8, 9, (n, hidden), generator=g, device="cuda") * 0.25).float()
    before = torch.randint(-8, 9, (vocab, hidden), generator=g, device="cuda").float()
    grad = before.clone()
    ws = scratch(lst.lst_embed_grad_workspace_bytes(n, hidden, vocab))
    lst.lst_embed_grad(lst.matrix(dout), lst.indices(t), lst.matrix(grad), 0.5, accumulate, ws.data_ptr(), ws.numel(), stream())
    exact = torch.zeros(vocab + 1, hidden, dtype=torch.float64, device="cuda").index_add_(0, t.long(), dout.double())[:vocab] * 0.5
    if accumulate:
        exact += before.double()
    assert torch.equal(grad.double(), exact)


def test_embed_grad_empty_and_non_finite():
    grad = torch.ones(50, 16, device="cuda")
    none = torch.empty(0, 16, device="cuda")
    tokens = torch.empty(0, dtype=torch.int64, device="cuda")
    ws = scratch(lst.lst_embed_grad_workspace_bytes(8, 16, 50))
    args = (ws.data_ptr(), ws.numel(), stream())
    lst.lst_embed_grad(lst.matrix(none), lst.indices(tokens), lst.matrix(grad), 1.0, True, *args)
    assert (grad == 1).all()
    lst.lst_embed_grad(lst.matrix(none), lst.indices(tokens), lst.matrix(grad), 1.0, False, *args)
    assert not grad.any()
    # a NaN row that belongs to a token outside the vocabulary reaches nothing; an infinity stays in its row
    dout = torch.ones(3, 16, device="cuda")
    dout[0], dout[1, 3] = float("nan"), float("inf")
    lst.lst_embed_grad(lst.matrix(dout), lst.indices(torch.tensor([-1, 7, 8], device="cuda")), lst.matrix(grad), 1.0, False,
                       *args)
    assert torch.isinf(grad[7, 3]) and float(grad[8].sum()) == 16.0
    assert torch.isfinite(grad).sum() == 50 * 16 - 1 and float(grad[:7].abs().sum() + grad[9:].abs().sum()) == 0.0


def test_embed_grad_is_the_gradient_of_embed():
    """<grad, D> against the difference of <embed(table), r> along D: the lookup is linear."""
    g = gen(3)
    table, d, r = (randn(g, *s).double() for s in ((60, 40), (60, 40), (500, 40)))
    tokens = torch.randint(0, 60, (500,), generator=g, device="cuda")
    dout = r.float()
    grad = torch.empty(60, 40, device="cuda")
    ws = scratch(lst.lst_embed_grad_workspace_bytes(500, 40, 60))
    lst.lst_embed_grad(lst.matrix(dout), lst.indices(tokens), lst.matrix(grad), 2.0, False, ws.data_ptr(), ws.numel(),
                       stream())
    f = lambda e: float((2.0 * (table + e * d)[tokens] * dout.double()).sum())  # noqa: E731
    diff = (f(0.5) - f(-0.5))
    # fp32 sums of at most 500 terms
    assert abs(float((grad.double() * d).sum()) - diff) <= 502 * U32 * 2.0 * float((d[tokens].abs() * dout.abs()).sum())


@pytest.mark.parametrize("vocab", [(1 << 30) - 1, 1 << 30])
def test_embed_grad_largest_vocabulary(vocab):
    """Keys 0..vocab of 30 and of 31 bits; 2^30 entries is the limit."""
    tokens = torch.tensor([vocab - 1, 5, 1 << 20, vocab - 1, 1023, vocab, -1, 1 << 10, 1 << 29], device="cuda")
    dout = torch.arange(1.0, 10.0, device="cuda")[:, None].bfloat16()
    grad = torch.ones(vocab, 1, dtype=torch.bfloat16, device="cuda")
    ws = scratch(lst.lst_embed_grad_workspace_bytes(9, 1, vocab))
    lst.lst_embed_grad(lst.matrix(dout), lst.indices(tokens), lst.matrix(grad), 1.0, False, ws.data_ptr(), ws.numel(), stream())
    seen = torch.tensor([vocab - 1, 5, 1 << 20, 1023, 1 << 10, 1 << 29], device="cuda")
    assert grad[seen, 0].tolist() == [5.0, 2.0, 3.0, 5.0, 8.0, 9.0]
    assert int(torch.count_nonzero(grad)) == 6


@pytest.mark.parametrize("n", [16384, 65521])
@pytest.mark.parametrize("vocab", [511, 512, 600, 1023, 262143, 262144, 300000, 1048575])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_wide_digits(n, vocab, accumulate):
    """Digits of 9 and 10 bits, one or two passes, in the sort of many tokens: its largest shared memory."""
    hidden = 8
    g = gen(n + vocab)
    t = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) ** 2 * (vocab + 1)).long()  # vocab itself is outside
    dout = torch.randint(-8, 9, (n, hidden), generator=g, device="cuda").float()
    before = torch.randint(-8, 9, (vocab, hidden), generator=g, device="cuda").float()
    grad = before.clone()
    ws = scratch(lst.lst_embed_grad_workspace_bytes(n, hidden, vocab))
    lst.lst_embed_grad(lst.matrix(dout), lst.indices(t), lst.matrix(grad), 1.0, accumulate, ws.data_ptr(), ws.numel(), stream())
    exact = torch.zeros(vocab + 1, hidden, dtype=torch.float64, device="cuda").index_add_(0, t, dout.double())[:vocab]
    assert torch.equal(grad.double(), exact + before.double() if accumulate else exact)  # whole numbers


@pytest.mark.parametrize("n", [100, 20000])
def test_embed_grad_from_two_threads(n):
    """Sorts with much and with little shared memory, launched by two host threads on streams of their own."""
    hidden, errors = 16, []

    def work(vocab, seed):
        try:
            g = gen(seed)
            tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
            dout = torch.randint(-4, 5, (n, hidden), generator=g, device="cuda").float()
            exact = torch.zeros(vocab, hidden, device="cuda").index_add_(0, tokens, dout)  # whole numbers: exact in any order
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                ws, grad = scratch(lst.lst_embed_grad_workspace_bytes(n, hidden, vocab)), torch.empty_like(exact)
                for _ in range(500):
                    lst.lst_embed_grad(lst.matrix(dout), lst.indices(tokens), lst.matrix(grad), 1.0, False, ws.data_ptr(),
                                       ws.numel(), s.cuda_stream)
                assert torch.equal(grad, exact)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in ((2, 1), (1000, 2))]  # digits of 2 and of 10 bits
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


# ---------------------------------------------------------------------------
# cross entropy
# ---------------------------------------------------------------------------
def xent_inputs(n, hidden, vocab, seed, spread=1.0, ignored=0.1, index=torch.int64):
    g = gen(seed)
    x = randn(g, n, hidden, dtype="bf16", std=spread)
    w = randn(g, vocab, hidden, dtype="bf16", std=hidden ** -0.5)
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    out = torch.rand(n, generator=g, device="cuda") < ignored
    return x, w, torch.where(out, IGNORE, t).to(index)


def xent_exact(x, w, t, scale=1.0):
    """Definition in 64 bits, and error bounds of the library's order of operations."""
    x, w, t = x.double(), w.double(), t.long()
    n, h = x.shape
    v = w.shape[0]
    z = x @ w.T
    mass = x.abs() @ w.abs().T
    dz = 2 * h * U32 * mass                       # error of a logit
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    # lse moves by at most the largest logit error; exp and the sums in fp32: 2 ulp per term, log2(V/128)
    # levels of joining; the logarithm and its sum with the maximum
    dlse = dz.max(1).values + (8 + math.log2(v + 1)) * 4 * U32 + 4 * U32 * lse.abs() + 4 * U32 * z.abs().max(1).values
    keep = t != IGNORE
    at = torch.where(keep, t, 0)[:, None]
    loss = torch.where(keep, lse - z.gather(1, at)[:, 0], 0.0)
    dloss = dlse + dz.gather(1, at)[:, 0] + U32 * loss.abs()
    count = int(keep.sum())
    d = p.clone().scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float64))
    d = torch.where(keep[:, None], d, 0.0) * (scale / max(1, count))
    # logit gradient: fixed point of 2^-12 in the exponent, logit and lse errors in it, rounding to bf16;
    # the target's entry from its own fp32 difference; entries more than 32 below their group's maximum saturate
    rel = 2.0 ** -12 * 1.01 + (dz + dlse[:, None]) * 1.01 + 64 * U32 + U16
    dd = rel * p * (scale / max(1, count)) + U16 * d.abs() + math.exp(-32) * scale / max(1, count)
    dd = torch.where(keep[:, None], dd.abs(), 0.0)
    return dict(loss=loss, lse=lse, dloss=dloss, dlse=dlse, d=d, dd=dd, dx=d @ w, dw=d.T @ x,
                bx=dd @ w.abs() + 2 * v * U32 * (d.abs() @ w.abs()),
                bw=dd.T @ x.abs() + 2 * n * U32 * (d.abs().T @ x.abs()),
                mean=float(loss.sum() / max(1, count)), count=count)


def xent_call(x, w, t, grad=True, scale=1.0, ws_bytes=None, dw=None, accumulate=False, pad=0, extra=0):
    n, h = x.shape
    v = w.shape[0]
    loss, lse = (torch.full((n,), -1.0, device="cuda") for _ in range(2))
    ws = scratch((lst.lst_xent_workspace_bytes(n, h, v, grad) if ws_bytes is None else ws_bytes) + extra)
    if not grad:
        lst.lst_xent_loss(lst.matrix(x), lst.matrix(w), lst.indices(t), IGNORE, loss.data_ptr(), lse.data_ptr(),
                          ws.data_ptr(), ws.numel(), stream())
        return dict(loss=loss, lse=lse)
    mean = torch.full((1,), -1.0, device="cuda")
    dx = strided(torch.zeros(n, h, dtype=torch.bfloat16, device="cuda"), pad)
    dw = strided(torch.zeros(v, h, dtype=torch.bfloat16, device="cuda"), pad) if dw is None else dw
    lst.lst_xent_grad(lst.matrix(x), lst.matrix(w), lst.indices(t), IGNORE, scale, loss.data_ptr(), lse.data_ptr(),
                      mean.data_ptr(), lst.matrix(dx), lst.matrix(dw), accumulate, ws.data_ptr(), ws.numel(), stream())
    return dict(loss=loss, lse=lse, mean=mean, dx=dx, dw=dw)


def xent_check(r, e, grad=True):
    within(r["lse"], e["lse"], e["dlse"], "lse")
    within(r["loss"], e["loss"], e["dloss"], "loss")
    if grad:
        assert abs(float(r["mean"]) - e["mean"]) <= float(e["dloss"].max()) + U32 * abs(e["mean"])
        within(r["dx"], e["dx"], e["bx"] + U16 * (e["dx"].abs() + e["bx"]), "dx")
        within(r["dw"], e["dw"], e["bw"] + U16 * (e["dw"].abs() + e["bw"]), "dw")
    lst.lst_operator_status()


XENT_SIZES = [(1, 8, 1), (1, 64, 500), (2, 16, 127), (16, 2048, 1000), (31, 40, 128), (33, 72, 129), (128, 64, 256),
              (255, 136, 257), (256, 256, 512), (257, 264, 5003), (600, 1000, 777), (1023, 520, 2049), (300, 2048, 4096)]


@pytest.mark.parametrize("n,hidden,vocab", XENT_SIZES)
def test_xent(n, hidden, vocab):
    x, w, t = xent_inputs(n, hidden, vocab, seed=n + vocab, ignored=0.1 if n > 1 else 0.0,
                          index=torch.int32 if n % 2 else torch.int64)
    e = xent_exact(x, w, t)
    r = xent_call(x, w, t)
    xent_check(r, e)
    only = xent_call(x, w, t, grad=False)
    assert torch.equal(only["loss"], r["loss"]) and torch.equal(only["lse"], r["lse"])
    again = xent_call(x, w, t)
    assert all(torch.equal(again[k], r[k]) for k in r)


@pytest.mark.parametrize("n,hidden,vocab", [(700, 264, 7001), (700, 1000, 3500)])
def test_xent_more_tiles_than_pairs(n, hidden, vocab):
    """84 tiles of logits, and 112 or 56 of dw with those of dx: a second wave of few tiles, which are formed in halves."""
    x, w, t = xent_inputs(n, hidden, vocab, seed=42)
    xent_check(xent_call(x, w, t), xent_exact(x, w, t))


@pytest.mark.parametrize("n", [1, 15, 17, 32, 48, 63, 64, 65])
def test_xent_few_tokens(n):
    """Tokens as the columns of narrow tiles (up to 64), more tiles than pairs, a vocabulary that ends inside one."""
    x, w, t = xent_inputs(n, 136, 40021, seed=n, ignored=0.0)
    t[-1] = 40020
    e = xent_exact(x, w, t)
    r = xent_call(x, w, t)
    xent_check(r, e)
    only = xent_call(x, w, t, grad=False)
    assert torch.equal(only["loss"], r["loss"]) and torch.equal(only["lse"], r["lse"])


@pytest.mark.parametrize("hidden,pad,shift", [(77, 0, 0), (1, 0, 0), (64, 3, 0), (64, 0, 1), (72, 8, 4), (63, 1, 0), (130, 6, 2)])
def test_xent_strides_and_odd_rows(hidden, pad, shift):
    """Rows that do not start on 16 bytes, padded rows, bases off 16 bytes."""
    n, vocab = 130, 300
    x, w, t = xent_inputs(n, hidden, vocab, seed=hidden)
    e = xent_exact(x, w, t)
    extra = 2 * (n + vocab) * (hidden + 8) + 1024
    r = xent_call(strided(x, pad, shift), strided(w, pad, shift), t, pad=pad, extra=extra)
    xent_check(r, e)


@pytest.mark.parametrize("n,hidden,vocab,pad,shift", [(130, 64, 300, 3, 0), (130, 64, 300, 0, 1), (16, 2048, 5000, 0, 1),
                                                      (16, 256, 5000, 4, 0), (130, 72, 300, 8, 4), (130, 77, 300, 0, 0),
                                                      (300, 64, 4000, 1, 3), (33, 104, 1000, 8, 0)])
@pytest.mark.parametrize("which", ["x", "w", "xw"])
def test_xent_workspace_for_strides(n, hidden, vocab, pad, shift, which):
    """Operands off 16 bytes in a workspace of exactly the size that is given for them: one piece, the results of
    contiguous operands bit for bit."""
    x, w, t = xent_inputs(n, hidden, vocab, seed=hidden + n)
    ref = xent_call(x, w, t)
    xs = strided(x, pad, shift) if "x" in which else x
    ws = strided(w, pad, shift) if "w" in which else w
    r = xent_call(xs, ws, t, ws_bytes=lst.lst_xent_workspace_bytes_for(lst.matrix(xs), lst.matrix(ws), True))
    assert all(torch.equal(r[k], ref[k]) for k in ref)
    only = xent_call(xs, ws, t, grad=False, ws_bytes=lst.lst_xent_workspace_bytes_for(lst.matrix(xs), lst.matrix(ws), False))
    assert torch.equal(only["loss"], ref["loss"]) and torch.equal(only["lse"], ref["lse"])


@pytest.mark.parametrize("n,hidden,vocab", [(300, 264, 5003), (40, 64, 3000), (1030, 96, 1500)])
def test_xent_small_workspaces(n, hidden, vocab):
    """Down to pieces of 256 columns: the same loss bit for bit, gradients within the same bounds."""
    x, w, t = xent_inputs(n, hidden, vocab, seed=5)
    e = xent_exact(x, w, t)
    full = lst.lst_xent_workspace_bytes(n, hidden, vocab, True)
    whole = xent_call(x, w, t)
    size, tried = full, 0
    while tried < 12:
        size = int(size * 0.8)
        try:
            r = xent_call(x, w, t, ws_bytes=size)
        except lst.LstError as err:
            assert err.status == lst.LST_ERR_INVALID_ARG
            break
        assert torch.equal(r["loss"], whole["loss"])
        xent_check(r, e)
        tried += 1
    assert tried >= 2


@pytest.mark.parametrize("most,n", [(65, 64), (200, 64), (300, 256), (600, 33), (1030, 700), (300, 300)])
def test_xent_workspace_of_a_larger_batch(most, n):
    """The workspace for the largest batch serves a shorter one in one piece: the results of its own workspace."""
    hidden, vocab = 264, 5003
    x, w, t = xent_inputs(n, hidden, vocab, seed=most + n)
    ref, large = xent_call(x, w, t), xent_call(x, w, t, ws_bytes=lst.lst_xent_workspace_bytes(most, hidden, vocab, True))
    assert all(torch.equal(large[k], ref[k]) for k in ref)
    only = xent_call(x, w, t, grad=False, ws_bytes=lst.lst_xent_workspace_bytes(most, hidden, vocab, False))
    assert torch.equal(only["loss"], ref["loss"])
    xent_check(large, xent_exact(x, w, t))


def test_xent_ignored_rows_reach_nothing():
    n, hidden, vocab = 300, 128, 1000
    x, w, t = xent_inputs(n, hidden, vocab, seed=8, ignored=0.3)
    out = t == IGNORE
    clean = x.clone()
    clean[out] = 0
    e = xent_exact(clean, w, t)
    x[out] = float("nan")
    x[out.nonzero()[0]] = float("inf")
    r = xent_call(x, w, t)
    assert (r["loss"][out] == 0).all() and not r["dx"][out].any()
    within(r["loss"], e["loss"], e["dloss"], "loss")
    within(r["dx"], e["dx"], e["bx"] + U16 * (e["dx"].abs() + e["bx"]), "dx")
    within(r["dw"], e["dw"], e["bw"] + U16 * (e["dw"].abs() + e["bw"]), "dw")


def test_xent_all_ignored_and_outside_targets():
    n, hidden, vocab = 70, 64, 400
    x, w, t = xent_inputs(n, hidden, vocab, seed=9, ignored=0.0)
    r = xent_call(x, w, torch.full_like(t, IGNORE))
    assert not r["loss"].any() and float(r["mean"]) == 0.0 and not r["dx"].any() and not r["dw"].any()
    keep = torch.full((vocab, hidden), 3.0, dtype=torch.bfloat16, device="cuda")
    r = xent_call(x, w, torch.full_like(t, IGNORE), dw=keep, accumulate=True)
    assert (keep == 3.0).all()
    bad = t.clone()
    bad[5], bad[6] = vocab, -7
    r = xent_call(x, w, bad)
    assert torch.isnan(r["loss"][[5, 6]]).all() and torch.isfinite(r["loss"]).sum() == n - 2
    assert not r["dx"][[5, 6]].any() and torch.isfinite(r["dx"]).all() and torch.isfinite(r["dw"]).all()
    # no targets at all
    none = torch.empty(0, hidden, dtype=torch.bfloat16, device="cuda")
    r = xent_call(none, w, t[:0])
    assert float(r["mean"]) == 0.0 and not r["dw"].any()


@pytest.mark.parametrize("spread", [0.0, 30.0, 300.0])
def test_xent_range_of_logits(spread):
    """Equal logits, and logits hundreds apart (probabilities of 0 and 1)."""
    x, w, t = xent_inputs(90, 64, 700, seed=11, spread=spread)
    top = (x.double() @ w.double().T).argmax(1)
    t[::2] = torch.where(t[::2] != IGNORE, top[::2], t[::2])  # half the targets are near certain
    xent_check(xent_call(x, w, t), xent_exact(x, w, t))


def test_xent_non_finite_rows_stay_in_their_rows():
    x, w, t = xent_inputs(64, 64, 300, seed=12, ignored=0.0)
    x[3, 5], x[9] = float("nan"), float("inf")
    r = xent_call(x, w, t)
    ok = torch.ones(64, dtype=torch.bool, device="cuda")
    ok[[3, 9]] = False
    assert torch.isnan(r["loss"][~ok]).all() and torch.isfinite(r["loss"][ok]).all()
    assert torch.isnan(r["dx"][~ok]).any(1).all() and not torch.isnan(xent_call(x, w, t, grad=False)["loss"][ok]).any()


@pytest.mark.parametrize("pieces", [1, 2])
def test_xent_logits_of_minus_infinity(pieces):
    """A vocabulary row whose logits pass below the type's range: probability 0, gradient 0 except where it is the target."""
    n, hidden, vocab, gone = 40, 64, 300, 7
    x, w, t = xent_inputs(n, hidden, vocab, seed=17, ignored=0.0)
    x = x.abs() + 0.5
    others = torch.arange(vocab, device="cuda") != gone
    t = torch.where(t == gone, gone + 1, t)
    e = xent_exact(x, w[others], t - (t > gone).long())
    w[gone] = torch.finfo(torch.bfloat16).min
    t[0] = gone
    scale = 1.0 / n
    z = x.double() @ w[others].double().T
    d = torch.zeros(n, vocab, dtype=torch.float64, device="cuda")
    d[:, others] = torch.softmax(z, 1) * scale
    d[torch.arange(n), t] -= scale
    dd = torch.zeros_like(d)
    dd[:, others] = e["dd"]
    dd[torch.arange(n), t] += U16 * scale
    dx, dw = d @ w.double(), d.T @ x.double()
    bx = dd @ w.double().abs() + 2 * vocab * U32 * (d.abs() @ w.double().abs())
    bw = dd.T @ x.double().abs() + 2 * n * U32 * (d.abs().T @ x.double().abs())
    size = lst.lst_xent_workspace_bytes(n, hidden, vocab, True)
    r = xent_call(x, w, t, ws_bytes=size if pieces == 1 else size - 1)
    assert torch.isinf(r["loss"][0]) and float(r["mean"]) == math.inf
    within(r["lse"], e["lse"], e["dlse"], "lse")
    within(r["loss"][1:], e["loss"][1:], e["dloss"][1:], "loss")
    within(r["dx"], dx, bx + U16 * (dx.abs() + bx), "dx")
    within(r["dw"], dw, bw + U16 * (dw.abs() + bw), "dw")
    only = xent_call(x, w, t, grad=False)
    assert torch.equal(only["loss"], r["loss"]) and torch.equal(only["lse"], r["lse"])


def test_xent_scale_and_accumulate():
    n, hidden, vocab = 200, 104, 900
    x, w, t = xent_inputs(n, hidden, vocab, seed=13)
    e = xent_exact(x, w, t, scale=64.0)
    before = randn(gen(14), vocab, hidden, dtype="bf16", std=0.1)
    dw = before.clone()
    r = xent_call(x, w, t, scale=64.0, dw=dw, accumulate=True)
    e["dw"] = e["dw"] + before.double()
    xent_check(r, e)


def test_xent_gradient_against_differences():
    """The mean loss in 64 bits, differenced along a direction, against <dx, D> and <dw, D>."""
    n, hidden, vocab = 120, 64, 500
    x, w, t = xent_inputs(n, hidden, vocab, seed=15)
    e = xent_exact(x, w, t)
    r = xent_call(x, w, t)
    g = gen(16)
    dx, dw = randn(g, n, hidden).double(), randn(g, vocab, hidden).double()
    keep = (t != IGNORE).nonzero()[:, 0]

    def f(eps, which):
        z = (x.double() + (eps * dx if which == "x" else 0)) @ (w.double() + (eps * dw if which == "w" else 0)).T
        return float((torch.logsumexp(z, 1)[keep] - z[keep, t[keep]]).mean())

    h = 1e-4  # the difference's own error: h^2 times a third derivative of order |D|^3
    for which, direction, got, bound in (("x", dx, r["dx"], e["bx"]), ("w", dw, r["dw"], e["bw"])):
        diff = (f(h, which) - f(-h, which)) / (2 * h)
        limit = float(((bound + U16 * got.double().abs()) * direction.abs()).sum()) + 1e-5
        assert abs(float((got.double() * direction).sum()) - diff) <= limit


# ---------------------------------------------------------------------------
# Newton-Schulz and Muon
# ---------------------------------------------------------------------------
COEF = (3.4445, -4.7750, 2.0315)


def ns_exact(u, steps=5, eps=1e-7):
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (x.norm() + eps)
    a, b, c = COEF
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    return x.T if tall else x


# A step stores X and up to five m x m products in fp16 (relative error uh each); near its fixed points the iteration
# passes an error on with a factor of at most 1.6 (the largest slope of a s + b s^3 + c s^5 there), in the directions
# that are still growing with 3.45, as the values themselves do: per step 6 uh, over 5 steps with a factor of 1.6 from
# step to step no more than 6 uh (1.6^5 - 1) / 0.6 in the 2-norm, taken half as large for roundings that do not line up
# (they are independent), plus the result's rounding to bf16.
NS_TOL = 0.5 * 6 * UH * (1.6 ** 5 - 1) / 0.6 + U16


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def ns_call(xs, steps=5, ws_bytes=None, outs=None, eps=1e-7):
    outs = [torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda") for x in xs] if outs is None else outs
    r, c = xs[0].shape
    ws = scratch(lst.lst_orthogonalize_workspace_bytes(len(xs), r, c) if ws_bytes is None else ws_bytes)
    lst.lst_orthogonalize([lst.matrix(x) for x in xs], [lst.matrix(o) for o in outs], lst.ns_params(steps, eps),
                          ws.data_ptr(), ws.numel(), stream())
    lst.lst_operator_status()
    return outs


def matrix_like(g, r, c, std=1e-3):
    k = max(1, min(16, min(r, c) // 4))
    low = randn(g, r, k) * (torch.arange(1, k + 1, device="cuda") ** -0.5) @ randn(g, k, c) / 3
    return (low + 0.5 * randn(g, r, c)) * std


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (16, 16), (17, 33), (64, 200), (200, 64), (128, 128),
                                       (255, 257), (256, 256), (257, 256), (300, 1030), (1030, 300), (513, 2049), (1000, 1001),
                                       (2048, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize(rows, cols, dtype):
    x = matrix_like(gen(rows * 7 + cols), rows, cols).to(DT[dtype])
    out = ns_call([x])[0]
    assert rel(out, ns_exact(x)) <= NS_TOL
    assert torch.equal(ns_call([x])[0], out)
    if min(rows, cols) > 4:
        s = torch.linalg.svdvals(out.double())
        # every singular value of these inputs is over a hundredth of the largest: all end near 1
        assert float(s.max()) < 1.25


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 8])
@pytest.mark.parametrize("rows,cols", [(96, 96), (96, 400)])  # single steps, and pairs of steps
def test_orthogonalize_steps(steps, rows, cols):
    x = matrix_like(gen(steps), rows, cols)
    tol = 0.5 * 6 * UH * (1.6 ** max(5, steps) - 1) / 0.6 + U16
    assert rel(ns_call([x], steps)[0], ns_exact(x, steps)) <= tol


@pytest.mark.parametrize("count,rows,cols", [(3, 130, 257), (9, 64, 48), (40, 20, 33)])
def test_orthogonalize_batches_and_strides(count, rows, cols):
    xs = [strided(matrix_like(gen(i), rows, cols).bfloat16(), 3) for i in range(count)]
    big = torch.full((rows, cols + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    outs = [big[:, 1:cols + 1] if i == 1 else torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
            for i in range(count)]
    ns_call(xs, outs=outs)
    for x, o in zip(xs, outs):
        assert rel(o, ns_exact(x)) <= NS_TOL
    assert (big[:, 0] == 7).all() and (big[:, cols + 1:] == 7).all()
    # one or a few matrices at a time: the same bits
    one = lst.lst_orthogonalize_workspace_bytes(1, rows, cols)
    for size in (one, 2 * one + 100):
        again = [torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(count)]
        ns_call(xs, ws_bytes=size, outs=again)
        assert all(torch.equal(a, o) for a, o in zip(again, outs))


@pytest.mark.parametrize("rows,cols", [(1300, 1700), (1703, 1301)])
def test_orthogonalize_more_tiles_than_pairs(rows, cols):
    """21 tiles of a symmetric product and 42 of X by four: a second wave of few tiles, which are formed in halves."""
    xs = [matrix_like(gen(40 + i), rows, cols).bfloat16() for i in range(4)]
    for x, o in zip(xs, ns_call(xs)):
        assert rel(o, ns_exact(x)) <= NS_TOL


def test_orthogonalize_zero_tiny_large_and_non_finite():
    g = gen(20)
    good = matrix_like(g, 100, 130)
    zero, nan = torch.zeros_like(good), good.clone()
    nan[3, 4] = float("nan")
    small, large = good * 1e-12, good * 1e15
    outs = ns_call([good, zero, nan, small, large])
    assert rel(outs[0], ns_exact(good)) <= NS_TOL
    assert not outs[1].any()
    assert torch.isnan(outs[2]).any()
    assert rel(outs[3], ns_exact(small)) <= NS_TOL   # |U|_F under eps: the result is as small as the formula's
    assert rel(outs[4], ns_exact(large)) <= NS_TOL


@pytest.mark.parametrize("rows,cols", [(100, 130), (300, 1030), (520, 200)])
@pytest.mark.parametrize("eps", [1e-20, 1e-36, 1e-40, 1e-45])
def test_orthogonalize_small_eps(rows, cols, eps):
    """Any eps above zero, the smallest number of fp32 among them: zero stays zero, others do not notice it."""
    x = matrix_like(gen(50), rows, cols)
    zero, out, low = ns_call([torch.zeros_like(x), x, x * 2.0 ** -50], eps=eps)
    assert not zero.any() and torch.isfinite(zero).all()
    assert rel(out, ns_exact(x, eps=float(np.float32(eps)))) <= NS_TOL
    assert rel(low, ns_exact(x * 2.0 ** -50, eps=float(np.float32(eps)))) <= NS_TOL


@pytest.mark.parametrize("rows,cols", [(100, 130), (128, 4000), (300, 1030), (1031, 301), (640, 512)])
@pytest.mark.parametrize("scale,eps", [(2.0 ** 69, 1e-7), (2.0 ** 110, 1e-7), (2.0 ** 130, 1e-7), (2.0 ** -78, 1e-37),
                                       (2.0 ** -105, 1e-45), (2.0 ** -90, 2.0 ** -95), (2.0 ** 100, 2.0 ** 100)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize_far_from_one(rows, cols, scale, eps, dtype):
    """Entries whose squares leave the range of fp32 at either end; at 2^130 |U|_F leaves it too."""
    x = (matrix_like(gen(51), rows, cols).double() * scale).to(DT[dtype])
    assert torch.isfinite(x).all() and int(torch.count_nonzero(x)) > 0.99 * x.numel()
    out, zero = ns_call([x, torch.zeros_like(x)], eps=eps)
    assert rel(out, ns_exact(x, eps=float(np.float32(eps)))) <= NS_TOL and not zero.any()


@pytest.mark.parametrize("rows,cols", [(90, 700), (700, 600)])
def test_orthogonalize_of_mixed_magnitudes(rows, cols):
    """Rows whose squares overflow, rows in the ordinary range, rows whose squares underflow, in one matrix; and
    matrices of each kind in one call."""
    x = matrix_like(gen(52), rows, cols)
    third = rows // 3
    parts = torch.ones(rows, 1, device="cuda")
    parts[:third], parts[2 * third:] = 2.0 ** 80, 2.0 ** -80
    mixed, low, high = x * parts, x.clone(), x.clone()
    low[:third] *= 2.0 ** -70
    high[0] *= 2.0 ** 75
    xs = [mixed, low, high, x, x * 2.0 ** -110, x * 2.0 ** 90]
    for got, a in zip(ns_call(xs, eps=1e-40), xs):
        assert rel(got, ns_exact(a, eps=float(np.float32(1e-40)))) <= NS_TOL


@pytest.mark.parametrize("fmt", ["L12", "L16F"])
@pytest.mark.parametrize("scale", [2.0 ** 75, 2.0 ** -75])
def test_muon_step_far_from_one(fmt, scale):
    """Gradients and momentum far from one in matrices of the one-kernel form and of the tiled one."""
    shapes = [(24, 96), (300, 403), (400, 304)]
    layout = Layout([(f"m{i}", s, 0) for i, s in enumerate(shapes)], fmt)
    blk = torch.zeros(layout.block_bytes(0), dtype=torch.uint8, device="cuda")
    v = muon_views(layout, fmt, 0, blk)
    g = gen(53)
    for (_, off, n), shape in zip(layout.spans(0), shapes):
        v["W"][off:off + n] = torch.randn(n, generator=g, device="cuda") * 0.02
        for f in ("G", "M"):
            v[f][off:off + n] = (matrix_like(g, *shape) * scale).reshape(-1)
    old = {f: x.clone() for f, x in v.items()}
    ws = scratch(lst.lst_muon_workspace_bytes(layout.handle))
    hp = lst.muon_hparams(lr=2e-2, momentum=0.9, weight_decay=0.1, rms_scale=0.2, eps=1e-40)
    lst.lst_muon_step(layout.handle, [blk.data_ptr()], hp, None, None, ws.data_ptr(), ws.numel(), stream())
    lst.lst_operator_status()
    for (name, off, n), shape in zip(layout.spans(0), shapes):
        s = slice(off, off + n)
        m = (old["M"][s] * np.float32(0.9)) + old["G"][s].float()
        assert torch.equal(v["M"][s], m), name  # once, although its sum of squares is taken twice
        u = old["G"][s].double() + float(np.float32(0.9)) * m.double()
        o = ns_exact(u.view(shape), eps=float(np.float32(1e-40))).reshape(-1)
        rms, w0 = 0.2 * math.sqrt(max(shape)), old["W"][s].double()
        w = w0 * (1 - 2e-2 * 0.1) - 2e-2 * rms * o
        limit = NS_TOL * 2e-2 * rms * o.norm() + 4 * U32 * (w0.norm() + w.norm()) + (U16 * w.norm() if fmt == "L12" else 0.0)
        assert float((v["W"][s].double() - w).norm()) <= float(limit), name


def test_orthogonalize_decaying_singular_values():
    """Values falling as 1/i over three decades: the smallest are still growing after five steps, by 3.45 a step, and
    so is their rounding: one more factor of 1.6 in the bound."""
    g = gen(21)
    n = 512
    u = torch.linalg.qr(randn(g, n, n).double())[0]
    v = torch.linalg.qr(randn(g, 1500, n).double())[0]
    x = ((u / torch.arange(1, n + 1, device="cuda")) @ v.T).float()
    assert rel(ns_call([x])[0], ns_exact(x)) <= 1.6 * NS_TOL


SPECS = [("q", (96, 96), 0), ("k", (24, 96), 0), ("norm", (96,), 0), ("up", (250, 96), 0), ("down", (96, 250), 1),
         ("odd", (33, 77), 1), ("scalar", (), 1), ("bias", (1000,), 1), ("conv", (4, 3, 5), 1), ("empty", (0, 7), 1)]
FMT_FIELDS = {"L12": ("W", "M", "V"), "L16M": ("MASTER", "M", "V", "W"), "L16F": ("W", "M", "V")}


def muon_blocks(layout, fmt, seed, guard=4096):
    """Blocks between canaries, tensors filled, padding zero."""
    g = gen(seed)
    blocks, backing = [], []
    for b in range(layout.n_layers):
        n = layout.block_bytes(b)
        full = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        blk = full[guard:guard + n]
        blk.zero_()
        views = muon_views(layout, fmt, b, blk)
        for name, off, n in layout.spans(b):
            shape = dict((s[0], s[1]) for s in SPECS)[name]
            w = torch.randn(n, generator=g, device="cuda") * 0.02
            for f in ("MASTER", "W"):
                if f in views:
                    views[f][off:off + n] = w
            for f in ("G", "M"):
                x = matrix_like(g, *shape).reshape(-1) if len(shape) == 2 and n else torch.randn(n, generator=g, device="cuda") * 1e-3
                views[f][off:off + n] = x
            views["V"][off:off + n] = (torch.randn(n, generator=g, device="cuda") * 1e-3) ** 2
        blocks.append(blk)
        backing.append(full)
    return blocks, backing


def muon_views(layout, fmt, b, blk):
    v = layout.torch_views(b, blk)
    return {f: (x.view(torch.bfloat16) if x.dtype == torch.int16 else x) for f, x in v.items()}


@pytest.mark.parametrize("fmt", ["L12", "L16M", "L16F"])
@pytest.mark.parametrize("nesterov,rms_scale,steps", [(True, 0.2, 5), (False, 0.0, 5), (True, 0.2, 3)])
def test_muon_step(fmt, nesterov, rms_scale, steps):
    layout = Layout(SPECS, fmt)
    blocks, backing = muon_blocks(layout, fmt, 30)
    before = [b.clone() for b in blocks]
    adam = [b.clone() for b in blocks]
    hp = lst.muon_hparams(lr=2e-2, momentum=0.9, weight_decay=0.1, rms_scale=rms_scale, nesterov=nesterov, ns_steps=steps)
    ahp = lst.adamw_hparams(lr=1e-3, step=4)
    ws = scratch(lst.lst_muon_workspace_bytes(layout.handle))
    lst.lst_muon_step(layout.handle, [b.data_ptr() for b in blocks], hp, ahp, None, ws.data_ptr(), ws.numel(), stream())
    lst.lst_adamw_step(layout.handle, [b.data_ptr() for b in adam], ahp, stream())
    lst.lst_operator_status()
    for b in range(layout.n_layers):
        got, old, ref = (muon_views(layout, fmt, b, x[b]) for x in (blocks, before, adam))
        assert torch.equal(got["G"], old["G"])
        covered = torch.zeros(layout.padded(b), dtype=torch.bool, device="cuda")
        for name, off, n in layout.spans(b):
            shape = dict((s[0], s[1]) for s in SPECS)[name]
            s = slice(off, off + n)
            covered[s] = True
            if len(shape) != 2:
                for f in FMT_FIELDS[fmt]:  # the update of lst_adamw_step, bit for bit
                    assert torch.equal(got[f][s], ref[f][s]), (name, f)
                continue
            if n == 0:
                continue
            assert torch.equal(got["V"][s], old["V"][s])
            m = (old["M"][s] * np.float32(0.9)) + old["G"][s].float()      # two fp32 operations
            assert torch.equal(got["M"][s], m), name
            u = old["G"][s].double() + float(np.float32(0.9)) * m.double() if nesterov else m.double()
            o = ns_exact(u.view(shape), steps).reshape(-1)
            scale = rms_scale * math.sqrt(max(shape)) if rms_scale else math.sqrt(max(1.0, shape[0] / shape[1]))
            field = "MASTER" if fmt == "L16M" else "W"
            w0 = old[field][s].double()
            w = w0 * (1 - 2e-2 * 0.1) - 2e-2 * scale * o
            err = (got[field][s].double() - w).norm()
            # the update to NS_TOL (its fp16 result, without the rounding to bf16, is nearer), the weight's arithmetic in fp32
            limit = NS_TOL * 2e-2 * scale * o.norm() + 4 * U32 * (w0.norm() + w.norm())
            if fmt == "L12":
                limit = limit + U16 * w.norm()
            assert float(err) <= float(limit), (name, float(err), float(limit))
            if fmt == "L16M":
                assert torch.equal(got["W"][s], got["MASTER"][s].bfloat16())
        for f in FMT_FIELDS[fmt]:
            assert not got[f][~covered].any(), f                              # padding stays zero
        assert (backing[b][:4096] == 0xA5).all() and (backing[b][-4096:] == 0xA5).all()


@pytest.mark.parametrize("fmt", ["L12", "L16M", "L16F"])
def test_muon_step_more_tiles_than_pairs(fmt):
    """Matrices of one long side and of two, so that launches hold sums of different lengths and a wave of half tiles."""
    shapes = [(1304, 1304), (1704, 1304), (1304, 1704), (1304, 1701)]
    layout = Layout([(f"m{i}", s, 0) for i, s in enumerate(shapes)], fmt)
    blk = torch.zeros(layout.block_bytes(0), dtype=torch.uint8, device="cuda")
    v = muon_views(layout, fmt, 0, blk)
    spans = list(layout.spans(0))
    field = "MASTER" if fmt == "L16M" else "W"
    g = gen(41)
    for (_, off, n), shape in zip(spans, shapes):
        v[field][off:off + n] = torch.randn(n, generator=g, device="cuda") * 0.02
        v["G"][off:off + n] = matrix_like(g, *shape).reshape(-1)
        v["M"][off:off + n] = matrix_like(g, *shape).reshape(-1)
    old = {f: x.clone() for f, x in v.items()}
    ws = scratch(lst.lst_muon_workspace_bytes(layout.handle))
    hp = lst.muon_hparams(lr=2e-2, momentum=0.9, weight_decay=0.1, rms_scale=0.2, nesterov=True)
    lst.lst_muon_step(layout.handle, [blk.data_ptr()], hp, None, None, ws.data_ptr(), ws.numel(), stream())
    lst.lst_operator_status()
    covered = torch.zeros(layout.padded(0), dtype=torch.bool, device="cuda")
    for (name, off, n), shape in zip(spans, shapes):
        s = slice(off, off + n)
        covered[s] = True
        m = (old["M"][s] * np.float32(0.9)) + old["G"][s].float()
        assert torch.equal(v["M"][s], m), name
        o = ns_exact((old["G"][s].double() + float(np.float32(0.9)) * m.double()).view(shape)).reshape(-1)
        scale, w0 = 0.2 * math.sqrt(max(shape)), old[field][s].double()
        w = w0 * (1 - 2e-2 * 0.1) - 2e-2 * scale * o
        limit = NS_TOL * 2e-2 * scale * o.norm() + (4 * U32 * (w0.norm() + w.norm())) + (U16 * w.norm() if fmt == "L12" else 0.0)
        err = (v[field][s].double() - w).norm()
        assert float(err) <= float(limit), (name, float(err), float(limit))
        if fmt == "L16M":
            assert torch.equal(v["W"][s], v["MASTER"][s].bfloat16())
    assert not v["M"][~covered].any() and not v[field][~covered].any()


# Roundings that do not line up add by their squares: a value rounded to fp16 is off by 0.4 uh (rms, over a binade);
# six such in a step, passed on with a factor of 1.6 from step to step, give 0.4 uh sqrt(6 sum 1.6^2k), k = 0..4, and
# the result's rounding to bf16 0.4 u16: 4.3e-3, taken as 5e-3.
NS_TIGHT = 5e-3


@pytest.mark.parametrize("rows,cols", [(64, 200), (128, 128), (128, 1000), (200, 64), (136, 144), (256, 256), (256, 1030), (300, 1030),
                                       (1030, 300), (513, 2049), (1600, 900)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize_coefficients(rows, cols, dtype):
    """Near enough that a coefficient off by 0.005 would show."""
    x = matrix_like(gen(60), rows, cols).to(DT[dtype])
    assert rel(ns_call([x])[0], ns_exact(x)) <= NS_TIGHT


def test_orthogonalize_tolerance_tells_coefficients():
    """What the bound above refuses: the definition in 64 bits with one coefficient changed."""
    x = matrix_like(gen(60), 300, 1030).cpu()
    exact = ns_exact(x)
    global COEF
    kept = COEF
    try:
        for i, d in ((0, 0.005), (0, -0.005), (1, 0.01), (1, -0.01), (2, 0.01), (2, -0.01)):
            COEF = tuple(c + (d if k == i else 0.0) for k, c in enumerate(kept))
            assert rel(ns_exact(x), exact) > 2 * NS_TIGHT
    finally:
        COEF = kept


def muon_shapes(shapes, fmt, seed):
    layout = Layout([(f"m{i}", s, 0) for i, s in enumerate(shapes)], fmt)
    blk = torch.zeros(layout.block_bytes(0), dtype=torch.uint8, device="cuda")
    v = muon_views(layout, fmt, 0, blk)
    g = gen(seed)
    for (_, off, n), shape in zip(layout.spans(0), shapes):
        v["MASTER" if fmt == "L16M" else "W"][off:off + n] = torch.randn(n, generator=g, device="cuda") * 0.02
        for f in ("G", "M"):
            v[f][off:off + n] = matrix_like(g, *shape).reshape(-1)
    return layout, blk


def muon_check(layout, fmt, shapes, old_blk, blk):
    """Weights, momenta and derived weights of a step with lr 0.02, momentum 0.9, decay 0.1, rms scale 0.2, nesterov."""
    old, new = muon_views(layout, fmt, 0, old_blk), muon_views(layout, fmt, 0, blk)
    field = "MASTER" if fmt == "L16M" else "W"
    for (name, off, n), shape in zip(layout.spans(0), shapes):
        s = slice(off, off + n)
        m = (old["M"][s] * np.float32(0.9)) + old["G"][s].float()
        assert torch.equal(new["M"][s], m), name
        o = ns_exact((old["G"][s].double() + float(np.float32(0.9)) * m.double()).view(shape)).reshape(-1)
        rms, w0 = 0.2 * math.sqrt(max(shape)), old[field][s].double()
        w = w0 * (1 - 2e-2 * 0.1) - 2e-2 * rms * o
        limit = NS_TIGHT * 2e-2 * rms * o.norm() + 4 * U32 * (w0.norm() + w.norm()) + (U16 * w.norm() if fmt == "L12" else 0.0)
        assert float((new[field][s].double() - w).norm()) <= float(limit), name
        if fmt == "L16M":
            assert torch.equal(new["W"][s], new["MASTER"][s].bfloat16())


def muon_call(layout, blk, ws_bytes):
    ws = scratch(ws_bytes)
    hp = lst.muon_hparams(lr=2e-2, momentum=0.9, weight_decay=0.1, rms_scale=0.2, nesterov=True)
    lst.lst_muon_step(layout.handle, [blk.data_ptr()], hp, None, None, ws.data_ptr(), ws.numel(), stream())
    lst.lst_operator_status()


@pytest.mark.parametrize("fmt", ["L12", "L16M", "L16F"])
@pytest.mark.parametrize("shapes", [[(300, 404)] * 3 + [(404, 300)] * 2 + [(300, 403)] * 2 + [(24, 96)] * 3 + [(96, 24)],
                                    [(136, 144)] * 70 + [(24, 40)] * 60, [(700, 200)] * 2 + [(150, 1700)] * 3])
def test_muon_several_matrices_of_a_shape(fmt, shapes):
    """Every matrix of a batch gets its own update: more of a shape than the tables of a launch hold, too."""
    layout, blk = muon_shapes(shapes, fmt, 61)
    old = blk.clone()
    muon_call(layout, blk, lst.lst_muon_workspace_bytes(layout.handle))
    muon_check(layout, fmt, shapes, old, blk)


@pytest.mark.parametrize("fmt", ["L12", "L16M", "L16F"])
def test_muon_fewer_matrices_at_a_time(fmt):
    """Tiled matrices in a workspace for one, for some and for all of them; the same workspace gives the same bits."""
    shapes = [(300, 404)] * 3 + [(404, 300)] * 2 + [(200, 520), (300, 403)]
    layout, blk = muon_shapes(shapes, fmt, 62)
    largest = max(lst.lst_orthogonalize_workspace_bytes(1, *s) for s in shapes)
    full = lst.lst_muon_workspace_bytes(layout.handle)
    assert full > 4 * largest
    for size in (largest, 2 * largest + 100, full // 2, full):
        new, again = blk.clone(), blk.clone()
        muon_call(layout, new, size)
        muon_check(layout, fmt, shapes, blk, new)
        muon_call(layout, again, size)
        assert torch.equal(new, again)


def test_muon_mask_and_no_adamw():
    layout = Layout(SPECS, "L16M")
    blocks, _ = muon_blocks(layout, "L16M", 31)
    before = [b.clone() for b in blocks]
    mask = [name in ("q", "odd") for name, _, _ in SPECS]
    ws = scratch(lst.lst_muon_workspace_bytes(layout.handle))
    args = (mask, ws.data_ptr(), ws.numel(), stream())
    lst.lst_muon_step(layout.handle, [b.data_ptr() for b in blocks], lst.muon_hparams(lr=0.02), None, *args)
    for b in range(layout.n_layers):
        got, old = (muon_views(layout, "L16M", b, x[b]) for x in (blocks, before))
        for name, off, n in layout.spans(b):
            same = all(torch.equal(got[f][off:off + n], old[f][off:off + n]) for f in ("MASTER", "M", "V", "W"))
            assert same == (name not in ("q", "odd")), name
    # with AdamW, the unmasked matrices take lst_adamw_step's update
    ahp = lst.adamw_hparams(step=2)
    ref = [b.clone() for b in before]
    new = [b.clone() for b in before]
    lst.lst_muon_step(layout.handle, [b.data_ptr() for b in new], lst.muon_hparams(lr=0.02), ahp, *args)
    lst.lst_adamw_step(layout.handle, [b.data_ptr() for b in ref], ahp, stream())
    for b in range(layout.n_layers):
        got, exp = (muon_views(layout, "L16M", b, x[b]) for x in (new, ref))
        for name, off, n in layout.spans(b):
            if name not in ("q", "odd"):
                assert all(torch.equal(got[f][off:off + n], exp[f][off:off + n]) for f in ("MASTER", "M", "V", "W")), name


def test_muon_small_workspace_is_bit_identical():
    layout = Layout(SPECS, "L16F")
    blocks, _ = muon_blocks(layout, "L16F", 32)
    hp = lst.muon_hparams(lr=0.02)
    results = []
    full = lst.lst_muon_workspace_bytes(layout.handle)
    largest = lst.lst_orthogonalize_workspace_bytes(1, 96, 250)
    for size in (full, largest, (full + largest) // 2):
        cur = [b.clone() for b in blocks]
        ws = scratch(size)
        lst.lst_muon_step(layout.handle, [b.data_ptr() for b in cur], hp, None, None, ws.data_ptr(), ws.numel(), stream())
        results.append(cur)
    # which steps are paired is decided for the matrices that run together, so results agree to rounding;
    # a set that runs together twice agrees to the bit
    for other in results[1:]:
        for a, b in zip(results[0], other):
            va, vb = a.view(torch.float32), b.view(torch.float32)
            assert float((va - vb).norm()) <= 2 * NS_TOL * 0.02 * float(va.norm() + 1)
    again = [b.clone() for b in blocks]
    ws = scratch(full, fill=0x3C)
    lst.lst_muon_step(layout.handle, [b.data_ptr() for b in again], hp, None, None, ws.data_ptr(), ws.numel(), stream())
    assert all(torch.equal(a, b) for a, b in zip(again, results[0]))


# ---------------------------------------------------------------------------
# streams, graphs, and all of them together
# ---------------------------------------------------------------------------
def test_operators_on_a_side_stream_and_in_a_graph():
    x, w, t = xent_inputs(300, 264, 1500, seed=40)
    m = matrix_like(gen(41), 130, 300)
    ref, ref_o = xent_call(x, w, t), ns_call([m])[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r, o = xent_call(x, w, t), ns_call([m])[0]
    side.synchronize()
    assert all(torch.equal(r[k], ref[k]) for k in ref) and torch.equal(o, ref_o)

    n, h, v = 300, 264, 1500
    loss, lse, mean = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(1, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    emb = torch.zeros(v, h, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(130, 300, dtype=torch.bfloat16, device="cuda")
    tok = torch.randint(0, v, (n,), device="cuda")
    ws = scratch(max(lst.lst_xent_workspace_bytes(n, h, v, True), lst.lst_embed_grad_workspace_bytes(n, h, v),
                     lst.lst_orthogonalize_workspace_bytes(1, 130, 300)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lst.lst_xent_grad(lst.matrix(x), lst.matrix(w), lst.indices(t), IGNORE, 1.0, loss.data_ptr(), lse.data_ptr(),
                          mean.data_ptr(), lst.matrix(dx), lst.matrix(dw), False, ws.data_ptr(), ws.numel(), stream())
        lst.lst_embed_grad(lst.matrix(dx), lst.indices(tok), lst.matrix(emb), 1.0, False, ws.data_ptr(), ws.numel(), stream())
        lst.lst_orthogonalize([lst.matrix(m)], [lst.matrix(out)], lst.ns_params(), ws.data_ptr(), ws.numel(), stream())
    for _ in range(2):
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, ref["loss"]) and torch.equal(dx, ref["dx"]) and torch.equal(dw, ref["dw"])
        assert torch.equal(out, ref_o) and torch.isfinite(emb).all()


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("pad,shift", [(3, 0), (8, 0), (1, 5), (16, 8)])
@pytest.mark.parametrize("hidden", [72, 77, 1032])
def test_results_leave_the_space_between_rows_alone(hidden, pad, shift):
    """Every result with padded rows, on and off 16 bytes: what lies before, between and behind the rows keeps its bits."""
    n, vocab = 133, 301
    x, w, t = xent_inputs(n, hidden, vocab, seed=70)
    tokens = torch.randint(0, vocab, (n,), generator=gen(71), device="cuda")
    ws = scratch(max(lst.lst_xent_workspace_bytes(n, hidden, vocab, True), lst.lst_embed_grad_workspace_bytes(n, hidden, vocab),
                     lst.lst_orthogonalize_workspace_bytes(1, n, hidden)))

    def result(rows, dtype):
        size = shift + rows * (hidden + pad) + 8
        buf = torch.full((size,), -7.0, dtype=DT[dtype], device="cuda")
        inside = torch.zeros(size, dtype=torch.bool, device="cuda")
        inside[shift:shift + rows * (hidden + pad)].view(rows, hidden + pad)[:, :hidden] = True
        return buf, buf[shift:shift + rows * (hidden + pad)].view(rows, hidden + pad)[:, :hidden], inside

    def check(made, what):
        torch.cuda.synchronize()
        for buf, view, inside in made:
            assert torch.equal(bits(buf[~inside]), bits(torch.full_like(buf[~inside], -7.0))), what
            assert torch.isfinite(view).all(), what

    for dtype in ("bf16", "f32"):
        out, grad = result(n, dtype), result(vocab, dtype)
        lst.lst_embed(lst.matrix(w), lst.indices(tokens), lst.matrix(out[1]), 1.0, stream())
        lst.lst_embed_grad(lst.matrix(x), lst.indices(tokens), lst.matrix(grad[1]), 1.0, False, ws.data_ptr(), ws.numel(), stream())
        check((out, grad), "embed " + dtype)
        lst.lst_embed_grad(lst.matrix(x), lst.indices(tokens), lst.matrix(grad[1]), 1.0, True, ws.data_ptr(), ws.numel(), stream())
        check((grad,), "embed, added " + dtype)
    dx, dw, o = result(n, "bf16"), result(vocab, "bf16"), result(n, "bf16")
    loss, lse, mean = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(1, device="cuda")
    for accumulate in (False, True):
        lst.lst_xent_grad(lst.matrix(x), lst.matrix(w), lst.indices(t), IGNORE, 1.0, loss.data_ptr(), lse.data_ptr(), mean.data_ptr(),
                          lst.matrix(dx[1]), lst.matrix(dw[1]), accumulate, ws.data_ptr(), ws.numel(), stream())
        check((dx, dw), f"xent {accumulate}")
    lst.lst_orthogonalize([lst.matrix(x)], [lst.matrix(o[1])], lst.ns_params(), ws.data_ptr(), ws.numel(), stream())
    check((o,), "orthogonalize")


@pytest.mark.parametrize("ignore", [0, 17, -1, 2 ** 40])
@pytest.mark.parametrize("n", [50, 200])
def test_xent_ignore_index_inside_the_vocabulary(n, ignore):
    """Targets equal to the index are ignored wherever it lies; -100 is then an ordinary target outside the vocabulary."""
    hidden, vocab = 64, 300
    x, w, t = xent_inputs(n, hidden, vocab, seed=72, ignored=0.0)
    t[::5] = ignore
    # the definition ignores IGNORE
    e = xent_exact(x, w, torch.where(t == ignore, IGNORE, t))
    loss, lse, mean = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(1, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    ws = scratch(lst.lst_xent_workspace_bytes(n, hidden, vocab, True))
    lst.lst_xent_grad(lst.matrix(x), lst.matrix(w), lst.indices(t), ignore, 1.0, loss.data_ptr(), lse.data_ptr(), mean.data_ptr(),
                      lst.matrix(dx), lst.matrix(dw), False, ws.data_ptr(), ws.numel(), stream())
    xent_check(dict(loss=loss, lse=lse, mean=mean, dx=dx, dw=dw), e)
    t[1] = -100
    lst.lst_xent_loss(lst.matrix(x), lst.matrix(w), lst.indices(t), ignore, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                      stream())
    assert torch.isnan(loss[1]) and int(torch.isnan(loss).sum()) == 1


def test_muon_and_embedding_in_a_graph_and_on_a_side_stream():
    shapes = [(300, 404), (300, 404), (404, 300), (24, 96), (64,)]
    layout = Layout([(f"m{i}", s, 0) for i, s in enumerate(shapes)], "L16M")
    blk = torch.zeros(layout.block_bytes(0), dtype=torch.uint8, device="cuda")
    v = muon_views(layout, "L16M", 0, blk)
    g = gen(73)
    for _, off, n in layout.spans(0):
        for f in ("MASTER", "G", "M"):
            v[f][off:off + n] = torch.randn(n, generator=g, device="cuda") * 0.01
    tokens = torch.randint(0, 50, (20000,), generator=g, device="cuda")
    table = randn(g, 50, 24, dtype="bf16")
    ws = scratch(max(lst.lst_muon_workspace_bytes(layout.handle), lst.lst_embed_grad_workspace_bytes(20000, 24, 50)))
    hp, ahp = lst.muon_hparams(lr=0.02), lst.adamw_hparams(step=3)
    out, grad = torch.zeros(20000, 24, dtype=torch.bfloat16, device="cuda"), torch.zeros(50, 24, device="cuda")

    def step(block):
        lst.lst_muon_step(layout.handle, [block.data_ptr()], hp, ahp, None, ws.data_ptr(), ws.numel(), stream())
        lst.lst_embed(lst.matrix(table), lst.indices(tokens), lst.matrix(out), 0.5, stream())
        lst.lst_embed_grad(lst.matrix(out), lst.indices(tokens), lst.matrix(grad), 0.5, False, ws.data_ptr(), ws.numel(), stream())

    ref = blk.clone()
    step(ref)
    ref_out, ref_grad = out.clone(), grad.clone()
    side, cur = torch.cuda.Stream(), blk.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_(), grad.zero_()
        step(cur)
    side.synchronize()
    assert torch.equal(cur, ref) and torch.equal(out, ref_out) and torch.equal(grad, ref_grad)
    cur = blk.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cur)
    for _ in range(2):
        cur.copy_(blk), out.zero_(), grad.zero_(), ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cur, ref) and torch.equal(out, ref_out) and torch.equal(grad, ref_grad)
    lst.lst_operator_status()


def test_example_trains():
    """The example's loss falls from about ln(1000) to near the noise floor of its data."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_next_token
    finally:
        sys.path.pop(0)
    means = train_next_token.train(60, log=None)
    # one target in ten is noise: the best possible loss is about 0.1 ln(1000) + H(0.1) = 1.0
    assert means[0] > 5.0 and min(means[-5:]) < 0.6 * means[0], means
