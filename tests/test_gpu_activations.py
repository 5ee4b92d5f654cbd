"""Residual norms, 8-bit checkpoints and their weight gradients on the GPU, against
plain implementations in 64 bits.

Checkpoints are compared bit for bit. Other tolerances are error bounds, written
out before the first run: u16 = 2^-8 and u32 = 2^-24 are the unit roundoffs of bf16
and fp32. A sum of squares over a row is added up by threads of at most 32 values
and then by trees over at most 512 threads, so a row's statistic has at most 32 + 10
roundings of nonnegative terms, and its reciprocal root half of that and two of its
own: ROW = 64 u32 covers it, with the products around it. A sum over n tokens has at
most n + 16 roundings. Products on the tensor cores are taken to be off by 2 n u32
times the sum of magnitudes (twice the textbook bound: they may truncate).
"""

from __future__ import annotations

import os
import sys
import threading

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from optimizer_update_gb300 import lst  # noqa: E402

U16, U32 = 2.0 ** -8, 2.0 ** -24
ROW = 64 * U32
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: U16, torch.float32: U32}
TOP = {"i8": 127.0, "e4m3": 448.0}
EPS = 1e-5


def stream():
    return torch.cuda.current_stream().cuda_stream


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(DT[dtype])


def strided(t, pad, shift=0, fill=float("nan")):
    """The same values with rows `pad` elements apart and `shift` elements into the storage."""
    if t is None:
        return None
    r, c = t.shape
    buf = torch.full((r * (c + pad) + shift,), fill, dtype=t.dtype, device=t.device)
    v = buf[shift:].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


def scratch(nbytes):
    return torch.full((max(1, nbytes),), 0xA5, dtype=torch.uint8, device="cuda")  # contents on entry do not matter


def mat(t):
    return None if t is None else lst.matrix(t)


def within(got, exact, bound, what):
    got, exact = got.double(), exact.double()
    assert torch.isfinite(got).all(), what
    over = (got - exact).abs() - bound
    assert float(over.max()) <= 0.0, f"{what}: {float(over.max()):.3g} over its bound"


# ---------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------
def reference_checkpoint(x, fmt):
    """(codes as values, scale bytes, values) in 64 bits: the smallest 2^k of all with max|x| <= top 2^k."""
    n, h = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -h % 32)).view(n, -1, 32)
    finite = torch.isfinite(v).all(dim=2)
    most = torch.where(finite, v.abs().amax(dim=2), torch.zeros((), dtype=torch.float64, device=x.device))
    steps = torch.tensor([2.0 ** k for k in range(-127, 128)], device=x.device, dtype=torch.float64)  # exact, as pow on a GPU need not be
    byte = torch.searchsorted(steps * TOP[fmt], most)
    scaled = torch.where(finite[..., None], v / steps[byte][..., None], torch.zeros_like(v))
    if fmt == "i8":
        q = torch.round(scaled)  # ties to even
    else:
        step = steps[torch.frexp(scaled.abs().clamp(min=2.0 ** -6))[1].long() - 4 + 127]  # 3 bits behind the leading one
        q = torch.round(scaled / step) * step
    values = torch.where(finite[..., None], q * steps[byte][..., None], torch.full_like(v, float("nan")))
    byte = torch.where(finite, byte, 255)
    return q.view(n, -1)[:, :h], byte.to(torch.uint8), values.view(n, -1)[:, :h]


def checkpoint(x, fmt):
    data, scales = lst.checkpoint_buffers(*x.shape)
    lst.lst_checkpoint_save(mat(x), lst.checkpoint(data, scales, fmt), stream())
    return data, scales, fmt


def codes(data, fmt):
    return data.contiguous().view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn).double()


def check_checkpoint(x, fmt, dst="f32", pad=0, shift=0):
    q, byte, values = reference_checkpoint(x, fmt)
    n, h = x.shape
    width = (h + 15) // 16 * 16 + 16
    data = torch.full((n + 2, width), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((n + 2, byte.shape[1] + 3), 0x5A, dtype=torch.uint8, device="cuda")
    c = (data[1:n + 1, :h], scales[1:n + 1, 1:1 + byte.shape[1]], fmt)
    lst.lst_checkpoint_save(mat(x), lst.checkpoint(*c), stream())
    assert torch.equal(codes(c[0], fmt), q) and torch.equal(c[1], byte)
    outside = torch.ones_like(data, dtype=torch.bool)
    outside[1:n + 1, :h] = False
    assert (data[outside] == 0xA5).all()
    outside = torch.ones_like(scales, dtype=torch.bool)
    outside[1:n + 1, 1:1 + byte.shape[1]] = False
    assert (scales[outside] == 0x5A).all()
    out = strided(torch.zeros(n, h, dtype=DT[dst], device="cuda"), pad, shift, 7.0)
    lst.lst_checkpoint_restore(lst.checkpoint(*c), mat(out), stream())
    assert torch.equal(torch.nan_to_num(out.double(), nan=-1e300), torch.nan_to_num(values.to(DT[dst]).double(), nan=-1e300))
    return out


@pytest.mark.parametrize("n,h,src,dst,pad,shift", [
    (1, 1, "bf16", "bf16", 0, 0), (1, 2048, "bf16", "bf16", 0, 0), (16, 2048, "f32", "f32", 0, 0), (3, 31, "bf16", "f32", 0, 0),
    (5, 33, "f32", "bf16", 1, 0), (7, 40, "bf16", "bf16", 8, 8), (513, 520, "bf16", "bf16", 0, 0), (64, 1000, "bf16", "bf16", 3, 1),
    (100, 511, "f32", "f32", 0, 3), (33, 513, "bf16", "f32", 0, 0), (4, 12293, "bf16", "bf16", 0, 0), (3001, 256, "bf16", "bf16", 0, 0),
    (2, 70000, "bf16", "bf16", 0, 0)])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_checkpoint(n, h, src, dst, pad, shift, fmt):
    g = gen(n + h)
    x = randn(g, n, h) * torch.exp(3 * randn(g, n, (h + 31) // 32).repeat_interleave(32, 1)[:, :h])
    check_checkpoint(strided(x.to(DT[src]), pad, shift), fmt, dst, pad, shift)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_checkpoint_at_the_borders(fmt):
    """Largest magnitudes around top * 2^k, ties, both zeros, subnormals, the ends of fp32's range, infinities and NaN."""
    top = torch.tensor(TOP[fmt], device="cuda")
    rows = []
    for k in (-140, -133, -127, -126, -100, -1, 0, 1, 7, 100, 119):
        m = torch.ldexp(torch.ldexp(top, torch.tensor(k // 2)), torch.tensor(k - k // 2))
        for first in (m, torch.nextafter(m, m * 2), torch.nextafter(m, m * 0), -m):
            r = torch.linspace(-1, 1, 32, device="cuda") * m
            r[0] = first
            rows.append(r)
    half = torch.arange(-16, 16, device="cuda") + 0.5  # ties between integers, and between e4m3 values
    rows += [torch.where(torch.arange(32, device="cuda") == 0, top, half), torch.where(torch.arange(32, device="cuda") == 0, top, half * 0.25),
             half * 0, half * -0.0, torch.full((32,), 2.0 ** -149, device="cuda"), torch.full((32,), 3.4028234e38, device="cuda"), half * 2.0 ** -130]
    for bad in (float("inf"), float("-inf"), float("nan")):
        r = half.clone()
        r[5] = bad
        rows.append(r)
    x = torch.stack(rows)
    check_checkpoint(x, fmt)
    check_checkpoint(x.bfloat16(), fmt)
    check_checkpoint(torch.cat([x, x[:, :5]], dim=1), fmt)  # rows off 16 bytes
    # all in one row: a bad block stays within itself
    check_checkpoint(x.reshape(1, -1), fmt)


def test_checkpoint_columns_of_a_wider_one():
    x = randn(gen(4), 50, 256, dtype="bf16")
    data, scales, fmt = checkpoint(x, "i8")
    part = lst.checkpoint(data[:, 64:168], scales[:, 2:6], fmt)
    out = torch.empty(50, 104, dtype=torch.bfloat16, device="cuda")
    lst.lst_checkpoint_restore(part, mat(out), stream())
    whole = torch.empty_like(x)
    lst.lst_checkpoint_restore(lst.checkpoint(data, scales, fmt), mat(whole), stream())
    assert torch.equal(out, whole[:, 64:168])


def test_checkpoint_past_32_bits():
    n, h = (1 << 20) + 3, 4112
    x = torch.zeros(n, h, dtype=torch.bfloat16, device="cuda")
    x[-2:] = randn(gen(2), 2, h, dtype="bf16")
    data, scales, fmt = checkpoint(x, "e4m3")
    q, byte, values = reference_checkpoint(x[-2:], fmt)
    assert torch.equal(codes(data[-2:], fmt), q) and torch.equal(scales[-2:], byte)
    x.fill_(1.0)
    lst.lst_checkpoint_restore(lst.checkpoint(data, scales, fmt), mat(x), stream())
    assert torch.equal(x[-2:], values.bfloat16()) and not x[:-2].any()


def test_checkpoint_empty():
    data, scales = lst.checkpoint_buffers(0, 64)
    x = torch.empty(0, 64, device="cuda")
    lst.lst_checkpoint_save(mat(x), lst.checkpoint(data, scales), stream())
    lst.lst_checkpoint_restore(lst.checkpoint(data, scales), mat(x), stream())


# ---------------------------------------------------------------------------
# residual norm
# ---------------------------------------------------------------------------
class Norm:
    """Inputs of a residual norm and its definition in 64 bits."""

    def __init__(self, n, h, dtype="bf16", wdtype="bf16", post=True, gate_rows=1, block=True, pre=True, alpha=1.0, beta=0.5, pad=0,
                 shift=0, seed=0):
        g = gen(seed + n + h)
        self.n, self.hidden, self.alpha, self.beta, self.pad, self.shift, self.t = n, h, alpha, beta, pad, shift, DT[dtype]
        self.x = strided(randn(g, n, h, dtype=dtype), pad, shift)
        self.y = strided(randn(g, n, h, dtype=dtype, std=0.7), pad, shift) if block else None
        self.w_post = (1 + randn(g, 1, h, std=0.2)).to(DT[wdtype]) if post else None
        self.w_pre = (1 + randn(g, 1, h, std=0.2)).to(DT[wdtype]) if pre else None
        self.gate = (randn(g, gate_rows, h)).to(DT[wdtype]) if gate_rows else None
        self.dh, self.dz = (strided(randn(g, n, h, dtype=dtype), pad, shift) for _ in range(2))
        self.params = lst.residual_params(alpha, beta, EPS)

    def new(self):
        return strided(torch.zeros(self.n, self.hidden, dtype=self.t, device="cuda"), self.pad, self.shift, 7.0)

    def per_token(self, v):
        return 1.0 if v is None else v.double().repeat_interleave(self.n // v.shape[0], dim=0)

    def forward(self, h8=None, y8=None):
        h, z = self.new(), self.new() if self.w_pre is not None else None
        lst.lst_residual_norm(mat(self.x), mat(self.y), mat(self.gate), mat(self.w_post), mat(self.w_pre), self.params, mat(h), mat(z),
                              h8 and lst.checkpoint(*h8), y8 and lst.checkpoint(*y8), stream())
        return h, z

    def check_forward(self, h, z):
        wide = self.alpha * self.x.double()
        size = wide.abs()
        if self.y is not None:
            u = self.y.double()
            if self.w_post is not None:
                u = u / (u.square().mean(1, keepdim=True) + EPS).sqrt() * self.w_post.double()
            u = self.beta * self.per_token(self.gate) * u
            wide, size = wide + u, size + u.abs()
        within(h, wide, U[self.t] * wide.abs() + 2 * ROW * size, "h")
        if self.w_pre is not None:
            rho = (wide.square().mean(1, keepdim=True) + EPS).rsqrt()
            exact = wide * rho * self.w_pre.double()
            # an error of h changes rho by at most its share of the row's norm
            share = 2 * ROW * size.norm(dim=1, keepdim=True) / wide.norm(dim=1, keepdim=True).clamp(min=1e-30)
            within(z, exact, (U[self.t] + 2 * ROW + share) * exact.abs() + 2 * ROW * size * rho * self.w_pre.double().abs(), "z")

    def backward(self, h, y, dh=True, dz=True, wdtype=None, accumulate=False, grads=None, pad=None):
        """h, y: matrices or checkpoints (data, scales, format). Returns dx, dy, dgate, dw_post, dw_pre."""
        def operand(v):
            return v if v is None else lst.checkpoint(*v) if isinstance(v, tuple) else mat(v)

        dx, dy = self.new(), self.new()
        if grads is None:
            grads = [None if v is None else torch.full(v.shape, float("nan"), dtype=DT[wdtype] if wdtype else v.dtype, device="cuda")
                     for v in (self.gate, self.w_post, self.w_pre if dz else None)]
        ws = scratch(lst.lst_residual_norm_grad_workspace_bytes(self.n, self.hidden, 0 if self.gate is None else self.gate.shape[0]))
        lst.lst_residual_norm_grad(mat(self.dh) if dh else None, mat(self.dz) if dz else None, operand(h), operand(y), mat(self.gate),
                                   mat(self.w_post), mat(self.w_pre) if dz else None, self.params, mat(dx), mat(dy), mat(grads[0]),
                                   mat(grads[1]), mat(grads[2]), accumulate, ws.data_ptr(), ws.numel(), stream())
        return dx, dy, *grads

    def check_backward(self, h, y, got, dh=True, dz=True, before=None):
        """h, y: the values in 64 bits. Bounds: each product and sum of the formulas in magnitudes, times the roundings."""
        dx, dy, dgate, dw_post, dw_pre = got
        zero = torch.zeros(self.n, self.hidden, dtype=torch.float64, device="cuda")
        d = self.dh.double() if dh else zero
        size = d.abs()
        sums = []  # (name, result, exact, magnitude)
        if dz:
            rho = (h.square().mean(1, keepdim=True) + EPS).rsqrt()
            m = self.dz.double() * self.w_pre.double()
            d = d + rho * (m - h * rho.square() * (m * h).mean(1, keepdim=True))
            size = size + rho * (m.abs() + h.abs() * rho.square() * (m * h).abs().mean(1, keepdim=True))
            t = self.dz.double() * h * rho
            sums.append(("dw_pre", dw_pre, t.sum(0, keepdim=True), t.abs().sum(0, keepdim=True)))
        within(dx, self.alpha * d, U[self.t] * (self.alpha * d).abs() + 2 * ROW * abs(self.alpha) * size, "dx")
        gate, w = self.per_token(self.gate), 1.0 if self.w_post is None else self.w_post.double()
        e, esize = self.beta * d * gate * w, abs(self.beta) * size * (gate if isinstance(gate, float) else gate.abs()) * (w if isinstance(w, float) else w.abs())
        tau = 1.0
        if self.w_post is not None:
            tau = (y.square().mean(1, keepdim=True) + EPS).rsqrt()
            exact = tau * (e - y * tau.square() * (e * y).mean(1, keepdim=True))
            esize = tau * (esize + y.abs() * tau.square() * (esize * y.abs()).mean(1, keepdim=True))
            t = self.beta * d * gate * y * tau
            b = (self.beta * gate * size * y * tau).abs()
            sums.append(("dw_post", dw_post, t.sum(0, keepdim=True), b.sum(0, keepdim=True)))
        else:
            exact = e
        within(dy, exact, U[self.t] * exact.abs() + 4 * ROW * esize, "dy")
        if dgate is not None:
            r = self.gate.shape[0]
            t, b = self.beta * d * y * tau * w, (self.beta * size * y * tau * w).abs()
            sums.append(("dgate", dgate, t.view(r, self.n // r, -1).sum(1), b.view(r, self.n // r, -1).sum(1)))
        for name, result, exact, magnitude in sums:
            if result is None:
                continue
            if before is not None:
                exact = exact + before[name].double()
            within(result, exact, U[result.dtype] * exact.abs() + (4 * ROW + 2 * (self.n + 16) * U32) * magnitude + U32 * exact.abs(), name)


SHAPES = [(1, 1), (1, 2048), (8, 2048), (3, 32), (37, 31), (5, 33), (700, 96), (64, 1000), (300, 2056), (41, 4096), (23, 4095), (9, 8192),
          (5, 12288), (3, 16384), (2, 16383), (3, 9001)]


@pytest.mark.parametrize("n,h", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm(n, h, dtype):
    p = Norm(n, h, dtype)
    p.check_forward(*p.forward())


@pytest.mark.parametrize("kw", [
    dict(post=False), dict(gate_rows=0), dict(post=False, gate_rows=0), dict(pre=False), dict(block=False, post=False, gate_rows=0),
    dict(wdtype="f32"), dict(gate_rows=2), dict(gate_rows=60), dict(gate_rows=15, wdtype="f32"), dict(alpha=0.0), dict(beta=-2.0, alpha=0.3),
    dict(pad=3), dict(pad=8, shift=8), dict(shift=1), dict(pad=16, dtype="f32"), dict(pad=1, dtype="f32", wdtype="f32")])
@pytest.mark.parametrize("h", [520, 777])
def test_norm_forms(kw, h):
    p = Norm(60, h, **kw)
    p.check_forward(*p.forward())


@pytest.mark.parametrize("n,h,dtype,pad", [(5, 2048, "bf16", 0), (33, 40, "bf16", 0), (17, 777, "bf16", 0), (9, 4100, "f32", 3), (6, 8200, "bf16", 8)])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_norm_writes_the_checkpoints(n, h, dtype, pad, fmt):
    p = Norm(n, h, dtype, pad=pad)
    h8, y8 = ((*lst.checkpoint_buffers(n, h), fmt) for _ in range(2))
    hh, z = p.forward(h8, y8)
    p.check_forward(hh, z)
    for c, source in ((h8, hh), (y8, p.y)):
        data, scales, _ = checkpoint(source, fmt)
        assert torch.equal(c[0], data) and torch.equal(c[1], scales)
    # h8 alone, without h
    again = (*lst.checkpoint_buffers(n, h), fmt)
    lst.lst_residual_norm(mat(p.x), mat(p.y), mat(p.gate), mat(p.w_post), None, p.params, None, None, lst.checkpoint(*again), None, stream())
    assert torch.equal(again[0], h8[0]) and torch.equal(again[1], h8[1])


@pytest.mark.parametrize("n,h,dtype,kw", [
    (30000, 33, "bf16", {}), (15000, 777, "bf16", dict(pad=3, shift=1)), (7300, 2047, "f32", {}), (4000, 4095, "bf16", dict(gate_rows=4000)),
    (20000, 264, "bf16", dict(pad=1)), (15000, 770, "f32", dict(gate_rows=5))])
def test_norm_odd_rows_over_many_turns(n, h, dtype, kw):
    """Rows off 16 bytes, eight or more turns of every CTA: its stages are filled again several times, the first rows' and
    the last ones' byte by byte, those between by whole pieces."""
    p = Norm(n, h, dtype, **kw)
    hh, z = p.forward()
    p.check_forward(hh, z)
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y))
    h8, y8 = ((*lst.checkpoint_buffers(n, h), f) for f in ("i8", "e4m3"))
    again, z_again = p.forward(h8, y8)
    assert torch.equal(again, hh) and torch.equal(z_again, z)
    for c, source in ((h8, hh), (y8, p.y)):
        assert all(torch.equal(a, b) for a, b in zip(c[:2], checkpoint(source, c[2])[:2]))


def test_norm_in_place():
    p = Norm(50, 300)
    h, z = p.forward()
    x, y = p.x.clone(), p.y.clone()
    lst.lst_residual_norm(mat(x), mat(y), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(x), mat(y), None, None, stream())
    assert torch.equal(x, h) and torch.equal(y, z)


def test_norm_rows_of_zeros_and_non_finite_ones():
    p = Norm(12, 264, post=True)
    p.x[3], p.y[3] = 0.0, 0.0
    p.x[5, 7], p.y[6, 9], p.y[7, 0] = float("inf"), float("nan"), float("inf")
    h, z = p.forward()
    assert not h[3].any() and not z[3].any()
    fine = [0, 1, 2, 4, 8, 9, 10, 11]
    bad = [5, 6, 7]
    for r in bad:
        assert not torch.isfinite(z[r]).all()
    clean = Norm(12, 264, post=True)
    ch, cz = clean.forward()
    assert torch.equal(h[fine], ch[fine]) and torch.equal(z[fine], cz[fine])
    # backward: the other rows as they are without the bad ones, zero rows finite
    dx, dy, *_ = p.backward(h, p.y)
    cdx, cdy, *_ = clean.backward(ch, clean.y)
    assert torch.equal(dx[fine], cdx[fine]) and torch.equal(dy[fine], cdy[fine])
    assert torch.isfinite(dx[3]).all() and torch.isfinite(dy[3]).all()


@pytest.mark.parametrize("h,dtype,gate_rows", [(4096, "bf16", 0), (4096, "f32", 1), (4096, "bf16", 16), (777, "bf16", 1), (16384, "bf16", 0), (12289, "f32", 1)])
def test_norm_rows_beyond_fp32_squares(h, dtype, gate_rows):
    """Rows of sizes 2^0 to 2^62, h and y pointing the same way, so that their product's sum overflows, too. Where a sum of
    squares is 2^128 or more its norm and that norm's gradient are zero; the other rows are as ever."""
    sizes = [(i, j) for i in (0, 40, 56, 62) for j in (0, 40, 56, 62)]
    n = len(sizes)
    p = Norm(n, h, dtype, gate_rows=gate_rows, beta=0.5)
    if gate_rows:
        p.gate.copy_(1 + 0.1 * p.gate.clamp(-4, 4))
    scale = torch.tensor([[2.0 ** i, 2.0 ** j] for i, j in sizes], device="cuda")
    p.y.copy_(p.x * scale[:, 1:])
    p.x.mul_(scale[:, :1])

    def inverse_rms(v):
        squares = v.square().sum(1, keepdim=True)
        assert not ((squares > 2.0 ** 127) & (squares < 2.0 ** 129)).any()
        return torch.where(squares < 2.0 ** 128, (squares / h + EPS).rsqrt(), 0.0)

    x, y, w_post, w_pre, dz, gate = p.x.double(), p.y.double(), p.w_post.double(), p.w_pre.double(), p.dz.double(), p.per_token(p.gate)
    hh, z = p.forward()
    u = 0.5 * gate * y * inverse_rms(y) * w_post
    wide, size = x + u, x.abs() + u.abs()
    within(hh, wide, U[p.t] * wide.abs() + 2 * ROW * size, "h")
    rho = inverse_rms(wide)
    share = 2 * ROW * size.norm(dim=1, keepdim=True) / wide.norm(dim=1, keepdim=True)
    within(z, wide * rho * w_pre, ((U[p.t] + 2 * ROW + share) * wide.abs() + 2 * ROW * size) * rho * w_pre.abs(), "z")
    # from x and y as they are
    dx, dy, dgate, dw_post, dw_pre = p.backward(p.x, p.y)
    rho, tau, m = inverse_rms(x), inverse_rms(y), dz * w_pre
    d = p.dh.double() + rho * (m - x * rho * (m * x * rho).mean(1, keepdim=True))
    size = p.dh.double().abs() + rho * (m.abs() + x.abs() * rho * (m * x * rho).abs().mean(1, keepdim=True))
    within(dx, d, U[p.t] * d.abs() + 2 * ROW * size, "dx")
    e, esize = 0.5 * d * gate * w_post, 0.5 * size * (gate * w_post).abs()
    exact = tau * (e - y * tau * (e * y * tau).mean(1, keepdim=True))
    esize = tau * (esize + y.abs() * tau * (esize * y.abs() * tau).mean(1, keepdim=True))
    within(dy, exact, U[p.t] * exact.abs() + 4 * ROW * esize, "dy")
    for name, g, t, most in (("dw_post", dw_post, 0.5 * d * gate * y * tau, 0.5 * size * gate * (y * tau).abs()), ("dw_pre", dw_pre, dz * x * rho, (dz * x * rho).abs())):
        exact = t.sum(0, keepdim=True)
        within(g, exact, (U[g.dtype] + U32) * exact.abs() + (4 * ROW + 2 * (n + 16) * U32) * most.sum(0, keepdim=True), name)
    assert dgate is None or torch.isfinite(dgate).all()


@pytest.mark.parametrize("n,h", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_grad(n, h, dtype):
    p = Norm(n, h, dtype, wdtype=dtype)
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y))


@pytest.mark.parametrize("kw", [
    dict(post=False), dict(gate_rows=0), dict(post=False, gate_rows=0), dict(wdtype="f32"), dict(gate_rows=2), dict(gate_rows=60),
    dict(gate_rows=60, post=False), dict(gate_rows=30), dict(gate_rows=15, wdtype="f32"), dict(alpha=0.0), dict(beta=-2.0, alpha=0.3), dict(pad=3),
    dict(pad=8, shift=8), dict(shift=1), dict(pad=16, dtype="f32"), dict(pad=1, dtype="f32", wdtype="f32")])
@pytest.mark.parametrize("h", [520, 777])
def test_norm_grad_forms(kw, h):
    p = Norm(60, h, **kw)
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y))


@pytest.mark.parametrize("n,h,rows", [(5000, 64, 2), (5000, 64, 5), (5000, 40, 1250), (5000, 64, 2500), (5000, 33, 5000), (2433, 520, 3), (6000, 1032, 4),
                                      (4999, 264, 1), (20000, 72, 20), (1500, 2056, 500)])
def test_norm_grad_gates_over_many_ctas(n, h, rows):
    p = Norm(n, h, wdtype="f32", gate_rows=rows)
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y))


@pytest.mark.parametrize("n,h,dtype,pad", [(33, 2048, "bf16", 0), (29, 40, "bf16", 0), (40, 777, "bf16", 0), (9, 4100, "f32", 3), (700, 256, "bf16", 8),
                                           (6, 8200, "bf16", 0), (3, 16384, "bf16", 0), (5, 12288, "f32", 0), (11, 6001, "f32", 0), (3, 16383, "f32", 0)])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_norm_grad_from_checkpoints(n, h, dtype, pad, fmt):
    p = Norm(n, h, dtype, pad=pad)
    h8, y8 = checkpoint(p.x, fmt), checkpoint(p.y, "i8" if fmt == "e4m3" else "e4m3")
    hv, yv = (reference_checkpoint(v, f)[2] for v, f in ((p.x, h8[2]), (p.y, y8[2])))
    p.check_backward(hv, yv, p.backward(h8, y8))
    p.check_backward(hv, p.y.double(), p.backward(h8, p.y))
    p.check_backward(p.x.double(), yv, p.backward(p.x, y8))


@pytest.mark.parametrize("n,h,dtype,kw", [
    (1, 2056, "bf16", {}), (2, 96, "bf16", {}), (17, 8168, "bf16", {}), (40, 8160, "f32", {}), (1300, 4104, "bf16", dict(gate_rows=0)),
    (5000, 264, "bf16", dict(gate_rows=4)), (2000, 32, "f32", dict(gate_rows=1000)), (901, 1032, "bf16", dict(post=False)), (64, 8, "bf16", {})])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_norm_grad_from_two_checkpoints_of_any_scale_rows(n, h, dtype, kw, fmt):
    """h and y kept alike, with rows of scales off 16 bytes, and their starts, too."""
    p = Norm(n, h, dtype, **kw)
    kept = []
    for x, at in ((p.x, 0), (p.y, 5)):
        data, scales, _ = checkpoint(x, fmt)
        blocks = torch.full((n, scales.shape[1] + at), 255, dtype=torch.uint8, device="cuda")
        blocks[:, at:] = scales
        kept.append((data, blocks[:, at:], fmt))
    p.check_backward(*(reference_checkpoint(x, fmt)[2] for x in (p.x, p.y)), p.backward(*kept))


@pytest.mark.parametrize("n,h,dtype", [(301, 264, "bf16"), (90, 4104, "bf16"), (33, 8192, "f32")])
@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("kw,dh", [(dict(post=False), True), (dict(post=False), False), (dict(), False), (dict(gate_rows=0, post=False), False),
                                   (dict(gate_rows=3, post=False), True)])
def test_norm_grad_forms_of_whole_units(n, h, dtype, fmt, kw, dh):
    """Rows on 16 bytes without dh, or with a gate's gradient but no norm behind the block; y's infinities stay out of dy there."""
    p = Norm(n // 3 * 3, h, dtype, **kw)
    h_in, y_in = (v if fmt is None else checkpoint(v, fmt) for v in (p.x, p.y))
    hv, yv = (v.double() if fmt is None else reference_checkpoint(v, fmt)[2] for v in (p.x, p.y))
    got = p.backward(h_in, y_in, dh=dh)
    p.check_backward(hv, yv, got, dh=dh)
    if p.w_post is None:
        p.y[1, 5] = float("inf")
        dx, dy, *_ = p.backward(h_in, y_in if fmt is None else checkpoint(p.y, fmt), dh=dh)
        assert torch.equal(dx, got[0]) and torch.equal(dy, got[1])


@pytest.mark.parametrize("n,h", [(40, 12), (7, 4100), (9, 8188), (5, 8196)])
def test_norm_grad_rows_on_16_bytes_of_half_units(n, h):
    p = Norm(n, h, "f32")
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y))


@pytest.mark.parametrize("h", [264, 4104, 9000])
@pytest.mark.parametrize("fmt", [None, "i8"])
def test_norm_grad_results_off_16_bytes(h, fmt):
    """The inputs on 16 bytes, dx and dy not."""
    p = Norm(40, h)
    p.pad, p.shift = 3, 1  # of what new() gives
    h_in, y_in = (v if fmt is None else checkpoint(v, fmt) for v in (p.x, p.y))
    hv, yv = (v.double() if fmt is None else reference_checkpoint(v, fmt)[2] for v in (p.x, p.y))
    p.check_backward(hv, yv, p.backward(h_in, y_in))


@pytest.mark.parametrize("n,h,dtype,kw,dh", [
    (700, 8200, "bf16", {}, True), (700, 8193, "bf16", dict(gate_rows=4), True), (160, 12288, "bf16", dict(gate_rows=160), True),
    (160, 12289, "f32", dict(gate_rows=80, post=False), False), (161, 9000, "f32", dict(gate_rows=0, post=False), True),
    (33, 16376, "bf16", dict(gate_rows=11), False), (1, 16384, "f32", {}, True), (1, 8201, "bf16", {}, False)])
@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
def test_norm_grad_wide_rows(n, h, dtype, kw, dh, fmt):
    p = Norm(n, h, dtype, **kw)
    h_in, y_in = (v if fmt is None else checkpoint(v, fmt) for v in (p.x, p.y))
    hv, yv = (v.double() if fmt is None else reference_checkpoint(v, fmt)[2] for v in (p.x, p.y))
    got = p.backward(h_in, y_in, dh=dh)
    p.check_backward(hv, yv, got, dh=dh)
    again = p.backward(h_in, y_in, dh=dh)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    p.check_backward(None, yv, p.backward(None, y_in, dz=False), dz=False)


@pytest.mark.parametrize("n,h", [(60, 40), (60, 2056), (700, 8), (900, 1), (40, 3), (333, 17), (50, 1032)])
def test_norm_grad_of_ragged_rows_beside_other_bytes(n, h):
    """Rows of checkpoints that end inside 16 bytes, with e4m3 NaN behind them; rows of a byte or a few."""
    p = Norm(n, h, post=True)
    kept = []
    for x in (p.x, p.y):
        data, scales, fmt = checkpoint(x, "e4m3")
        wide = torch.full((n, (h + 15) // 16 * 16 + 16), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, :h] = data
        blocks = torch.full((n, scales.shape[1] + 3), 255, dtype=torch.uint8, device="cuda")
        blocks[:, 1:1 + scales.shape[1]] = scales
        kept.append((wide[:, :h], blocks[:, 1:1 + scales.shape[1]], fmt))
    p.check_backward(*(reference_checkpoint(x, "e4m3")[2] for x in (p.x, p.y)), p.backward(*kept))
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y))


@pytest.mark.parametrize("h", [264, 333])
def test_norm_grad_parts(h):
    """Either gradient alone, and outputs left out."""
    p = Norm(200, h)
    p.check_backward(p.x.double(), p.y.double(), p.backward(p.x, p.y, dh=False), dh=False)
    p.check_backward(None, p.y.double(), p.backward(None, p.y, dz=False), dz=False)
    full = p.backward(p.x, p.y)
    ws = scratch(lst.lst_residual_norm_grad_workspace_bytes(200, h, 1))

    def only(which, y=True):
        out = [torch.full_like(v, 3.0) if i == which else None for i, v in enumerate(full)]
        lst.lst_residual_norm_grad(mat(p.dh), mat(p.dz), mat(p.x), mat(p.y) if y else None, mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params,
                                   *map(mat, out), False, ws.data_ptr(), ws.numel(), stream())
        return out[which]

    for i, v in enumerate(full):
        assert torch.equal(only(i), v), i
    # without a norm behind the block, dy needs no y
    p = Norm(200, h, post=False, gate_rows=0)
    dx, dy, *_ = p.backward(p.x, None)
    assert torch.equal(dx, p.backward(p.x, p.y)[0]) and torch.equal(dy, p.backward(p.x, p.y)[1])


@pytest.mark.parametrize("rows,n", [(1, 300), (300, 300), (3, 300), (150, 300), (2, 4000)])
@pytest.mark.parametrize("wdtype", ["bf16", "f32"])
def test_norm_grad_accumulates(rows, n, wdtype):
    p = Norm(n, 136, gate_rows=rows, wdtype=wdtype)
    g = gen(9)
    before = dict(dgate=randn(g, rows, 136, dtype=wdtype, std=10.0), dw_post=randn(g, 1, 136, dtype=wdtype, std=10.0),
                  dw_pre=randn(g, 1, 136, dtype=wdtype, std=10.0))
    got = p.backward(p.x, p.y, accumulate=True, grads=[before[k].clone() for k in ("dgate", "dw_post", "dw_pre")])
    p.check_backward(p.x.double(), p.y.double(), got, before=before)


@pytest.mark.parametrize("n,h,rows", [
    (300, 2056, 1), (300, 2056, 3), (300, 2056, 300), (900, 2056, 450), (900, 4104, 1), (900, 4104, 300), (300, 4101, 3), (300, 8201, 1), (300, 8201, 3),
    (300, 8201, 300), (600, 8201, 300), (300, 12288, 1), (300, 12288, 3), (300, 12288, 300), (600, 12288, 300), (90, 16384, 45)])
@pytest.mark.parametrize("wdtype,fmt,shift", [("bf16", None, 0), ("f32", "i8", 0), ("bf16", "e4m3", 1)])
def test_norm_grad_accumulates_in_every_form(n, h, rows, wdtype, fmt, shift):
    """One row a CTA at a time and rows in two launches; gate rows of one CTA, of several, of every token; results on 16
    bytes and off them."""
    p = Norm(n, h, gate_rows=rows, wdtype=wdtype)
    g = gen(9)
    before = {k: strided(randn(g, r, h, dtype=wdtype, std=10.0), 0, shift) for k, r in (("dgate", rows), ("dw_post", 1), ("dw_pre", 1))}
    h_in, y_in = (v if fmt is None else checkpoint(v, fmt) for v in (p.x, p.y))
    hv, yv = (v.double() if fmt is None else reference_checkpoint(v, fmt)[2] for v in (p.x, p.y))
    grads = [strided(before[k], 0, shift) for k in ("dgate", "dw_post", "dw_pre")]
    got = p.backward(h_in, y_in, accumulate=True, grads=grads)
    p.check_backward(hv, yv, got, before=before)


@pytest.mark.parametrize("n,h,dtype,kw", [
    (7000, 2056, "bf16", {}), (7000, 2048, "f32", dict(gate_rows=7)), (4000, 4096, "bf16", {}), (3000, 8192, "bf16", dict(gate_rows=0)),
    (1600, 12288, "bf16", {}), (1600, 12288, "f32", dict(gate_rows=1600)), (1300, 16384, "bf16", dict(post=False)), (30000, 64, "bf16", dict(gate_rows=15)),
    (20000, 264, "f32", dict(block=False, post=False, gate_rows=0)), (1500, 9001, "bf16", {})])
def test_norm_over_many_turns(n, h, dtype, kw):
    """Every CTA fills its stages again several times, and no two rows are alike; all results, with the checkpoints."""
    p = Norm(n, h, dtype, **kw)
    h8 = (*lst.checkpoint_buffers(n, h), "i8")
    y8 = (*lst.checkpoint_buffers(n, h), "e4m3") if p.y is not None else None
    hh, z = p.forward(h8, y8)
    p.check_forward(hh, z)
    for c, source in ((h8, hh), (y8, p.y)):
        assert c is None or all(torch.equal(a, b) for a, b in zip(c[:2], checkpoint(source, c[2])[:2]))


@pytest.mark.parametrize("n,h,kw", [(9000, 264, {}), (5000, 1032, dict(gate_rows=5)), (3000, 4096, {}), (1500, 8192, dict(gate_rows=3)), (1500, 8200, {}), (9000, 33, {})])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_norm_grad_of_a_matrix_and_a_checkpoint_over_many_turns(n, h, kw, fmt):
    p = Norm(n, h, **kw)
    h8, y8 = checkpoint(p.x, fmt), checkpoint(p.y, fmt)
    p.check_backward(reference_checkpoint(p.x, fmt)[2], p.y.double(), p.backward(h8, p.y))
    p.check_backward(p.x.double(), reference_checkpoint(p.y, fmt)[2], p.backward(p.x, y8))


def test_norm_grad_in_place_and_again():
    p = Norm(900, 520)
    first = p.backward(p.x, p.y)
    second = p.backward(p.x, p.y)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    dh, dz = p.dh.clone(), p.dz.clone()
    ws = scratch(lst.lst_residual_norm_grad_workspace_bytes(900, 520, 1))
    lst.lst_residual_norm_grad(mat(dh), mat(dz), mat(p.x), mat(p.y), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(dh), mat(dz), None, None,
                               None, False, ws.data_ptr(), ws.numel(), stream())
    assert torch.equal(dh, first[0]) and torch.equal(dz, first[1])


def test_norm_grad_of_no_tokens():
    p = Norm(4, 64)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    for accumulate in (False, True):
        g = [torch.ones_like(v) for v in (p.gate, p.w_post, p.w_pre)]
        lst.lst_residual_norm_grad(mat(empty), mat(empty), mat(empty), mat(empty), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(empty),
                                   mat(empty), *map(mat, g), accumulate, 0, 0, stream())
        assert all((v == float(accumulate)).all() for v in g)
    lst.lst_residual_norm(mat(empty), mat(empty), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(empty), mat(empty), None, None, stream())


def test_norm_grad_against_differences():
    """Central differences of the forward call's own results. Step e = 2^-6 on values of size 1: the loss's third
    derivative leaves e^2, about 2e-4, of its size, and fp32 roundings 2^-24 sqrt(H) / e, under 1e-4; bound 2e-3."""
    n, h, e = 6, 48, 2.0 ** -6
    p = Norm(n, h, "f32", "f32", gate_rows=2, alpha=0.8, beta=0.6)
    got = dict(zip(("x", "y", "gate", "w_post", "w_pre"), _grads_at_forward(p)))

    def loss():
        hh, z = p.forward()
        return float((hh.double() * p.dh.double()).sum() + (z.double() * p.dz.double()).sum())

    g = gen(77)
    for name in got:
        v = getattr(p, name)
        direction = torch.randn(v.shape, generator=g, device="cuda")
        keep = v.clone()
        v.copy_(keep + e * direction)
        up = loss()
        v.copy_(keep - e * direction)
        down = loss()
        v.copy_(keep)
        slope, expected = (up - down) / (2 * e), float((got[name].double() * direction.double()).sum())
        size = float(got[name].double().norm() * direction.double().norm())
        assert abs(slope - expected) <= 2e-3 * size, name


def _grads_at_forward(p):
    h, _ = p.forward()
    return p.backward(h, p.y)


def test_norm_past_32_bits():
    n, h = (1 << 19) + 5, 4104
    x = torch.zeros(n, h, dtype=torch.bfloat16, device="cuda")
    x[-2:] = randn(gen(8), 2, h, dtype="bf16")
    w = torch.ones(1, h, device="cuda")
    lst.lst_residual_norm(mat(x), None, None, None, mat(w), lst.residual_params(2.0, 1.0, EPS), None, mat(x), None, None, stream())
    src = randn(gen(8), 2, h, dtype="bf16").double() * 2
    exact = src * (src.square().mean(1, keepdim=True) + EPS).rsqrt()
    within(x[-2:], exact, (U16 + 4 * ROW) * exact.abs(), "z")
    assert not x[:-2].any()


# ---------------------------------------------------------------------------
# weight gradient from a checkpoint
# ---------------------------------------------------------------------------
def wgrad(dy, c, weight, dw, accumulate, ws=None):
    if ws is None:
        ws = scratch(lst.lst_checkpoint_wgrad_workspace_bytes(mat(dy), lst.checkpoint(*c), mat(dw)))
    lst.lst_checkpoint_wgrad(mat(dy), lst.checkpoint(*c), mat(weight), EPS, mat(dw), accumulate, ws.data_ptr(), ws.numel(), stream())
    return dw


def check_wgrad(n, o, h, fmt="i8", norm=None, out="bf16", accumulate=False, pad=0, shift=0, dw_pad=0, dw_shift=0, c_pad=0):
    g = gen(n + o + h)
    dy = strided(randn(g, n, o, dtype="bf16"), pad, shift)
    x = randn(g, n, h, dtype="bf16") * torch.exp(randn(g, n, 1)).bfloat16()
    data, scales, _ = checkpoint(x, fmt)
    if c_pad:  # rows of a wider checkpoint: other bytes behind the last column (an e4m3 NaN)
        wide = torch.full((n, (h + 15) // 16 * 16 + 16 * c_pad), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, :h] = data
        data = wide[:, :h]
    else:
        full = data.as_strided((n, data.stride(0)), (data.stride(0), 1)) if n > 1 else None
        if full is not None:
            full[:, h:] = 0x7F
    weight = (1 + randn(g, 1, h, std=0.3)).to(DT[norm]) if norm else None
    before = randn(g, o, h, dtype=out, std=3.0)
    dw = wgrad(dy, (data, scales, fmt), weight, strided(before, dw_pad, dw_shift), accumulate)
    v = reference_checkpoint(x, fmt)[2]
    per_column = 1.0
    if norm:
        v = v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()
        per_column = weight.double()
    exact, size = (dy.double().T @ v) * per_column, (dy.double().abs().T @ v.abs()) * (per_column if isinstance(per_column, float) else per_column.abs())
    if accumulate:
        exact = exact + before.double()
    bound = (2 * (n + 64) * U32 + ((U16 + ROW) if norm else 0.0)) * size + (U[DT[out]] + 2 * U32) * exact.abs()
    within(dw, exact, bound, "dw")
    return dw


@pytest.mark.parametrize("n,o,h", [(1, 1, 1), (1, 256, 2048), (16, 8, 32), (63, 16, 40), (64, 128, 128), (65, 129, 127), (200, 256, 256), (130, 300, 520),
                                   (1000, 256, 2048), (4096, 256, 512), (2500, 1000, 96), (129, 2000, 777), (8192, 24, 33), (70, 5632, 2048),
                                   (5, 31, 12293), (300, 4999, 2047)])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_wgrad(n, o, h, fmt):
    check_wgrad(n, o, h, fmt)


@pytest.mark.parametrize("kw", [dict(norm="bf16"), dict(norm="f32"), dict(out="f32"), dict(out="f32", norm="f32"), dict(accumulate=True),
                                dict(out="f32", accumulate=True, norm="bf16"), dict(pad=3), dict(pad=8, shift=8), dict(shift=1), dict(dw_pad=3), dict(dw_shift=1),
                                dict(dw_pad=2, out="f32"), dict(dw_pad=8, accumulate=True), dict(c_pad=1, fmt="e4m3"), dict(dw_shift=1, accumulate=True)])
@pytest.mark.parametrize("n,o,h", [(100, 200, 264), (300, 333, 301), (3000, 40, 72)])
def test_wgrad_forms(kw, n, o, h):
    check_wgrad(n, o, h, **kw)


@pytest.mark.parametrize("n,o,h,dw_pad", [(300, 333, 301, 3), (900, 520, 301, 3), (300, 5000, 2047, 1), (2500, 300, 77, 3), (300, 333, 300, 4)])
@pytest.mark.parametrize("kw", [dict(), dict(out="f32"), dict(norm="bf16"), dict(norm="f32", out="f32")])
def test_wgrad_accumulates_where_rows_on_16_bytes_end_inside_them(n, o, h, dw_pad, kw):
    check_wgrad(n, o, h, accumulate=True, dw_pad=dw_pad, **kw)
    check_wgrad(n, o, h, accumulate=False, dw_pad=dw_pad, **kw)


@pytest.mark.parametrize("n,o,h", [(1, 40, 300), (3, 256, 2048), (512, 300, 264), (513, 300, 264), (511, 64, 17000)])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_wgrad_normed(n, o, h, fmt):
    check_wgrad(n, o, h, fmt, norm="f32")
    check_wgrad(n, o, h, fmt, norm="bf16", out="f32", pad=3)


def test_wgrad_normed_of_few_tokens_is_near():
    """Two bf16 parts of a value leave 2^-16 of it (half a step of the rest): with it the statistic's error and the sums'."""
    n, o, h = 5, 64, 520
    g = gen(3)
    dy, x = randn(g, n, o, dtype="bf16"), randn(g, n, h, dtype="bf16")
    weight = 1 + randn(g, 1, h, std=0.3)
    c = checkpoint(x, "i8")
    dw = wgrad(dy, c, weight, torch.empty(o, h, device="cuda"), False)
    v = reference_checkpoint(x, "i8")[2]
    v = v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()
    size = (dy.double().abs().T @ v.abs()) * weight.double().abs()
    within(dw, (dy.double().T @ v) * weight.double(), (2.0 ** -16 + ROW + 2 * (2 * n + 64) * U32) * size, "dw")


@pytest.mark.parametrize("n", [64, 513, 1000, 3001])
@pytest.mark.parametrize("out,accumulate", [("bf16", False), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("terms", [1, None])
def test_wgrad_normed_is_near_for_any_count(n, out, accumulate, terms):
    """What the parts leave of a value (two 2^-15 at most, three nothing), the statistic's error and the sums' over all
    parts; then the result's own rounding. With one token per output the sums are three terms and zeros, so that what is
    left of a value shows."""
    o, h = 300, 264
    g = gen(n)
    dy, x = randn(g, n, o, dtype="bf16"), randn(g, n, h, dtype="bf16")
    if terms:
        dy *= torch.arange(n, device="cuda")[:, None] == torch.randint(0, n, (1, o), generator=g, device="cuda")
    weight, before = 1 + randn(g, 1, h, std=0.3), randn(g, o, h, dtype=out)
    dw = wgrad(dy, checkpoint(x, "i8"), weight, before.clone(), accumulate)
    v = reference_checkpoint(x, "i8")[2]
    v = v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()
    size, exact = (dy.double().abs().T @ v.abs()) * weight.double().abs(), (dy.double().T @ v) * weight.double()
    if accumulate:
        exact = exact + before.double()
    left = 2.0 ** -15 if out == "bf16" else 0.0
    within(dw, exact, (left + ROW + 2 * (3 * (terms or n) + 64) * U32) * size + (U[DT[out]] + 2 * U32) * exact.abs(), "dw")


@pytest.mark.parametrize("n,o,h,norm", [(200, 4096, 5120, None), (1100, 5000, 4000, "bf16"), (70, 20000, 1300, None)])
def test_wgrad_more_tiles_than_pairs(n, o, h, norm):
    check_wgrad(n, o, h, norm=norm)
    check_wgrad(n, o, h, norm=norm, fmt="e4m3", out="f32", accumulate=True)


def test_wgrad_workspace_of_more_tokens():
    dy, x = randn(gen(1), 5000, 256, dtype="bf16"), randn(gen(2), 5000, 520, dtype="bf16")
    c = checkpoint(x, "i8")
    dw = torch.empty(256, 520, dtype=torch.bfloat16, device="cuda")
    ws = scratch(lst.lst_checkpoint_wgrad_workspace_bytes(mat(dy), lst.checkpoint(*c), mat(dw)))
    weight = torch.ones(1, 520, device="cuda")
    for n in (1, 64, 100, 511, 512, 513, 1024, 2049, 4999):
        for w in (None, weight):
            a = wgrad(dy[:n], (c[0][:n], c[1][:n], "i8"), w, torch.empty_like(dw), False, ws)
            assert torch.equal(a, wgrad(dy[:n], (c[0][:n], c[1][:n], "i8"), w, dw, False))


def test_wgrad_of_no_tokens():
    dy = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    c = (*lst.checkpoint_buffers(0, 32), "i8")
    for t in (torch.bfloat16, torch.float32):
        dw = torch.ones(16, 32, dtype=t, device="cuda")
        lst.lst_checkpoint_wgrad(mat(dy), lst.checkpoint(*c), None, EPS, mat(dw), True, 0, 0, stream())
        assert (dw == 1).all()
        lst.lst_checkpoint_wgrad(mat(dy), lst.checkpoint(*c), None, EPS, mat(dw), False, 0, 0, stream())
        assert not dw.any()


@pytest.mark.parametrize("norm", [False, True])
def test_wgrad_non_finite_blocks_stay_in_their_columns(norm):
    n, o, h = 300, 40, 256
    dy, x = randn(gen(1), n, o, dtype="bf16"), randn(gen(2), n, h, dtype="bf16")
    x[7, 70] = float("nan")
    weight = torch.ones(1, h, device="cuda") if norm else None
    dw = wgrad(dy, checkpoint(x, "i8"), weight, torch.empty(o, h, device="cuda"), False)
    bad = torch.zeros(h, dtype=torch.bool, device="cuda")
    bad[slice(None) if norm else slice(64, 96)] = True  # the norm of a row with a NaN is NaN in all of it
    assert torch.isnan(dw[:, bad]).all() and torch.isfinite(dw[:, ~bad]).all()


@pytest.mark.parametrize("n", [40, 700])
@pytest.mark.parametrize("norm,out", [(False, "bf16"), (True, "bf16"), (True, "f32")])
def test_wgrad_infinities_of_dy(n, norm, out):
    """An infinity in dy gives what it gives in the formula: infinities of the values' signs, NaN times a zero, NaN
    where two of them differ."""
    o, h = 48, 2056
    g = gen(n)
    dy, x = randn(g, n, o, dtype="bf16"), randn(g, n, h, dtype="bf16")
    x[3, 1000:1100] = 0.0
    dy[3, 5], dy[7, 6], dy[n - 1, 9], dy[2, 9], dy[1, 11] = float("inf"), -float("inf"), float("inf"), float("inf"), float("nan")
    weight = 1 + 0.1 * torch.rand(1, h, generator=g, device="cuda") if norm else None
    c = checkpoint(x, "i8")
    dw = wgrad(dy, c, weight, torch.empty(o, h, dtype=DT[out], device="cuda"), False)
    v = reference_checkpoint(x, "i8")[2]
    if norm:
        v = v * (v.square().mean(1, keepdim=True) + EPS).rsqrt() * weight.double()
    exact = dy.double().T @ v
    for bad in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(bad(dw), bad(exact))
    assert torch.isfinite(dw[[i for i in range(o) if i not in (5, 6, 9, 11)]]).all()
    zero = checkpoint(torch.zeros_like(x), "i8")  # all parts of a zero are zero
    dy = torch.full_like(dy, 3.0e38)
    assert not wgrad(dy, zero, weight, torch.full_like(dw, 7.0), False).any()


def test_wgrad_zero_rows_and_largest_values():
    """Rows of zeros; values near the ends of bf16's range, whose products stay in fp32's."""
    n, o, h = 128, 64, 96
    x = torch.zeros(n, h, dtype=torch.bfloat16, device="cuda")
    x[1], x[2] = 2.0 ** 120, 2.0 ** -120
    dy = torch.zeros(n, o, dtype=torch.bfloat16, device="cuda")
    dy[0], dy[1], dy[2] = 5.0, 2.0 ** -10, 2.0 ** 10
    dw = wgrad(dy, checkpoint(x, "i8"), None, torch.empty(o, h, device="cuda"), False)
    assert (dw == 2.0 ** 110).all()
    x[1] = 0
    dw = wgrad(dy, checkpoint(x, "e4m3"), None, torch.empty(o, h, device="cuda"), False)
    assert (dw == 2.0 ** -110).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Layer:
    """A forward and backward step of a layer boundary with its checkpoints, in buffers of its own."""

    def __init__(self, n=257, h=264, o=136, seed=3):
        self.p = Norm(n, h, gate_rows=1, seed=seed)
        self.dq = randn(gen(seed), n, o, dtype="bf16")
        self.h, self.z, self.dx, self.dy = (self.p.new() for _ in range(4))
        self.h8, self.y8 = ((*lst.checkpoint_buffers(n, h), f) for f in ("i8", "e4m3"))
        self.dw = torch.empty(o, h, dtype=torch.bfloat16, device="cuda")
        self.grads = [torch.empty_like(v) for v in (self.p.gate, self.p.w_post, self.p.w_pre)]
        self.ws = scratch(max(lst.lst_residual_norm_grad_workspace_bytes(n, h, 1),
                              lst.lst_checkpoint_wgrad_workspace_bytes(mat(self.dq), lst.checkpoint(*self.h8), mat(self.dw))))

    def step(self):
        p, ws, s = self.p, self.ws, stream()
        lst.lst_residual_norm(mat(p.x), mat(p.y), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(self.h), mat(self.z),
                              lst.checkpoint(*self.h8), lst.checkpoint(*self.y8), s)
        lst.lst_checkpoint_wgrad(mat(self.dq), lst.checkpoint(*self.h8), mat(p.w_pre), EPS, mat(self.dw), False, ws.data_ptr(), ws.numel(), s)
        lst.lst_residual_norm_grad(mat(p.dh), mat(p.dz), lst.checkpoint(*self.h8), lst.checkpoint(*self.y8), mat(p.gate), mat(p.w_post), mat(p.w_pre),
                                   p.params, mat(self.dx), mat(self.dy), *map(mat, self.grads), False, ws.data_ptr(), ws.numel(), s)
        lst.lst_checkpoint_restore(lst.checkpoint(*self.h8), mat(self.h), s)

    def results(self):
        return [t.clone() for t in (self.h, self.z, self.dx, self.dy, self.dw, *self.grads, self.h8[0], self.y8[1])]

    def clear(self):
        for t in (self.h, self.z, self.dx, self.dy, self.dw, *self.grads):
            t.fill_(float("nan"))


def test_side_stream_and_graph():
    a = Layer()
    a.step()
    expected = a.results()
    torch.cuda.synchronize()
    a.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), expected))
    a.clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(3):
        a.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.results(), expected))
    # new inputs in the same memory
    a.p.x.mul_(-0.5)
    graph.replay()
    replayed = a.results()
    a.step()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), replayed)) and not torch.equal(replayed[2], expected[2])
    lst.lst_operator_status()


def test_two_threads_on_two_streams():
    layers = [Layer(seed=3), Layer(n=700, h=777, o=300, seed=5)]
    expected = []
    for layer in layers:
        layer.step()
        expected.append(layer.results())
        layer.clear()
    torch.cuda.synchronize()
    failed = []

    def work(layer, want):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                layer.step()
            s.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(layer.results(), want)):
                failed.append(layer)

    threads = [threading.Thread(target=work, args=t) for t in zip(layers, expected)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("h,pad,shift", [(520, 8, 0), (520, 3, 1), (777, 0, 0)])
def test_results_leave_the_space_between_rows_alone(h, pad, shift):
    p = Norm(40, h, pad=pad, shift=shift)
    h8 = checkpoint(p.x, "i8")
    outs = [p.new() for _ in range(4)]
    dw = strided(torch.zeros(72, h, dtype=torch.bfloat16, device="cuda"), pad, shift, 7.0)
    ws = scratch(lst.lst_residual_norm_grad_workspace_bytes(40, h, 1))
    lst.lst_residual_norm(mat(p.x), mat(p.y), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(outs[0]), mat(outs[1]), None, None, stream())
    lst.lst_residual_norm_grad(mat(p.dh), mat(p.dz), mat(p.x), mat(p.y), mat(p.gate), mat(p.w_post), mat(p.w_pre), p.params, mat(outs[2]), mat(outs[3]),
                               None, None, None, False, ws.data_ptr(), ws.numel(), stream())
    wgrad(randn(gen(1), 40, 72, dtype="bf16"), h8, None, dw, False)
    for t in outs + [dw]:
        base = t._base if t._base is not None else t
        whole = base.flatten() if base.dim() == 1 else base.reshape(-1)
        keep = torch.ones_like(whole, dtype=torch.bool)
        keep[shift:].view(t.shape[0], h + pad)[:, :h] = False
        assert (whole[keep] == 7.0).all()
        assert torch.isfinite(t).all() and t.any()


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_checkpointed_layers
    finally:
        sys.path.pop(0)
    return train_checkpointed_layers


def test_example_runs():
    means = example().train(3, log=None)
    assert len(means) == 3 and all(m == m and 0.0 < m < 100.0 for m in means)


def test_example_gradients():
    """Against the same model in 64 bits by autograd. Expected: integers keep values to 0.8 % (RMS), which enters a
    gradient twice, 1 %; bf16 roundings of 0.1 to 0.2 % each, some twenty in a row, 1 %; one in some 700 of the MLP's
    inner values lies so near zero that the rounded sum has the other sign, which replaces as many entries of its
    gradient, sqrt(1 / 700) = 4 %. Sum 6 %, bound 10 %."""
    e = example()
    model = e.Model(7)
    g = torch.Generator(device="cuda").manual_seed(11)
    for name, w in model.w.items():  # norms and gates other than one
        if w.shape[0] == 1:
            w.mul_(1 + 0.2 * torch.randn(w.shape, generator=g, device="cuda"))
    tokens, targets = (torch.randint(0, e.VOCAB, (e.TOKENS,), generator=g, device="cuda") for _ in range(2))
    mean = model.gradients(tokens, targets)
    lst.lst_operator_status()
    w = {k: v.double().requires_grad_() for k, v in model.w.items()}

    def norm(x, weight):
        return x / (x.square().mean(1, keepdim=True) + e.EPS).sqrt() * weight

    x = w["embed_tokens"][tokens]
    for i in range(e.LAYERS):
        out = torch.relu(norm(x, w[f"norm_{i}"]) @ w[f"up_{i}"].T) @ w[f"down_{i}"].T
        x = x + e.BRANCH * w[f"gate_{i}"] * norm(out, w[f"post_norm_{i}"])
    loss = torch.nn.functional.cross_entropy(norm(x, w["final_norm"]) @ w["lm_head"].T, targets)
    loss.backward()
    assert abs(float(mean) - loss.item()) <= 0.01 * loss.item()
    for name, v in w.items():
        off = float((model.g[name].double() - v.grad).norm() / v.grad.norm())
        assert off <= 0.1, f"{name}: {off:.3f}"
