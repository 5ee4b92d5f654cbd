"""Residual norms and checkpoints without a GPU: argument validation that happens
before any CUDA call, workspace sizes, and the C structs against the binding."""

import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def L():
    from optimizer_update_gb300 import lst
    if not os.path.exists(lst.LIB_PATH):
        from optimizer_update_gb300 import build
        build.build()
    return lst


P = 1 << 20  # a plausible, never dereferenced, aligned address
BAD, MISALIGNED = 1, 2


def mat(L, rows, cols, dtype=0, stride=None, data=P):
    return L.lst_matrix(data, rows, cols, cols if stride is None else stride, dtype)


def kept(L, rows, cols, fmt=0, stride=None, scale_stride=None, data=P, scales=P):
    return L.lst_checkpoint(data, scales, rows, cols, (cols + 15) // 16 * 16 if stride is None else stride,
                            (cols + 31) // 32 if scale_stride is None else scale_stride, fmt)


def refused(L, status, fn, *args):
    with pytest.raises(L.LstError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


def test_checkpoint_refusals(L):
    x, c = mat(L, 4, 40), kept(L, 4, 40)
    for m, k, status in [
            (None, c, BAD), (x, None, BAD), (mat(L, 5, 40), c, BAD), (mat(L, 4, 41), c, BAD), (mat(L, 4, 40, dtype=2), c, BAD),
            (mat(L, 4, 40, data=None), c, BAD), (mat(L, 4, 40, data=P + 1), c, MISALIGNED), (x, kept(L, 4, 40, fmt=2), BAD),
            (x, kept(L, 4, 40, fmt=-1), BAD), (x, kept(L, 4, 40, stride=32), BAD), (x, kept(L, 4, 40, scale_stride=1), BAD),
            (x, kept(L, 4, 40, stride=40), MISALIGNED), (x, kept(L, 4, 40, data=P + 8), MISALIGNED), (x, kept(L, 4, 40, data=None), BAD),
            (x, kept(L, 4, 40, scales=None), BAD), (mat(L, -1, 40), kept(L, -1, 40), BAD), (x, kept(L, 4, 40, stride=1 << 37), BAD)]:
        refused(L, status, L.lst_checkpoint_save, m, k)
        refused(L, status, L.lst_checkpoint_restore, k, m)
    L.lst_checkpoint_save(mat(L, 0, 40, data=None), kept(L, 0, 40, data=None, scales=None))  # nothing to do
    L.lst_checkpoint_restore(kept(L, 0, 40, data=None, scales=None), mat(L, 0, 40, data=None))


def test_norm_refusals(L):
    n, h = 6, 64
    r, v, p = mat(L, n, h), mat(L, 1, h), L.residual_params()
    ok = (r, r, mat(L, 2, h), v, v, p, r, r, kept(L, n, h), kept(L, n, h))
    for change, status in [
            ({0: None}, BAD), ({1: mat(L, n, h + 1)}, BAD), ({1: mat(L, n, h, dtype=1)}, BAD), ({2: mat(L, 4, h)}, BAD),
            ({2: mat(L, 0, h)}, BAD), ({2: mat(L, 2, h + 8)}, BAD), ({3: mat(L, 2, h)}, BAD), ({4: mat(L, 1, h - 1)}, BAD),
            ({5: None}, BAD), ({5: L.residual_params(eps=0.0)}, BAD), ({5: L.residual_params(eps=float("nan"))}, BAD),
            ({5: L.residual_params(residual_scale=float("inf"))}, BAD), ({5: L.residual_params(branch_scale=float("nan"))}, BAD),
            ({6: mat(L, n - 1, h)}, BAD), ({7: None}, BAD), ({4: None}, BAD), ({7: mat(L, n, h, dtype=1)}, BAD),
            ({8: kept(L, n, h + 32)}, BAD), ({9: kept(L, n + 1, h)}, BAD), ({1: None}, BAD), ({1: None, 2: None, 3: None}, BAD),
            ({4: None, 6: None, 7: None, 8: None}, BAD), ({6: mat(L, n, h, data=P + 1)}, MISALIGNED), ({8: kept(L, n, h, data=P + 4)}, MISALIGNED),
            ({3: mat(L, 1, h, dtype=1, data=P + 2)}, MISALIGNED)]:
        refused(L, status, L.lst_residual_norm, *[change.get(i, a) for i, a in enumerate(ok)])
    big = mat(L, 1, 16385)
    refused(L, BAD, L.lst_residual_norm, big, None, None, None, mat(L, 1, 16385), p, None, big)
    refused(L, BAD, L.lst_residual_norm, mat(L, 3, 0), None, None, None, None, p, mat(L, 3, 0), None)
    e = mat(L, 0, h, data=None)
    L.lst_residual_norm(e, e, None, v, v, p, e, e)  # nothing to do


def test_norm_grad_refusals(L):
    n, h = 6, 64
    r, v, g, p = mat(L, n, h), mat(L, 1, h), mat(L, 2, h), L.residual_params()
    ws = L.lst_residual_norm_grad_workspace_bytes(n, h, 2)
    assert ws > L.lst_residual_norm_grad_workspace_bytes(n, h, 0) > 0
    #      dh dz h  y  gate post pre params dx dy dgate dpost dpre acc ws bytes
    ok = (r, r, r, r, g, v, v, p, r, r, g, v, v, False, P, ws)
    for change, status in [
            ({0: None, 1: None}, BAD), ({0: mat(L, n + 1, h)}, BAD), ({1: mat(L, n, h, dtype=1)}, BAD), ({2: None}, BAD),
            ({2: mat(L, n, h, dtype=1)}, BAD), ({2: kept(L, n, h + 1)}, BAD), ({3: None}, BAD), ({3: mat(L, n, h, dtype=1)}, BAD),
            ({4: None}, BAD), ({4: mat(L, 3, h)}, BAD), ({4: mat(L, 4, h), 10: mat(L, 4, h)}, BAD), ({5: None}, BAD), ({6: None}, BAD),
            ({1: None}, BAD), ({1: None, 6: None}, BAD), ({7: None}, BAD), ({7: L.residual_params(eps=-1.0)}, BAD),
            ({8: mat(L, n, h, dtype=1)}, BAD), ({9: mat(L, n, h - 8)}, BAD), ({10: mat(L, 1, h)}, BAD), ({11: mat(L, 1, h + 1)}, BAD),
            ({12: mat(L, 2, h)}, BAD), ({14: 0}, BAD), ({15: ws - 1}, BAD), ({14: P + 128}, MISALIGNED), ({8: mat(L, n, h, data=P + 1)}, MISALIGNED)]:
        refused(L, status, L.lst_residual_norm_grad, *[change.get(i, a) for i, a in enumerate(ok)])
    # h as a matrix and as a checkpoint
    with pytest.raises(L.LstError):
        L._check(L.lib().lst_residual_norm_grad(r, r, r, kept(L, n, h), r, None, g, v, v, p, r, r, g, v, v, 0, P, ws, None))
    for args in ((0, h, 0), (n, 0, 0), (n, 16385, 0), (n, h, -1), (n, h, n + 1), (1 << 31, h, 0)):
        assert L.lst_residual_norm_grad_workspace_bytes(*args) == 0


@pytest.mark.parametrize("h", [1, 40, 2048, 4096, 16384])
def test_norm_grad_workspace_serves_fewer_tokens(L, h):
    counts = [1, 2, 7, 100, 151, 152, 153, 1000, 5000, 100000]
    for rows in (0, 1):
        sizes = [L.lst_residual_norm_grad_workspace_bytes(n, h, rows) for n in counts]
        assert sizes == sorted(sizes)
    assert L.lst_residual_norm_grad_workspace_bytes(1000, h, 1) == L.lst_residual_norm_grad_workspace_bytes(1000, h, 1000)
    assert sizes[-1] < 64 << 20  # sums per CTA, not per token


def test_wgrad_refusals(L):
    n, o, h = 100, 48, 64
    dy, c, dw, w = mat(L, n, o), kept(L, n, h), mat(L, o, h), mat(L, 1, h)
    ws = L.lst_checkpoint_wgrad_workspace_bytes(dy, c, dw)
    assert ws > 0
    ok = (dy, c, w, 1e-5, dw, False, P, ws)
    for change, status in [
            ({0: None}, BAD), ({1: None}, BAD), ({4: None}, BAD), ({0: mat(L, n, o, dtype=1)}, BAD), ({0: mat(L, n + 1, o)}, BAD),
            ({0: mat(L, n, o + 1)}, BAD), ({1: kept(L, n, h + 32)}, BAD), ({1: kept(L, n, h, fmt=7)}, BAD), ({2: mat(L, 2, h)}, BAD),
            ({2: mat(L, 1, h + 1)}, BAD), ({3: 0.0}, BAD), ({3: float("nan")}, BAD), ({4: mat(L, o, h, dtype=5)}, BAD), ({6: 0}, BAD),
            ({7: ws - 257}, BAD), ({6: P + 16}, MISALIGNED), ({1: kept(L, n, h, data=P + 8)}, MISALIGNED), ({4: mat(L, o, h, data=P + 1)}, MISALIGNED)]:
        refused(L, status, L.lst_checkpoint_wgrad, *[change.get(i, a) for i, a in enumerate(ok)])
    many = (1 << 24) + 1
    refused(L, BAD, L.lst_checkpoint_wgrad, mat(L, many, o), kept(L, many, h), None, 0.0, dw, False, P, 1 << 60)
    for bad in ((None, c, dw), (dy, None, dw), (dy, c, None), (mat(L, many, o), kept(L, many, h), dw), (mat(L, n + 1, o), c, dw), (dy, c, mat(L, o, h + 1))):
        assert L.lst_checkpoint_wgrad_workspace_bytes(*bad) == 0
    # rows of dy off 16 bytes are copied: more (up to 512 tokens there is room for a copy of them anyway)
    many = kept(L, 1100, h)
    assert L.lst_checkpoint_wgrad_workspace_bytes(mat(L, 1100, o, data=P + 2), many, dw) > L.lst_checkpoint_wgrad_workspace_bytes(mat(L, 1100, o), many, dw)


@pytest.mark.parametrize("o,h", [(1, (1 << 31) - 1), (1, (1 << 31) - 4096), (1, (1 << 31) - (1 << 14) + 1), ((1 << 31) - 1, 1), ((1 << 31) - 255, 8)])
def test_wgrad_refuses_columns_that_32_bits_do_not_step_past(L, o, h):
    """A thread's next column is up to 4096 further, a tile's last one up to 256, and both are 32-bit numbers."""
    dy, c, dw = mat(L, 1, o), kept(L, 1, h), mat(L, o, h)
    assert L.lst_checkpoint_wgrad_workspace_bytes(dy, c, dw) == 0
    for norm in (None, mat(L, 1, h)):
        refused(L, BAD, L.lst_checkpoint_wgrad, dy, c, norm, 1e-5, dw, False, P, 1 << 60)
    widest = (1 << 31) - (1 << 14)
    o, h = min(o, widest), min(h, widest)
    assert L.lst_checkpoint_wgrad_workspace_bytes(mat(L, 1, o), kept(L, 1, h), mat(L, o, h)) > 0


@pytest.mark.parametrize("o,h", [(1, 1), (256, 2048), (11008, 4096), (300, 777), (16, 12293)])
def test_wgrad_workspace_serves_fewer_tokens(L, o, h):
    counts = sorted({max(1, (1 << i) + d) for i in range(17) for d in (-1, 0, 1, 100)})
    for data in (P, P + 2):
        sizes = [L.lst_checkpoint_wgrad_workspace_bytes(mat(L, n, o, data=data), kept(L, n, h), mat(L, o, h)) for n in counts]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_checkpoint_of_tensors(L):
    torch = pytest.importorskip("torch")
    values, scales = L.checkpoint_buffers(5, 40, "cpu")
    assert values.shape == (5, 40) and values.stride() == (48, 1) and scales.shape == (5, 2)
    c = L.checkpoint(values, scales, "e4m3")
    assert (c.rows, c.cols, c.stride, c.scale_stride, c.format, c.host) == (5, 40, 48, 2, L.LST_CHECKPOINT_E4M3, True)
    u8 = torch.uint8
    for v, s, fmt in [(values, scales, "int8"), (values[0], scales, "i8"), (values, scales[:4], "i8"), (values, scales[:, :1], "i8"),
                      (values.t(), scales, "i8"), (values.float(), scales, "i8"), (values, scales.float(), "i8"),
                      (torch.empty(1, 40, dtype=u8).expand(5, 40), scales, "i8"), (values, torch.empty(1, 2, dtype=u8).expand(5, 2), "i8"),
                      (torch.empty(5 * 48 - 8, dtype=u8).as_strided((5, 40), (48, 1)), scales, "i8")]:
        with pytest.raises(ValueError):
            L.checkpoint(v, s, fmt)
    with pytest.raises(ValueError, match="host memory"):
        L.lst_checkpoint_save(L.matrix(torch.zeros(5, 40)), c)
    assert L.checkpoint(values.view(torch.int8), scales).format == L.LST_CHECKPOINT_I8
    assert L.checkpoint(values[:1], scales[:1]).stride == 48


def test_c_structs_match_the_binding(L, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = {"lst_checkpoint": L.lst_checkpoint, "lst_residual_params": L.lst_residual_params}
    lines = []
    for name, s in fields.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in s._fields_]
    src = tmp_path / "offsets.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"lst.h\"\nint main(void) {" + "\n".join(lines) + "return 0; }\n")
    exe = tmp_path / "offsets"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for s in fields.values():
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want
