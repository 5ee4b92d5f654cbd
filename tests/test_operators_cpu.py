"""The training operators without a GPU: argument validation that happens before
any CUDA call, workspace sizes, and the C structs against the binding."""

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


def mat(L, rows, cols, dtype=0, stride=None, data=P):
    return L.lst_matrix(data, rows, cols, cols if stride is None else stride, dtype)


def idx(L, count, bits=64, data=P):
    return L.lst_indices(data, count, bits)


def refused(L, status, fn, *args):
    with pytest.raises(L.LstError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


def test_embed_refusals(L):
    bad, misaligned = L.LST_ERR_INVALID_ARG, L.LST_ERR_ALIGNMENT
    ok = (mat(L, 100, 8), idx(L, 4), mat(L, 4, 8))
    for args, status in [
            ((None, ok[1], ok[2]), bad), ((ok[0], None, ok[2]), bad), ((ok[0], ok[1], None), bad),
            ((ok[0], ok[1], mat(L, 5, 8)), bad), ((ok[0], ok[1], mat(L, 4, 9)), bad),
            ((mat(L, 100, 8, dtype=2), ok[1], ok[2]), bad), ((mat(L, 100, 8, stride=7), ok[1], ok[2]), bad),
            ((mat(L, -1, 8), ok[1], ok[2]), bad), ((ok[0], idx(L, 4, bits=16), ok[2]), bad),
            ((mat(L, 100, 8, data=None), ok[1], ok[2]), bad), ((ok[0], idx(L, 4, data=None), ok[2]), bad),
            ((mat(L, 100, 8, data=P + 1), ok[1], ok[2]), misaligned), ((ok[0], idx(L, 4, data=P + 4), ok[2]), misaligned),
            ((ok[0], ok[1], mat(L, 4, 8, dtype=1, data=P + 2)), misaligned)]:
        refused(L, status, L.lst_embed, *args)
    L.lst_embed(mat(L, 100, 8), idx(L, 0, data=None), mat(L, 0, 8, data=None))  # nothing to do


def test_embed_grad_refusals(L):
    ws = L.lst_embed_grad_workspace_bytes(4, 8, 100)
    assert ws > 0
    ok = (mat(L, 4, 8), idx(L, 4), mat(L, 100, 8), 1.0, False, P, ws)
    for change, status in [({0: None}, 1), ({1: idx(L, 5)}, 1), ({2: mat(L, 100, 9)}, 1), ({5: 0}, 1), ({6: ws - 1}, 1),
                           ({5: P + 128}, 2), ({2: mat(L, (1 << 30) + 1, 8)}, 1)]:
        args = [change.get(i, a) for i, a in enumerate(ok)]
        refused(L, status, L.lst_embed_grad, *args)


def test_xent_refusals(L):
    n, h, v = 4, 16, 1000
    ws = L.lst_xent_workspace_bytes(n, h, v, False)
    ok = (mat(L, n, h), mat(L, v, h), idx(L, n), -100, P, P, P, ws)
    for change, status in [({0: mat(L, n, h, dtype=1)}, 1), ({1: mat(L, v, h + 1)}, 1), ({2: idx(L, n + 1)}, 1),
                           ({1: mat(L, 0, h)}, 1), ({4: 0}, 1), ({5: 0}, 1), ({4: P + 2}, 2), ({6: 0}, 1), ({6: P + 8}, 2),
                           ({7: ws - 1}, 1), ({0: None}, 1)]:
        refused(L, status, L.lst_xent_loss, *[change.get(i, a) for i, a in enumerate(ok)])
    wg = L.lst_xent_workspace_bytes(n, h, v, True)
    assert wg > ws
    ok = (mat(L, n, h), mat(L, v, h), idx(L, n), -100, 1.0, P, P, P, mat(L, n, h), mat(L, v, h), False, P, wg)
    for change, status in [({8: mat(L, n + 1, h)}, 1), ({9: mat(L, v, h, dtype=1)}, 1), ({8: None}, 1), ({7: 0}, 1),
                           ({4: float("inf")}, 1), ({11: 0}, 1), ({12: 4096}, 1), ({7: P + 1}, 2)]:
        refused(L, status, L.lst_xent_grad, *[change.get(i, a) for i, a in enumerate(ok)])


@pytest.mark.parametrize("n,h,v,xs,ws,xo,wo", [(512, 2048, 32000, 3, 0, 0, 0), (512, 2048, 32000, 0, 0, 0, 2),
                                               (16, 2048, 32000, 0, 0, 0, 2), (16, 2048, 32000, 4, 4, 0, 0),
                                               (300, 64, 300, 0, 0, 6, 0), (300, 63, 300, 1, 1, 0, 0), (300, 63, 300, 0, 0, 0, 0),
                                               (270, 72, 500, 8, 16, 0, 0)])
def test_xent_workspace_for_the_operands(L, n, h, v, xs, ws, xo, wo):
    """The size for operands as they lie is what the loss asks for: enough, and not a granule less."""
    x, w, t = mat(L, n, h, stride=h + xs, data=P + xo), mat(L, v, h, stride=h + ws, data=P + wo), idx(L, n)
    off = any((m.data | m.stride * 2) % 16 for m in (x, w))
    for grad in (False, True):
        need = L.lst_xent_workspace_bytes_for(x, w, grad)
        plain = L.lst_xent_workspace_bytes_for(mat(L, n, (h + 7) // 8 * 8), mat(L, v, (h + 7) // 8 * 8), grad)
        assert need > plain if off else need >= plain - 4096
        if h % 8 == 0:
            assert plain == L.lst_xent_workspace_bytes(n, h, v, grad)
    need = L.lst_xent_workspace_bytes_for(x, w, False)
    refused(L, L.LST_ERR_INVALID_ARG, L.lst_xent_loss, x, w, t, -100, P, P, P, need - 1)
    # one row's copy more than the sizes alone give is not enough for a w off 16 bytes
    if ws % 8 or wo:
        refused(L, L.LST_ERR_INVALID_ARG, L.lst_xent_loss, x, w, t, -100, P, P, P, need - v * h * 2)
    for bad in ((None, w), (x, None), (x, mat(L, v, h + 1)), (mat(L, 0, h), w), (mat(L, (1 << 24) + 1, h), w)):
        assert L.lst_xent_workspace_bytes_for(*bad, True) == 0


@pytest.mark.parametrize("h,v", [(64, 300), (2048, 32000), (4096, 131072), (77, 50257), (256, 1000)])
def test_xent_workspace_serves_smaller_counts(L, h, v):
    """A workspace sized for the largest batch is enough for a shorter one."""
    counts = sorted({max(1, k + d) for k in [2 ** i for i in range(17)] + [3 * 2 ** i for i in range(6, 14)] for d in (-1, 0, 1, 5)})
    for grad in (False, True):
        sizes = [L.lst_xent_workspace_bytes(n, h, v, grad) for n in counts]
        assert sizes == sorted(sizes)
    for n in (1, 31, 63, 64, 65, 70, 128, 255, 256, 300):
        with pytest.raises(L.LstError, match="at least [0-9]+ needed") as e:
            L.lst_xent_loss(mat(L, n, h), mat(L, v, h), idx(L, n), -100, P, P, P, 256)
        need = int(str(e.value).split("at least ")[1].split()[0])
        assert all(L.lst_xent_workspace_bytes(m, h, v, False) >= need for m in counts if m >= n)


def test_orthogonalize_refusals(L):
    ws = L.lst_orthogonalize_workspace_bytes(2, 16, 32)
    a, o, p = mat(L, 16, 32), mat(L, 16, 32), L.ns_params()
    for args, status in [
            (([a], [mat(L, 16, 32, dtype=1)], p, P, ws), 1), (([a, mat(L, 16, 33)], [o, o], p, P, ws), 1),
            (([a, mat(L, 16, 32, dtype=1)], [o, o], p, P, ws), 1), (([a], [o], L.ns_params(steps=0), P, ws), 1),
            (([a], [o], L.ns_params(steps=21), P, ws), 1), (([a], [o], L.ns_params(eps=0.0), P, ws), 1),
            (([a], [o], p, 0, ws), 1), (([a], [o], p, P, 1000), 1), (([a], [o], p, P + 16, ws), 2),
            (([mat(L, 16, 32, data=P + 1)], [o], p, P, ws), 2)]:
        refused(L, status, L.lst_orthogonalize, *args)
    with pytest.raises(ValueError):
        L.lst_orthogonalize([a], [], p, P, ws)
    L.lst_orthogonalize([], [], p, 0, 0)


def test_muon_refusals(L):
    from optimizer_update_gb300 import Layout
    lay = Layout([("a", (16, 32), 0), ("n", (16,), 0)], "L12")
    ws = L.lst_muon_workspace_bytes(lay.handle)
    ok = [lay.handle, [P], L.muon_hparams(), L.adamw_hparams(), None, P, ws]
    for change, status in [({0: None}, 1), ({1: [0]}, 1), ({1: [P + 8]}, 2), ({2: None}, 1),
                           ({2: L.muon_hparams(lr=float("nan"))}, 1), ({2: L.muon_hparams(momentum=1.0)}, 1),
                           ({2: L.muon_hparams(rms_scale=-1.0)}, 1), ({2: L.muon_hparams(eps=0.0)}, 1),
                           ({2: L.muon_hparams(ns_steps=0)}, 1), ({3: L.adamw_hparams(step=0)}, 1),
                           ({4: [True, True]}, 1), ({5: 0}, 1), ({6: ws // 2}, 1), ({5: P + 64}, 2)]:
        refused(L, status, L.lst_muon_step, *[change.get(i, a) for i, a in enumerate(ok)])
    assert L.lst_muon_workspace_bytes(None) == 0


def test_workspace_sizes(L):
    # the loss alone needs statistics only: 8 bytes per token and 128 vocabulary entries, and little else
    n, h, v = 4096, 4096, 32000
    assert L.lst_xent_workspace_bytes(n, h, v, False) < n * 4 + n * (v // 128) * 8 + (1 << 16)
    # the gradient's pieces are bounded: 1 GiB of columns, however large the vocabulary
    big = L.lst_xent_workspace_bytes(n, 128, 1 << 20, True)
    assert (1 << 30) <= big < (1 << 30) + n * (1 << 20) // 128 * 8 + 40 * n * 128 * 4
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, -1)):
        assert L.lst_xent_workspace_bytes(*bad, True) == 0
    assert L.lst_orthogonalize_workspace_bytes(0, 8, 8) == 0
    # many matrices: no more than 4 GiB at a time
    assert L.lst_orthogonalize_workspace_bytes(1000, 4096, 4096) <= 4 << 30
    assert L.lst_embed_grad_workspace_bytes(-1, 8, 8) == 0


@pytest.mark.parametrize("hidden", [1, 1024, 2048, 4095, 3000000])
def test_embed_grad_workspace_serves_smaller_counts(L, hidden):
    """A workspace sized for the largest batch is enough for a shorter one, whatever the kernels do with few tokens."""
    counts = sorted({k + d for k in [2 ** i for i in range(18)] + [2432 * 32 // s for s in (1, 2, 4)] for d in (-31, -1, 0, 1, 32)
                     if k + d > 0})
    sizes = [L.lst_embed_grad_workspace_bytes(n, hidden, 32000) for n in counts]
    assert sizes == sorted(sizes)
    # and no less than the call itself asks for: one byte less than its own need is refused
    args = [mat(L, 9, hidden), idx(L, 9), mat(L, 32000, hidden), 1.0, False, P]
    need = L.lst_embed_grad_workspace_bytes(9, hidden, 32000)
    refused(L, 1, L.lst_embed_grad, *args, need - 257 if hidden < 3000000 else 1000)


def test_sizes_past_64_bits(L):
    """Sizes that no memory holds: no workspace of a size that wrapped around, and a refusal instead of a call with it."""
    top, big = (1 << 31) - 1, 1 << 30
    for rows, cols in ((1 << 40, 1 << 40), (top, top), (top + 1, 1), (1, top + 1), (1 << 62, 4)):
        assert L.lst_orthogonalize_workspace_bytes(1, rows, cols) == 0
    assert L.lst_xent_workspace_bytes(4, top, top, True) == 0 and L.lst_xent_workspace_bytes(4, 8, top + 1, False) == 0
    assert L.lst_embed_grad_workspace_bytes(4, top + 1, 8) == 0 and L.lst_embed_grad_workspace_bytes(1 << 30, 1 << 62, 8) == 0
    assert L.lst_orthogonalize_workspace_bytes(1, top, 64) > top * 64 * 2 and L.lst_embed_grad_workspace_bytes(1 << 30, 4096, 8) > 0
    assert L.lst_xent_workspace_bytes(1 << 24, 4096, 131072, True) > 0
    m = mat(L, top, top)
    refused(L, L.LST_ERR_INVALID_ARG, L.lst_orthogonalize, [m], [m], L.ns_params(), P, big)
    refused(L, L.LST_ERR_INVALID_ARG, L.lst_xent_loss, mat(L, 4, top), m, idx(L, 4), -100, P, P, P, big)


def test_tensor_arguments(L):
    import torch
    x = torch.zeros(6, 10)
    m = L.matrix(x[:, 2:7])
    assert (m.rows, m.cols, m.stride, m.dtype) == (6, 5, 10, L.LST_F32) and m.data == x.data_ptr() + 8
    assert L.matrix(torch.zeros(3, 4, dtype=torch.bfloat16)).dtype == L.LST_BF16
    for bad in (x.T, torch.zeros(3), torch.zeros(2, 2, dtype=torch.float16)):
        with pytest.raises(ValueError):
            L.matrix(bad)
    assert L.indices(torch.zeros(5, dtype=torch.int32)).bits == 32
    for bad in (torch.zeros(5), torch.zeros(5, 2, dtype=torch.int64)[:, 0]):
        with pytest.raises(ValueError):
            L.indices(bad)


def test_tensor_arguments_overlapping_rows(L):
    """Rows that share memory (an expanded gradient, a sliding window) are no matrix: their stride is below the column
    count, and a stride of the column count would reach past the storage."""
    import torch
    for bad in (torch.zeros(1, 4).expand(3, 4), torch.zeros(4).expand(3, 4), torch.zeros(9).as_strided((3, 4), (2, 1)),
                torch.zeros(1, 1).expand(3, 1), torch.zeros(3, 1, dtype=torch.bfloat16).expand(3, 4)):
        with pytest.raises(ValueError):
            L.matrix(bad)
    # one row, or none: the stride means nothing
    m = L.matrix(torch.zeros(1, 4).expand(1, 4))
    assert (m.rows, m.cols, m.stride) == (1, 4, 4)
    m = L.matrix(torch.zeros(5, 9)[2:3, 1:4])
    assert (m.rows, m.cols) == (1, 3) and m.stride >= 3
    m = L.matrix(torch.zeros(0, 4))
    assert (m.rows, m.cols) == (0, 4) and m.stride >= 4
    m = L.matrix(torch.zeros(7, 1)[::2])
    assert (m.rows, m.cols, m.stride) == (4, 1, 2)
    # a row stride is what the tensor says, also where rows are one element
    m = L.matrix(torch.zeros(4, 6)[:, 2:3])
    assert (m.rows, m.cols, m.stride) == (4, 1, 6)


def test_host_tensors_are_refused(L):
    """A tensor in host memory can be described, but no operator takes it: its kernels would read host addresses."""
    import torch
    m, w, t, p = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(10, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), P
    x, table, i = L.matrix(m), L.matrix(w), L.indices(t)
    dx, dw, di = mat(L, 4, 8), mat(L, 10, 8), idx(L, 4)  # stand for device memory
    big = 1 << 30
    for fn, args in [(L.lst_embed, (table, di, dx)), (L.lst_embed, (dw, i, dx)), (L.lst_embed, (dw, di, x)),
                     (L.lst_embed_grad, (x, di, dw, 1.0, False, p, big)), (L.lst_embed_grad, (dx, i, dw, 1.0, False, p, big)),
                     (L.lst_embed_grad, (dx, di, table, 1.0, False, p, big)),
                     (L.lst_xent_loss, (x, dw, di, -100, p, p, p, big)), (L.lst_xent_loss, (dx, table, di, -100, p, p, p, big)),
                     (L.lst_xent_loss, (dx, dw, i, -100, p, p, p, big)),
                     (L.lst_xent_grad, (x, dw, di, -100, 1.0, p, p, p, dx, dw, False, p, big)),
                     (L.lst_xent_grad, (dx, table, di, -100, 1.0, p, p, p, dx, dw, False, p, big)),
                     (L.lst_xent_grad, (dx, dw, i, -100, 1.0, p, p, p, dx, dw, False, p, big)),
                     (L.lst_xent_grad, (dx, dw, di, -100, 1.0, p, p, p, x, dw, False, p, big)),
                     (L.lst_xent_grad, (dx, dw, di, -100, 1.0, p, p, p, dx, table, False, p, big)),
                     (L.lst_orthogonalize, ([dx, x], [dx, dx], L.ns_params(), p, big)),
                     (L.lst_orthogonalize, ([dx, dx], [dx, x], L.ns_params(), p, big))]:
        with pytest.raises(ValueError):
            fn(*args)


def test_muon_arguments_cover_the_layout(L):
    """The library reads a mask entry per tensor and a pointer per block; a shorter list would be read past its end."""
    from optimizer_update_gb300 import Layout
    lay = Layout([("a", (200, 300), 0), ("n", (16,), 0), ("b", (16, 32), 1)], "L12")
    ws, hp = L.lst_muon_workspace_bytes(lay.handle), L.muon_hparams()
    for blocks, mask in [([P], None), ([P, P, P], None), ([P, P], [True]), ([P, P], []), ([P, P], [1, 0, 1, 0])]:
        with pytest.raises(ValueError):
            L.lst_muon_step(lay.handle, blocks, hp, None, mask, P, ws)
    # as long as the layout: on to the library, which wants more workspace
    refused(L, 1, L.lst_muon_step, lay.handle, [P, P], hp, None, [True, False, False], P, 0)
    refused(L, 1, L.lst_muon_step, lay.handle, [P, P], hp, None, None, P, 0)


STRUCTS = {"lst_matrix": ("data", "rows", "cols", "stride", "dtype"), "lst_indices": ("data", "count", "bits"),
           "lst_ns_params": ("steps", "eps"),
           "lst_muon_hparams": ("lr", "momentum", "weight_decay", "rms_scale", "eps", "nesterov", "ns_steps")}


def test_c_structs_match_the_binding(L, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = "".join(f'printf("{s} - %zu 0\\n", sizeof({s}));' + "".join(
        f'printf("{s} {f} %zu %zu\\n", offsetof({s}, {f}), sizeof((({s}*)0)->{f}));' for f in fs) for s, fs in STRUCTS.items())
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lst.h"\nint main(void) {' + lines + "return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n"):
        if not line:
            continue
        name, field, off, size = line.split()
        T = getattr(L, name)
        if field == "-":
            assert ctypes.sizeof(T) == int(off), name
        else:
            d = getattr(T, field)
            assert (d.offset, d.size) == (int(off), int(size)), (name, field)
    for name, fields in STRUCTS.items():
        assert [f for f, _ in getattr(L, name)._fields_] == list(fields)
