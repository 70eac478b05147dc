"""include/zq_layers.h without a GPU: the library exports what the header
declares, every refusal comes before anything is enqueued (the pointers here are
made up), the workspace helpers, and the binding's own checks."""
import os
import re
import shutil
import subprocess

import pytest
import torch

from weight_communication_zero_amd import zq

L = zq.lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000000
GB = 1 << 30
OK, NULL, SIZE, BLOCK, ALIGN, ALIAS, DTYPE = (zq.ZQ_OK, zq.ZQ_ERR_NULL, zq.ZQ_ERR_SIZE, zq.ZQ_ERR_BLOCK,
                                              zq.ZQ_ERR_ALIGN, zq.ZQ_ERR_ALIAS, zq.ZQ_ERR_DTYPE)


def at(i):
    return FAKE + i * GB


def test_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "zq_layers.h")) as f:
        names = set(re.findall(r"^(?:zq_status|size_t)\s+(zq_\w+)\s*\(", f.read(), re.M))
    assert len(names) == 10
    for name in names:
        assert hasattr(L, name), name


def swiglu(gate=at(0), up=at(1), t=1, n=100, block=64, h=at(2), gc=at(3), gs=at(4), uc=at(5), us=at(6)):
    return L.zq_swiglu_int8(gate, up, t, n, block, h, gc, gs, uc, us, None)


def swiglu_grad(gc=at(0), gs=at(1), uc=at(2), us=at(3), block=64, dh=at(4), t=1, n=100, dg=at(5), du=at(6), h=None):
    return L.zq_swiglu_grad_int8(gc, gs, uc, us, block, dh, t, n, dg, du, h, None)


def test_swiglu_refusals():
    for call, outs, ins in ((swiglu, ("h", "gc", "uc", "gs", "us"), ("gate", "up")),
                            (swiglu_grad, ("dg", "du"), ("gc", "gs", "uc", "us", "dh"))):
        for t in (-1, 3):
            assert call(t=t) == DTYPE
        for b in (0, 16, 48, 8192):
            assert call(block=b) == BLOCK
        assert call(n=(1 << 60) + 1) == SIZE
        assert call(n=0, **{k: None for k in outs + ins}) == OK
        for k in outs + ins:
            assert call(**{k: None}) == NULL
            assert call(**{k: at(9) + (2 if k in ("gs", "us") else 8)}) == ALIGN
        for o in outs:  # an output on the last bytes of another buffer
            for k in set(outs + ins) - {o}:
                size = {"gs": 8, "us": 8}.get(k, 100 if k in ("gc", "uc") else 200)
                assert call(**{k: at(9), o: at(9) + (size - 1) // 16 * 16}) == ALIAS, (o, k)
    assert swiglu_grad(h=at(4)) == ALIAS
    assert swiglu_grad(h=at(7) + 4) == ALIGN


def linear(dy=at(0), t=1, codes=at(1), scales=at(2), block=64, n=10, o=24, i=40, grad=at(3), g=0, mode=0, ws=at(4),
           wb=None):
    wb = L.zq_linear_grad_workspace(n, o, i) if wb is None else wb
    return L.zq_linear_grad_int8(dy, t, codes, scales, block, n, o, i, grad, g, mode, ws, wb, None)


def test_linear_grad_refusals():
    for k in ({"t": 0}, {"t": 3}, {"g": -1}, {"mode": 2}, {"mode": -1}):
        assert linear(**k) == DTYPE
    assert linear(block=100) == BLOCK
    for k in ({"n": (1 << 20) + 1}, {"o": 0}, {"i": 0}, {"o": (1 << 20) + 1}, {"i": (1 << 20) + 1},
              {"o": 1 << 18, "i": (1 << 18) + 1}):
        assert linear(**k) == SIZE
        assert L.zq_linear_grad_workspace(k.get("n", 10), k.get("o", 24), k.get("i", 40)) == 0
    assert linear(wb=L.zq_linear_grad_workspace(10, 24, 40) - 1) == SIZE
    for k in ("dy", "codes", "scales", "grad", "ws"):
        assert linear(**{k: None}) == NULL
        assert linear(**{k: at(9) + 2}) == ALIGN
    assert linear(n=0, mode=1, dy=None, codes=None, scales=None, ws=None, grad=None) == OK
    assert linear(n=0, grad=None) == NULL and linear(n=0, grad=at(3) + 4) == ALIGN
    assert linear(grad=at(0) + 10 * 24 * 2 - 16) == ALIAS
    assert linear(grad=at(1) + 10 * 40 - 16) == ALIAS
    assert linear(ws=at(3) + 24 * 40 * 4 - 16) == ALIAS
    assert linear(g=1, grad=at(2) - 24 * 40 * 2 + 16) == ALIAS


def loss(x=at(0), t=1, n=10, d=64, w=at(1), rows=50, ids=at(2), it=1, loss=at(3), lse=at(4), piece=0, ws=at(5),
         wb=None):
    wb = L.zq_ce_loss_workspace(n, rows, d, piece) if wb is None else wb
    return L.zq_ce_loss(x, t, n, d, w, rows, ids, it, 1.0, loss, lse, piece, ws, wb, None)


def loss8(block=64, scales=at(6), x=at(0), t=1, n=10, d=64, w=at(1), rows=50, ids=at(2), it=1, loss=at(3), lse=at(4),
          piece=0, ws=at(5), wb=None):
    wb = L.zq_ce_loss_workspace(n, rows, d, piece) if wb is None else wb
    return L.zq_ce_loss_int8(x, t, n, d, w, scales, block, rows, ids, it, 1.0, loss, lse, piece, ws, wb, None)


def grad(x=at(0), t=1, n=10, d=64, w=at(1), rows=50, ids=at(2), it=1, lse=at(3), dl=at(4), dx=at(5), dw=at(6), g=0,
         mode=0, piece=0, ws=at(7), wb=None):
    wb = L.zq_ce_grad_workspace(n, rows, d, piece) if wb is None else wb
    return L.zq_ce_grad(x, t, n, d, w, rows, ids, it, 1.0, lse, dl, dx, dw, g, mode, piece, ws, wb, None)


def grad8(block=64, scales=at(8), x=at(0), t=1, n=10, d=64, w=at(1), rows=50, ids=at(2), it=1, lse=at(3), dl=at(4),
          dx=at(5), dw=at(6), g=0, mode=0, piece=0, ws=at(7), wb=None):
    wb = L.zq_ce_grad_workspace(n, rows, d, piece) if wb is None else wb
    return L.zq_ce_grad_int8(x, t, n, d, w, scales, block, rows, ids, it, 1.0, lse, dl, dx, dw, g, mode, piece, ws, wb,
                             None)


@pytest.mark.parametrize("call", [loss, loss8, grad, grad8])
def test_ce_refusals(call):
    for k in ({"t": 0}, {"t": 3}, {"it": 2}):
        assert call(**k) == DTYPE
    helper = L.zq_ce_grad_workspace if call in (grad, grad8) else L.zq_ce_loss_workspace
    for k in ({"rows": 0}, {"d": 0}, {"rows": (1 << 24) + 1}, {"d": (1 << 20) + 1}, {"n": (1 << 20) + 1},
              {"n": 1 << 18, "d": (1 << 18) + 1}):
        assert call(**k) == SIZE
        assert helper(k.get("n", 10), k.get("rows", 50), k.get("d", 64), 0) == 0
    assert call(wb=helper(10, 50, 64, 0) - 1) == SIZE
    names = ["x", "w", "ids", "lse", "ws"] + (["dl"] if call in (grad, grad8) else ["loss"])
    if call in (loss8, grad8):
        names.append("scales")
        for b in (0, 16, 33, 8192):
            assert call(block=b) == BLOCK
    for k in names:
        assert call(**{k: None}) == NULL, k
        assert call(**{k: at(9) + 2}) == ALIGN, k
    assert call(ids=at(9) + 4) == ALIGN and call(x=at(9) + 8) == ALIGN
    assert call(ws=at(0) + 10 * 64 * 2 - 16) == ALIAS
    assert call(ws=at(2) + 64) == ALIAS
    if call in (loss, loss8):
        assert call(lse=at(3) + 36) == ALIAS and call(loss=at(0) + 1276) == ALIAS
        assert call(n=0, x=None, w=None, ids=None, loss=None, lse=None, ws=None) == OK
    else:
        for k in ({"g": 3}, {"mode": 2}):
            assert call(**k) == DTYPE
        assert call(dx=None, dw=None) == NULL
        assert call(dx=at(5) + 4) == ALIGN and call(dw=at(6) + 4) == ALIGN
        assert call(dx=at(6) + 50 * 64 * 4 - 16) == ALIAS and call(dw=at(4)) == ALIAS
        assert call(g=1, dx=at(1) + (50 * 64 - 16 if call is grad8 else 50 * 128 - 16)) == ALIAS
        assert call(n=0, mode=1, x=None, w=None, ids=None, lse=None, dl=None, dx=None, dw=None, ws=None) == OK
        assert call(n=0, dw=None) == OK and call(n=0, dw=at(6) + 8) == ALIGN


def test_workspace_grows_with_the_piece_and_is_bounded():
    for helper in (L.zq_ce_loss_workspace, L.zq_ce_grad_workspace):
        small, mid, whole = (helper(4096, 32000, 2048, p) for p in (256, 8192, 32000))
        assert 0 < small < mid < whole
        assert helper(4096, 32000, 2048, 1) == small                   # pieces are multiples of 256
        assert helper(4096, 32000, 2048, 1 << 40) == whole             # and no larger than the vocabulary
        assert helper(1 << 20, 1 << 24, 1 << 16, 1 << 60) > 0
    # The default piece: about 512 MiB each of probabilities and of staged rows, beside what the tokens need.
    n, d = 16384, 4096
    tokens = n * (4 * 4 + 2 * d + 4 * d)
    assert L.zq_ce_grad_workspace(n, 1 << 24, d, 0) < tokens + 2 * (1 << 29) + (1 << 28)


def test_binding_refuses_what_it_can_see():
    cpu = torch.zeros(8, 8, dtype=torch.bfloat16)
    i8 = torch.zeros(8, 8, dtype=torch.int8)
    f = torch.zeros(8)
    ws = torch.zeros(64, dtype=torch.uint8)
    ids = torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError, match="gate must be a GPU tensor"):
        zq.zq_swiglu_int8(cpu, cpu, 32, cpu, i8, f, i8, f)
    with pytest.raises(ValueError, match="gate_codes must be a GPU tensor"):
        zq.zq_swiglu_grad_int8(i8, f, i8, f, 32, cpu, cpu, cpu)
    with pytest.raises(ValueError, match="dy has 8 columns, grad 4 rows"):
        zq.zq_linear_grad_int8(cpu, i8, f, 32, torch.zeros(4, 8), 0, ws)
    with pytest.raises(ValueError, match="two dimensions"):
        zq.zq_linear_grad_int8(cpu.reshape(-1), i8, f, 32, torch.zeros(4, 8), 0, ws)
    with pytest.raises(ValueError, match="two dimensions"):
        zq.zq_ce_loss(cpu, cpu.reshape(-1), ids, 1.0, f, f, ws)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        zq.zq_ce_loss(cpu, cpu, ids, 1.0, f, f, ws)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        zq.zq_ce_grad_int8(cpu, i8, f, 32, ids, 1.0, f, f, cpu, cpu, 0, ws)


def test_header_is_c99_and_the_library_links_from_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    src = tmp_path / "use_zq_layers.c"
    src.write_text(r'''
#include <stdio.h>
#include "zq_layers.h"
int main(void) {
    if (zq_linear_grad_workspace(0, 10, 10) != 0 || zq_linear_grad_workspace(7, 10, 10) == 0) return 1;
    if (zq_ce_loss_workspace(3, 10, 8, 0) == 0 || zq_ce_grad_workspace(3, 0, 8, 0) != 0) return 2;
    if (zq_swiglu_int8(NULL, NULL, ZQ_BF16, 5, 64, NULL, NULL, NULL, NULL, NULL, NULL) != ZQ_ERR_NULL) return 3;
    if (zq_ce_loss(NULL, ZQ_FP32, 3, 8, NULL, 5, NULL, ZQ_I64, 1.0f, NULL, NULL, 0, NULL, 0, NULL) != ZQ_ERR_DTYPE)
        return 4;
    puts("ok");
    return 0;
}
''')
    exe = tmp_path / "use_zq_layers"
    lib = os.path.join(ROOT, "weight_communication_zero_amd", "libzq.so")
    r = subprocess.run([gcc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), lib, "-Wl,-rpath," + os.path.dirname(lib), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
