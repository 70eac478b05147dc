"""include/zq_train.h without a GPU: the library exports what the header
declares, the host helpers, and every refusal of the C ABI and of the binding
(all pointers below are fake and never dereferenced: each call fails
validation, or is a no-op, before any device work)."""
import ctypes as C
import os
import re
import shutil
import subprocess

import pytest
import torch

from weight_communication_zero_amd import zq

L = zq.lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000
MB = 0x100000
OK, NULL, SIZE, BLOCK, ALIGN, ALIAS, DTYPE = (zq.ZQ_OK, zq.ZQ_ERR_NULL, zq.ZQ_ERR_SIZE, zq.ZQ_ERR_BLOCK,
                                              zq.ZQ_ERR_ALIGN, zq.ZQ_ERR_ALIAS, zq.ZQ_ERR_DTYPE)
INF = float("inf")


def test_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "zq_train.h")) as f:
        names = set(re.findall(r"^(?:zq_status|size_t)\s+(zq_\w+)\s*\(", f.read(), re.M))
    assert names == {"zq_embed_lookup", "zq_embed_lookup_int8", "zq_embed_grad", "zq_embed_grad_workspace",
                     "zq_grad_sumsq_batched", "zq_grad_sumsq_workspace", "zq_grad_clip_batched"}
    for name in names:
        assert hasattr(L, name), name


def lookup(table=FAKE, tt=0, rows=10, dim=64, ids=FAKE + MB, it=1, n=4, out=FAKE + 2 * MB, ot=0):
    return L.zq_embed_lookup(table, tt, rows, dim, ids, it, n, 1.0, out, ot, None)


def test_lookup_refusals():
    for k in ({"tt": 3}, {"ot": -1}, {"it": 2}):
        assert lookup(**k) == DTYPE
    for k in ({"rows": 0}, {"dim": 0}, {"rows": 2 ** 31 - 1}, {"dim": 2 ** 31}, {"n": 2 ** 30 + 1},
              {"rows": 2 ** 30, "dim": 2 ** 30 + 1}, {"n": 2 ** 30, "dim": 2 ** 30 + 1}):
        assert lookup(**k) == SIZE
    assert lookup(n=0, table=None, ids=None, out=None) == OK
    for k in ("table", "ids", "out"):
        assert lookup(**{k: None}) == NULL
    assert lookup(table=FAKE + 8) == ALIGN
    assert lookup(ids=FAKE + MB + 4) == ALIGN
    assert lookup(ids=FAKE + MB + 2, it=0) == ALIGN
    assert lookup(out=FAKE + 2 * MB + 4) == ALIGN
    assert lookup(out=FAKE + 10 * 64 * 4 - 16) == ALIAS            # the table's last 16 bytes
    assert lookup(ids=FAKE + 2 * MB + 4 * 64 * 4 - 8) == ALIAS     # the output's last 8 bytes
    assert lookup(ids=FAKE + 2 * MB + 4 * 64 * 2 - 8, ot=1) == ALIAS


def lookup8(codes=FAKE, scales=FAKE + MB, block=128, rows=10, dim=64, ids=FAKE + 2 * MB, it=1, n=4,
            out=FAKE + 3 * MB, ot=1):
    return L.zq_embed_lookup_int8(codes, scales, block, rows, dim, ids, it, n, 1.0, out, ot, None)


def test_lookup_int8_refusals():
    assert lookup8(ot=7) == DTYPE and lookup8(it=-1) == DTYPE
    for b in (0, 16, 48, 8192):
        assert lookup8(block=b) == BLOCK
    assert lookup8(rows=0) == SIZE and lookup8(dim=0) == SIZE
    assert lookup8(n=0, codes=None, scales=None) == OK
    for k in ("codes", "scales", "ids", "out"):
        assert lookup8(**{k: None}) == NULL
    assert lookup8(codes=FAKE + 8) == ALIGN and lookup8(scales=FAKE + MB + 2) == ALIGN
    assert lookup8(out=FAKE + 624) == ALIAS
    assert lookup8(out=FAKE + MB) == ALIAS
    assert lookup8(scales=FAKE + 3 * MB + 508) == ALIAS            # 5 scales, the output's last 4 bytes


WS = 1 << 22


def grad(dout=FAKE, dt=1, ids=FAKE + MB, it=1, n=100, rows=10, dim=64, g=FAKE + 2 * MB, gt=0, mode=0, cb=0,
         ws=FAKE + 16 * MB, wb=WS):
    return L.zq_embed_grad(dout, dt, ids, it, n, rows, dim, 1.0, g, gt, mode, 1, cb, ws, wb, None)


def test_embed_grad_refusals():
    for k in ({"dt": 3}, {"gt": 9}, {"it": 5}, {"mode": 3}, {"mode": -1}, {"mode": 2, "gt": 0}, {"mode": 2, "gt": 2}):
        assert grad(**k) == DTYPE
    for k in ({"rows": 0}, {"dim": 0}, {"n": 2 ** 30 + 1}, {"rows": 2 ** 31 - 1}, {"dim": 2 ** 31},
              {"cb": 2 ** 64 - 600}, {"wb": 0},
              {"wb": L.zq_embed_grad_workspace(100, 10, 64) - 1}):
        assert grad(**k) == SIZE
    for m in (1, 2):
        assert grad(n=0, mode=m, gt=1, g=None, dout=None, ids=None, ws=None, wb=0) == OK
    assert grad(n=0, g=None) == NULL                               # the write mode clears grad
    assert grad(n=0, g=FAKE + 4) == ALIGN
    for k in ("dout", "ids", "g", "ws"):
        assert grad(**{k: None}) == NULL
    for k in ({"dout": FAKE + 2}, {"ids": FAKE + MB + 4}, {"ids": FAKE + MB + 2, "it": 0}, {"g": FAKE + 2 * MB + 8},
              {"ws": FAKE + 16 * MB + 8}):
        assert grad(**k) == ALIGN
    need = L.zq_embed_grad_workspace(100, 10, 64)
    assert grad(g=FAKE + 100 * 64 * 2 - 16) == ALIAS               # dout's end
    assert grad(ids=FAKE + 2 * MB + 10 * 64 * 4 - 8) == ALIAS      # grad's end
    assert grad(ws=FAKE + 2 * MB + 10 * 64 * 4 - 16) == ALIAS
    assert grad(ws=FAKE + 100 * 64 * 2 - 16) == ALIAS
    assert grad(ids=FAKE + 16 * MB + (need - 8) // 8 * 8) == ALIAS


def test_embed_grad_workspace():
    f = L.zq_embed_grad_workspace
    assert f(0, 10, 64) == 0 and f(5, 0, 64) == 0 and f(5, 10, 0) == 0 and f(2 ** 30 + 1, 10, 8) == 0
    # Keys and positions, and at most an eighth of an fp32 copy of dout (an
    # eighth only up to some 64 MB of it) for the partials of long runs.  A
    # workspace made for some number of tokens serves every smaller number.
    for dim in (1, 768, 4096, 2 ** 23):
        last = 0
        for n in sorted({1, 16, 17, 64, 65, 8192, 131072, 131073, 10 ** 6} | set(range(90, 140000, 997))):
            b = f(n, 32000, dim)
            assert last <= b
            assert 8 * n <= b <= 17 * n + 2 ** 20 + max(n * dim // 8 + 8 * dim + 64, 2 ** 26)
            last = b
    assert zq.embed_grad_workspace(100, 10, 64) == f(100, 10, 64)


def call(fn, segs, dt=0, n_seg=None, **k):
    arr = (zq.GradSegment * max(len(segs), 1))(*segs)
    p = C.cast(arr, C.c_void_p) if segs is not None else None
    n = len(segs) if n_seg is None else n_seg
    if fn == "sumsq":
        return L.zq_grad_sumsq_batched(p if not k.get("null") else None, n, dt, 0, k.get("sumsq", FAKE),
                                       k.get("ws", FAKE + MB), k.get("wb", 1 << 24), None)
    return L.zq_grad_clip_batched(p if not k.get("null") else None, n, dt, k.get("sumsq", FAKE),
                                  k.get("max_norm", 1.0), k.get("eps", 1e-6), k.get("norm", None), None)


def seg(g, n=1000, out=None):
    return zq.GradSegment(g, g if out is None else out, n)


G = FAKE + 64 * MB


def test_sumsq_refusals():
    ok = seg(G)
    assert call("sumsq", [ok], dt=3) == DTYPE
    assert call("sumsq", [ok], n_seg=65537) == SIZE
    assert call("sumsq", [seg(G, 2 ** 40 + 1)]) == SIZE
    assert call("sumsq", [seg(G, 2 ** 39), seg(G, 2 ** 39), seg(G, 1)]) == SIZE
    assert call("sumsq", [ok], wb=L.zq_grad_sumsq_workspace(1) - 1) == SIZE
    assert call("sumsq", [ok], null=True) == NULL
    assert call("sumsq", [ok], sumsq=None) == NULL and call("sumsq", [ok], ws=None) == NULL
    assert call("sumsq", [zq.GradSegment(None, None, 5)]) == NULL
    assert call("sumsq", [seg(G + 8)]) == ALIGN
    assert call("sumsq", [ok], sumsq=FAKE + 4) == ALIGN and call("sumsq", [ok], ws=FAKE + MB + 8) == ALIGN
    assert call("sumsq", [ok], sumsq=G + 3992) == ALIAS
    assert call("sumsq", [ok], ws=G + 3984) == ALIAS
    assert call("sumsq", [ok], sumsq=FAKE + MB + 16) == ALIAS
    assert L.zq_grad_sumsq_workspace(65537) == 0
    sizes = [L.zq_grad_sumsq_workspace(n) for n in (0, 1, 128, 129, 65536)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


def test_clip_refusals():
    ok = seg(G)
    assert call("clip", [ok], dt=-2) == DTYPE
    assert call("clip", [ok], n_seg=65537) == SIZE
    assert call("clip", [seg(G, 2 ** 40 + 1)]) == SIZE
    for bad in (-1.0, INF, float("nan")):
        assert call("clip", [ok], max_norm=bad) == SIZE
        assert call("clip", [ok], eps=bad) == SIZE
    assert call("clip", [ok], null=True) == NULL and call("clip", [ok], sumsq=None) == NULL
    assert call("clip", [zq.GradSegment(G, None, 5)]) == NULL
    assert call("clip", [zq.GradSegment(None, G, 5)]) == NULL
    assert call("clip", [seg(G + 8)]) == ALIGN and call("clip", [seg(G, out=G + MB + 4)]) == ALIGN
    assert call("clip", [ok], norm=FAKE + MB + 2) == ALIGN
    assert call("clip", [seg(G, out=G + 16)]) == ALIAS              # shifted onto itself
    assert call("clip", [ok, ok]) == ALIAS                          # clipped twice
    assert call("clip", [seg(G, out=G + MB), seg(G + MB, out=G + 2 * MB)]) == ALIAS
    assert call("clip", [ok], norm=G + 8) == ALIAS
    assert call("clip", [ok], sumsq=G) == ALIAS
    assert call("clip", [ok], norm=FAKE + 4) == ALIAS               # over sumsq


def test_binding_refusals():
    cpu = torch.zeros(4, 8)
    ids = torch.zeros(2, dtype=torch.int64)
    out = torch.zeros(2, 8)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="table must be a GPU tensor"):
        zq.zq_embed_lookup(cpu, ids, 1.0, out)
    with pytest.raises(ValueError, match="two dimensions"):
        zq.zq_embed_lookup(cpu.reshape(-1), ids, 1.0, out)
    with pytest.raises(ValueError, match="codes must be a GPU tensor"):
        zq.zq_embed_lookup_int8(cpu.to(torch.int8), torch.zeros(1), 32, ids, 1.0, out)
    with pytest.raises(ValueError, match="dout must be a GPU tensor"):
        zq.zq_embed_grad(out, ids, 1.0, cpu, zq.ZQ_GRAD_WRITE, ws)
    with pytest.raises(ValueError, match="two dimensions"):
        zq.zq_embed_grad(out, ids, 1.0, cpu.reshape(-1), zq.ZQ_GRAD_WRITE, ws)
    with pytest.raises(ValueError, match="g must be a GPU tensor"):
        zq.zq_grad_sumsq_batched([(cpu, None)], torch.zeros(1, dtype=torch.float64), ws)


def test_header_is_c99_and_the_library_links_from_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    src = tmp_path / "use_zq_train.c"
    src.write_text(r'''
#include <stdio.h>
#include "zq_train.h"
int main(void) {
    zq_grad_segment s = {NULL, NULL, 5};
    double q = 0;
    if (zq_embed_grad_workspace(0, 10, 10) != 0 || zq_embed_grad_workspace(7, 10, 10) == 0) return 1;
    if (zq_grad_sumsq_workspace(3) == 0) return 2;
    if (zq_embed_lookup(NULL, ZQ_BF16, 5, 8, NULL, ZQ_I32, 3, 1.0f, NULL, ZQ_FP32, NULL) != ZQ_ERR_NULL) return 3;
    if (zq_embed_grad(NULL, ZQ_BF16, NULL, ZQ_I64, 3, 5, 8, 1.0f, NULL, ZQ_FP32, ZQ_GRAD_ADD_SR, 0, 0, NULL, 0,
                      NULL) != ZQ_ERR_DTYPE) return 4;
    if (zq_grad_clip_batched(&s, 1, ZQ_FP16, &q, 1.0f, 0.0f, NULL, NULL) != ZQ_ERR_NULL) return 5;
    puts("ok");
    return 0;
}
''')
    exe = tmp_path / "use_zq_train"
    lib = os.path.join(ROOT, "weight_communication_zero_amd", "libzq.so")
    r = subprocess.run([gcc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), lib, "-Wl,-rpath," + os.path.dirname(lib), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
