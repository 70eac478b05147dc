"""The host side of the layer calls' launches (pieces, tiles, splits, the workspace's
parts, grids) for some 20,000 sizes up to the accepted ones, under AddressSanitizer
and UndefinedBehaviorSanitizer, with a stub in place of the launch that checks what
each kernel is handed.  Builds with a planted mistake in a layout, and with a planted
out-of-bounds read, must fail.  Every sanitizer flag on a hipcc line sits behind
-Xarch_host."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_communication_zero_amd", "csrc")
DRIVER = os.path.join(ROOT, "tests", "sanitize", "layers_plan_driver.cpp")
HIPCC = "/opt/rocm/bin/hipcc"
CLANGXX = "/opt/rocm/llvm/bin/clang++"


def _run(tmp_path, part, driver=DRIVER, flags=()):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)):
        pytest.skip("hipcc / clang++ not installed")
    obj, exe = str(tmp_path / "plan.o"), str(tmp_path / "plan")
    for cmd in ([HIPCC, "--cuda-host-only", "-O1", "-g", "-std=c++17", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
                 "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                 f"-I{os.path.join(ROOT, 'include')}", f"-DPART={part}", *flags, "-c", "-o", obj, "-x", "hip", driver],
                # (The kernels' device code, which the registration names, is not there.)
                [CLANGXX, "-fsanitize=address,undefined", "-Wl,--unresolved-symbols=ignore-all", "-o", exe, obj]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
    return subprocess.run([exe], capture_output=True, text=True, timeout=600)


@pytest.mark.parametrize("part", [0, 1, 2])
def test_launches_stay_in_their_buffers(tmp_path, part):
    r = _run(tmp_path, part)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr[-4000:]
    assert "runtime error" not in r.stderr


def test_a_planted_read_past_the_end_aborts(tmp_path):
    r = _run(tmp_path, 0, flags=["-DZQ_SANITIZER_CANARY"])
    assert r.returncode != 0 and "Sanitizer" in r.stderr


@pytest.mark.parametrize("part,file,old,new", [
    (0, "zq_linear_grad.hip", "n_tok * l.ldx * 2", "n_tok * in_dim * 2"),
    (0, "zq_mm_plan.h", "* M * round_up(N, 4)", "* M * N"),
    (1, "zq_ce_loss.hip", "div_up(l.piece, tile_cols(l.logits.kind)) * n_pad * 8", "l.piece / 256 * n_pad * 8"),
    (1, "zq_ce.h", "l.w = take(l.piece * l.kp * 2)", "l.w = take(l.piece * (l.kp - 32) * 2)"),
    (2, "zq_ce_grad.hip", "(uint64_t)n_tok * l.piece * 2 * l.parts", "(uint64_t)n_tok * l.piece * 2"),
    (2, "zq_ce_grad.hip", "for (uint32_t n : {l.piece, l.rows_of(l.n_pieces - 1, rows)})", "for (uint32_t n : {l.piece})"),
])
def test_a_planted_mistake_in_a_layout_is_found(tmp_path, part, file, old, new):
    """The planted copy lies in a folder of its own; no kernel of it is ever run."""
    src = tmp_path / "weight_communication_zero_amd" / "csrc"
    src.mkdir(parents=True)
    for name in os.listdir(CSRC):
        if name.startswith("zq_") and name.endswith((".h", ".hip")):
            with open(os.path.join(CSRC, name)) as f:
                text = f.read()
            if name == file:
                assert text.count(old) == 1
                text = text.replace(old, new)
            (src / name).write_text(text)
    os.symlink(os.path.join(ROOT, "include"), tmp_path / "include")
    (tmp_path / "tests" / "sanitize").mkdir(parents=True)
    driver = tmp_path / "tests" / "sanitize" / "layers_plan_driver.cpp"
    with open(DRIVER) as f:
        driver.write_text(f.read())
    r = _run(tmp_path, part, driver=str(driver))
    assert r.returncode == 1 and "do not lie in" in r.stderr, r.stdout + r.stderr[-2000:]
