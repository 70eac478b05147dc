"""The vocabulary projection's cross entropy where its values are extreme, on the
GPU, against its formula in 64 bits.

What the tolerances count (2^-24 is half a step of binary32 relative to the value):
  a sum of K products of 16-bit operands  (K + 8) 2^-24 times the sum of their sizes,
          the worst order; the scale's product 2^-24 of the logit more
  lse     what the logits are off by, and 2^-23 (64 + V / 2048 + |lse|) for the
          exponentials and their sum
"""
import math

import pytest
import torch

from weight_communication_zero_amd import zq

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16}
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def near(got, want, bound, what=""):
    got, want = got.double(), want.double()
    fine = want.isfinite()
    assert torch.equal(fine, got.isfinite()), what + ": another set of finite values"
    assert torch.equal(want.isnan(), got.isnan()), what + ": NaN elsewhere"
    inf = want.isinf()
    assert torch.equal(want[inf], got[inf]), what + ": infinities"
    bound = torch.as_tensor(bound, dtype=torch.float64, device="cuda").expand(want.shape)
    off = ((got - want).abs() - bound)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, (what, float(off.max()), float((got - want).abs()[fine].max()))


def ce_loss(x, w, ids, scale=1.0, piece=0):
    n, (rows, d) = ids.numel(), w.shape
    loss, lse = (torch.full((n,), 77.0, device="cuda") for _ in range(2))
    ws = torch.full((zq.ce_loss_workspace(n, rows, d, piece),), 0xFF, dtype=torch.uint8, device="cuda")
    zq.zq_ce_loss(x, w, ids, scale, loss, lse, ws, piece=piece)
    return loss, lse


def ce_grad(x, w, ids, scale, lse, dloss, piece=0):
    n, (rows, d) = ids.numel(), w.shape
    dx, dw = torch.full_like(x, 77.0), torch.full((rows, d), 77.0, device="cuda")
    ws = torch.full((zq.ce_grad_workspace(n, rows, d, piece),), 0xFF, dtype=torch.uint8, device="cuda")
    zq.zq_ce_grad(x, w, ids, scale, lse, dloss, dx, dw, zq.ZQ_GRAD_WRITE, ws, piece=piece)
    return dx, dw


def some_ids(n, rows, seed):
    return torch.randint(0, rows, (n,), generator=gen(seed), device="cuda")


# Few tokens take small tiles, some hundred and many the larger ones; no vocabulary here is whole tiles.
@pytest.mark.parametrize("n,rows", [(5, 257), (300, 999), (700, 50257), (3, 1), (700, 8191)])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_a_scale_of_zero_gives_equal_logits(n, rows, scale):
    x, w = randn((n, 64), 1, torch.bfloat16), randn((rows, 64), 2, torch.bfloat16)
    ids = some_ids(n, rows, 3)
    for piece in (0, 256):
        loss, lse = ce_loss(x, w, ids, scale, piece)
        want = torch.full((n,), math.log(rows), dtype=torch.float64, device="cuda")
        bound = 2.0 ** -23 * (64 + rows / 2048 + math.log(rows))
        near(lse, want, bound, "lse")
        near(loss, want, bound, "loss")
    dx, dw = ce_grad(x, w, ids, scale, lse, randn((n,), 4), piece)
    assert not bool((dx != 0).any()) and not bool((dw != 0).any())


def test_a_scale_of_zero_and_infinite_sums():
    """0 times an infinity is NaN, as the formula has it."""
    x, w = randn((40, 64), 1, torch.bfloat16).abs(), randn((300, 64), 2, torch.bfloat16)
    x[3, 0], w[7, 0] = INF, 1.0
    loss, lse = ce_loss(x, w, some_ids(40, 300, 3), 0.0)
    bad = torch.arange(40, device="cuda") == 3
    assert torch.equal(lse.isnan(), bad) and torch.equal(loss.isnan(), bad)


@pytest.mark.parametrize("scale", [2.0 ** -140, 1e-30, 0.3, -1e30])
def test_far_scales(scale):
    """Logits of ordinary size (of none, with a scale of no normal size) from scales far from 1."""
    n, d, rows = 70, 64, 999
    size = 2.0 ** 16 if abs(scale) < 1e-20 else 1.0 if abs(scale) < 1 else 2.0 ** -48
    x, w = randn((n, d), 1, torch.bfloat16, size), randn((rows, d), 2, torch.bfloat16, size * 0.1)
    ids = some_ids(n, rows, 3)
    loss, lse = ce_loss(x, w, ids, scale)
    z = x.double() @ w.double().t() * float(torch.tensor(scale))
    off = (d + 16) * 2.0 ** -24 * abs(scale) * (x.double().abs() @ w.double().abs().t())
    bound = off.max(1).values + 2.0 ** -23 * (64 + z.abs().max(1).values)
    want = torch.logsumexp(z, 1)
    near(lse, want, bound, "lse")
    near(loss, want - z.gather(1, ids[:, None])[:, 0], 2 * bound, "loss")


@pytest.mark.parametrize("scale", [1.0, -2.0, 0.3])
@pytest.mark.parametrize("size", [1e10, 1e20, 1e37])
@pytest.mark.parametrize("n,rows", [(5, 257), (300, 999), (700, 5000)])
def test_huge_finite_logits(n, rows, size, scale):
    """Half a unit in the last place of such a logit is an exponent of its own; sums go up to some 10^38."""
    x, w = randn((n, 64), 1, torch.bfloat16, 0.1 * size ** 0.5), randn((rows, 64), 2, torch.bfloat16, size ** 0.5)
    ids = some_ids(n, rows, 3)
    z = x.double() @ w.double().t() * float(torch.tensor(scale))
    off = (64 + 16) * 2.0 ** -24 * abs(scale) * (x.double().abs() @ w.double().abs().t()).max(1).values
    want = torch.logsumexp(z, 1)
    for piece in (0, 512):
        loss, lse = ce_loss(x, w, ids, scale, piece)
        near(lse, want, off + 2.0 ** -23 * (64 + want.abs()), "lse")
        near(loss, want - z.gather(1, ids[:, None])[:, 0], 2 * off + 2.0 ** -22 * (64 + want.abs()), "loss")
