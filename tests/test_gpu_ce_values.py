"""The vocabulary projection's cross entropy where its values are extreme, on the
GPU, against its formula in 64 bits.

What the tolerances count (2^-24 is half a step of binary32 relative to the value):
  a sum of K products of 16-bit operands  (K + 8) 2^-24 times the sum of their sizes,
          the worst order; the scale's product 2^-24 of the logit more
  lse     what the logits are off by, and 2^-23 (64 + V / 2048 + |lse|) for the
          exponentials and their sum
  loss    relative, at the tests that count it
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


def exact_operands(n, d, rows, dtype, seed, sign):
    """Whole numbers, so that every sum is exact: rows of w in -4 .. 4, hidden states that
    lean to their token by 0, 1, 2 or 3 times its row (sign -1: away from it)."""
    w = torch.randint(-4, 5, (rows, d), generator=gen(seed), device="cuda")
    ids = some_ids(n, rows, seed + 1)
    lean = torch.arange(n, device="cuda")[:, None] % 4 * sign
    x = torch.randint(-2, 3, (n, d), generator=gen(seed + 2), device="cuda") + lean * w[ids]
    return x.to(T[dtype]), w.to(T[dtype]), ids


@pytest.mark.parametrize("dtype,scale", [("bf16", 2.0 ** -6), ("fp16", 0.02), ("bf16", -0.02)])
@pytest.mark.parametrize("n,rows", [(1, 2), (7, 1000), (300, 999), (300, 50257), (700, 2), (700, 8191)])
def test_losses_of_sure_tokens_keep_their_digits(n, rows, dtype, scale):
    """loss = log1p(X), X the sum over j != t of exp(z_j - z_t), M the largest z but z_t.  An
    exponent z_j - M or M - z_t in base 2 has a difference's rounding, the factor's two and
    the product's, 2^-24 each, and the exponential itself 2^-23: X is off by those of its
    terms and by 2^-23 (64 + V / 2048) of itself for the sum, the loss by that over 1 + X
    and 2^-22 of itself for the last steps.  A term below 2^-126 may vanish."""
    sure = 0
    for seed in (10, 20):
        x, w, ids = exact_operands(n, 128, rows, dtype, seed, 1 if scale > 0 else -1)
        if n == 1:
            x = (x + 3 * math.copysign(1, scale) * w[ids]).to(x.dtype)
        z = x.double() @ w.double().t() * float(torch.tensor(scale))
        t = z.gather(1, ids[:, None])
        others = z.scatter(1, ids[:, None], -INF)
        top = others.max(1, keepdim=True).values
        e = torch.exp(others - t)
        total = e.sum(1)
        e = torch.where(e > 0, e * ((others - top).abs() + (top - t).abs() + 2), 0.0)
        want = torch.log1p(total)
        bound = 2.0 ** -22 * e.sum(1) + 2.0 ** -23 * (64 + rows / 2048) * total + rows * 2.0 ** -126
        bound = bound / (1 + total) + 2.0 ** -22 * want
        assert bool((bound < 2e-4 * want + 1e-30).all())
        sure += int((want < 1e-3).sum())
        for piece in (0, 512):
            loss, lse = ce_loss(x, w, ids, scale, piece)
            assert bool((loss >= 0).all())
            near(loss, want, bound, "loss")
            near(lse, torch.logsumexp(z, 1), bound + 2.0 ** -23 * (1 + z.abs().max(1).values), "lse")
    assert sure > 0


def test_a_token_that_has_the_vocabulary_to_itself():
    x, w, ids = randn((9, 64), 1, torch.bfloat16), randn((1, 64), 2, torch.bfloat16), some_ids(9, 1, 3)
    loss, lse = ce_loss(x, w, ids)
    z = (x.double() @ w.double().t())[:, 0]
    assert not bool(loss.view(torch.int32).any())
    near(lse, z, 80 * 2.0 ** -24 * (x.double().abs() @ w.double().abs().t())[:, 0])


@pytest.mark.parametrize("piece", [0, 256])
def test_infinite_and_nan_logits_of_targets_and_others(piece):
    """Each token has its own mixture: an infinity (of either sign) or NaN at its target,
    at another row, at both, everywhere else."""
    rows, n = 700, 12
    w = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(n, rows, dtype=torch.float64, device="cuda")
    ids = torch.full((n,), 300, device="cuda")
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[300] = False
    one = torch.zeros(rows, dtype=torch.bool, device="cuda")
    one[600] = True
    plan = [(~rest, INF), (~rest, -INF), (~rest, NAN), (one, INF), (one, -INF), (one, NAN), (rest, -INF), (rest, INF),
            (~rest | one, INF), (~rest | one, -INF), (rest | ~rest, -INF), (~rest, 0.0)]
    for t, (where, value) in enumerate(plan):
        # Token t reads column t of w alone: 0 but where its value stands.
        x[t] = 0
        w[where, t] = 2.0 ** 100 if value == INF else -2.0 ** 100 if value == -INF else value
        z[t, where] = value
    # 2^100 times 2^100 is infinite; NaN stands in w, where all tokens meet it: its token comes apart.
    for t in range(n):
        ww = torch.zeros_like(w)
        ww[:, t] = w[:, t]
        xx = torch.zeros_like(x)
        xx[t, t] = 2.0 ** 100
        loss, lse = ce_loss(xx, ww, ids, 1.0, piece)
        want = torch.logsumexp(z[t], 0)
        near(lse[t:t + 1], want[None], 2.0 ** -16, f"lse {t}")
        near(loss[t:t + 1], (want - z[t, 300])[None], 2.0 ** -16, f"loss {t}")


@pytest.mark.parametrize("scale", [1.0, -0.3])
@pytest.mark.parametrize("n,rows", [(7, 257), (300, 1500)])
def test_gradient_at_huge_finite_logits(n, rows, scale):
    """Sums are exact (whole numbers times 2^30), lse is the largest logit rounded once: every
    probability is 1 or 0, and with loss gradients that are powers of two every q is exact.
    dx then rounds once, dw (fp32) not at all."""
    x, w, ids = exact_operands(n, 64, rows, "bf16", 5, 1 if scale > 0 else -1)
    ids = torch.where(torch.arange(n, device="cuda") % 3 == 0, some_ids(n, rows, 9), ids)
    x, w = (x.float() * 2 ** 14).bfloat16(), (w.float() * 2 ** 16).bfloat16()
    z = (x.double() @ w.double().t() * float(torch.tensor(scale))).float()
    lse = z.max(1).values
    got_lse = ce_loss(x, w, ids, scale)[1]
    top = z.double().topk(2, 1).values
    single = top[:, 0] - top[:, 1] > 0
    near(got_lse[single], lse[single], 0.0, "lse")
    dloss = torch.tensor([1.0, -0.5, 0.25], device="cuda")[torch.arange(n, device="cuda") % 3]
    for piece in (0, 256):
        dx, dw = ce_grad(x, w, ids, scale, lse, dloss, piece)
        q = torch.exp(z.double() - lse[:, None].double())
        assert bool(((q == 0) | (q == 1)).all())
        q.scatter_add_(1, ids[:, None], torch.full_like(q[:, :1], -1.0))
        q *= dloss[:, None].double()
        want = q @ w.double() * float(torch.tensor(scale))
        near(dx, want, (2.0 ** -8 + 2.0 ** -22) * want.abs(), "dx")
        want = q.t() @ x.double() * float(torch.tensor(scale))
        near(dw, want, 2.0 ** -22 * want.abs(), "dw")
