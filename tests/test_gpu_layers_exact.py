"""Weight gradients of the most tokens, and operands beyond 4 GiB, with inputs for which
every sum is exact in binary32, so that a lost, doubled or misplaced row shows in any
element.

The operands are whole numbers (times a power of two) whose sums stay below 2^24.  In the
cross entropy that power is 2^30: logits differ by 2^30 or not at all, so each
probability is 0 or 1, lse is the largest logit, and with loss gradients of +-1 q is
-1, 0 or 1 (or 2 steps of a tie) in 16 bits.
"""
import pytest
import torch

from weight_communication_zero_amd import zq

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(shape, most, seed, dtype=BF, factor=1.0):
    return (torch.randint(-most, most + 1, shape, generator=gen(seed), device="cuda").float() * factor).to(dtype)


def workspace(size):
    return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("n,o,i", [(1 << 20, 9, 16), ((1 << 20) - 5, 130, 70), (300001, 264, 24)])
def test_linear_grad_of_the_most_tokens(n, o, i):
    """The sum of the sizes is below 7 2^20 halves."""
    dy, codes = whole((n, o), 1, 1), whole((n, i), 7, 2, torch.int8)
    block = 4096
    scales = torch.full((-(-n * i // block),), 0.5, device="cuda")
    want = torch.zeros(o, i, dtype=torch.float64, device="cuda")
    for k in range(0, n, 1 << 17):
        want += dy[k:k + (1 << 17)].double().t().contiguous() @ codes[k:k + (1 << 17)].double() * 0.5
    ws = workspace(zq.linear_grad_workspace(n, o, i))
    for mode in (zq.ZQ_GRAD_WRITE, zq.ZQ_GRAD_ADD):
        grad = torch.full((o, i), 3.0, device="cuda")
        zq.zq_linear_grad_int8(dy, codes, scales, block, grad, mode, ws)
        assert torch.equal(grad.double(), want + (3.0 if mode == zq.ZQ_GRAD_ADD else 0.0))
    assert float(want.abs().max()) > 1000


def step(x, w, ids, dloss, dw_dtype):
    n, (rows, d) = ids.numel(), w.shape
    loss, lse = (torch.full((n,), 77.0, device="cuda") for _ in range(2))
    ws = workspace(zq.ce_loss_workspace(n, rows, d))
    zq.zq_ce_loss(x, w, ids, 1.0, loss, lse, ws)
    del ws
    dx, dw = torch.full_like(x, 77.0), torch.full((rows, d), 77.0, dtype=dw_dtype, device="cuda")
    ws = workspace(zq.ce_grad_workspace(n, rows, d))
    zq.zq_ce_grad(x, w, ids, 1.0, lse, dloss, dx, dw, zq.ZQ_GRAD_WRITE, ws)
    return loss, lse, dx, dw


def check_loss(loss, lse, z, ids):
    """z: exact logits.  Where the target ties with the largest the loss is the logarithm
    of a small whole number, otherwise a difference that is exact."""
    top = z.max(1, keepdim=True).values
    ties = (z == top).sum(1).double()
    assert torch.equal(lse.double(), top[:, 0])
    want = (top - z.gather(1, ids[:, None]))[:, 0]
    assert torch.equal(loss.double()[want > 0], want[want > 0])
    assert bool(((loss.double() - ties.log()).abs()[want == 0] <= 2.0 ** -20).all())


def probabilities(z, lse, ids, dloss):
    q = torch.exp(z - lse.double()[:, None])
    assert bool(((q == 0) | (q == 1)).all())
    q.scatter_add_(1, ids[:, None], torch.full_like(q[:, :1], -1.0))
    return q * dloss.double()[:, None]


@pytest.mark.parametrize("pad", [0, 10, 60, 99])
def test_ce_of_the_most_tokens(pad):
    """Of dw the sum of the sizes is below 2^20 times 2 times 7."""
    n, d, rows = 1 << 20, 8, 5
    x, w = whole((n, d), 7, 1, factor=2.0 ** 14), whole((rows, d), 4, 2, factor=2.0 ** 16)
    ids = torch.randint(0, rows, (n,), generator=gen(3), device="cuda")
    z = x.double() @ w.double().t()
    # (Where the largest logit is 0, the logarithm of its ties would be seen in lse.)
    there = (torch.rand(n, generator=gen(4), device="cuda") * 100 >= pad) & (z.max(1).values != 0)
    dloss = whole((n,), 1, 5, torch.float32)
    loss, lse, dx, dw = step(x, w, torch.where(there, ids, -1), dloss, torch.float32)
    z = z[there]
    assert not bool(loss[~there].any()) and not bool(lse[~there].any()) and not bool(dx[~there].any())
    check_loss(loss[there], lse[there], z, ids[there])
    q = probabilities(z, lse[there], ids[there], dloss[there])
    assert torch.equal(dx[there], (q @ w.double()).to(BF))
    want = q.t().contiguous() @ x[there].double()
    assert torch.equal(dw.double(), want)
    assert float(want.abs().max()) > 2.0 ** 14 * 10


def rows_in_pieces(big, small):
    """small @ big^T in 64 bits, big in pieces of rows."""
    return torch.cat([small.double() @ big[i:i + 8192].double().t() for i in range(0, big.shape[0], 8192)], 1)


def test_ce_of_hidden_states_beyond_4_gib():
    n, d, rows = 140000, 16384, 64                 # row 131072 starts at 2^32 bytes
    x = torch.empty(n, d, dtype=BF, device="cuda")
    for i in range(0, n, 10000):
        x[i:i + 10000] = whole((10000, d), 2, 100 + i, factor=2.0 ** 14)
    w = whole((rows, d), 4, 2, factor=2.0 ** 16)
    ids = torch.randint(0, rows, (n,), generator=gen(3), device="cuda")
    dloss = whole((n,), 1, 5, torch.float32)
    loss, lse, dx, dw = step(x, w, ids, dloss, torch.float32)
    want = torch.zeros(rows, d, dtype=torch.float64, device="cuda")
    for i in range(0, n, 10000):
        s = slice(i, i + 10000)
        xs = x[s].double()
        z = xs @ w.double().t()
        check_loss(loss[s], lse[s], z, ids[s])
        q = probabilities(z, lse[s], ids[s], dloss[s])
        assert torch.equal(dx[s], (q @ w.double()).to(BF)), i
        want += q.t().contiguous() @ xs
    assert torch.equal(dw.double(), want)


def test_ce_of_a_projection_beyond_4_gib():
    n, d, rows = 64, 16384, 140000                 # row 131072 starts at 2^32 bytes
    w = torch.empty(rows, d, dtype=BF, device="cuda")
    for i in range(0, rows, 10000):
        w[i:i + 10000] = whole((10000, d), 4, 100 + i, factor=2.0 ** 16)
    # Half of the targets past the border; three tokens of four lean to their target (or to
    # the row 8928 before it, or to a far row), which then is the largest logit.
    k = torch.arange(n, device="cuda")
    ids = torch.where(k % 2 == 0, 131072 + 139 * k % 8928, torch.randint(0, rows, (n,), generator=gen(3), device="cuda"))
    near = torch.stack([ids, ids - 8928, 139999 - 7 * k, ids])[k % 4, k].clamp(min=0)
    lean = (k % 4 != 3).to(BF)[:, None]
    x = whole((n, d), 2, 1, factor=2.0 ** 14) + w[near] * 2.0 ** -2 * lean
    dloss = torch.where(k % 3 == 0, -1.0, 1.0)
    loss, lse, dx, dw = step(x, w, ids, dloss, torch.float32)
    z = rows_in_pieces(w, x)
    check_loss(loss, lse, z, ids)
    q = probabilities(z, lse, ids, dloss)
    want = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 8192):
        s = slice(i, i + 8192)
        want += q[:, s].contiguous() @ w[s].double()
        assert torch.equal(dw[s].double(), q[:, s].t().contiguous() @ x.double()), i
    assert torch.equal(dx, want.to(BF))
    assert int((z.argmax(1) >= 131072).sum()) > 16
