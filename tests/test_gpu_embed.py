"""Embedding lookup and its gradient on the GPU.

Lookups are compared bit for bit with the formula's binary32 products on the
host.  Gradients are compared with sums in 64 bits: a binary32 sum of L terms
x, times a scale, added to an old value, is off by at most
    (L + 3) 2^-24 (|scale| sum|x| + |old|)
to first order (L - 1 additions, the product, the addition; one more covers
the second order), and rounding to a 16-bit type adds half a step of the
result, eps / 2, or half its smallest subnormal.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from weight_communication_zero_amd import zq

pytestmark = pytest.mark.gpu

T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"fp32": 2.0 ** -150, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half the smallest subnormal
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def guarded(shape, dtype, fill=float("nan")):
    """A view of `shape` followed by canaries, and the function that checks them."""
    n = math.prod(shape)
    buf = torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")
    buf[n:] = 7
    return buf[:n].view(shape), lambda: bool((buf[n:] == 7).all())


def same(got, exp):
    """Equal values, NaN for NaN, and equal signs of zeros."""
    got, exp = got.cpu(), exp.cpu()
    ok = (got == exp) & (torch.signbit(got) == torch.signbit(exp))
    return bool((ok | (got.isnan() & exp.isnan())).all())


def expect_lookup(table32, ids, scale, dtype):
    ids = ids.cpu().long().reshape(-1)
    there = (ids >= 0) & (ids < table32.shape[0])
    w = table32[torch.where(there, ids, 0)] * torch.tensor(scale, dtype=torch.float32)
    return torch.where(there[:, None], w, torch.zeros(())).to(dtype)


def make_ids(n, rows, dtype, seed, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((n,), rows - 1, dtype=dtype)
    if kind == "none":
        return torch.tensor([-1, rows, -(2 ** 31), 2 ** 31 - 1])[torch.randint(0, 4, (n,), generator=g)].to(dtype)
    if kind == "distinct":
        return torch.randperm(rows, generator=g)[:n].to(dtype)
    u = torch.rand(n, generator=g, dtype=torch.float64)
    ids = ((rows + 1.0) ** u).long().sub_(1).clamp_(0, rows - 1)
    ids = (ids * 7919 + 13) % rows
    if kind == "mixed":
        bad = torch.rand(n, generator=g)
        ids = torch.where(bad < 0.05, -1, ids)
        ids = torch.where(bad > 0.97, rows, ids)
    return ids.to(dtype)


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("table", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,dim,n", [(1, 1, 1), (7, 8, 3), (50, 17, 33), (300, 768, 100), (129, 1001, 65),
                                        (64, 513, 8), (33, 4096, 5)])
def test_lookup(table, out, rows, dim, n):
    g = torch.Generator().manual_seed(rows * dim + n)
    w = torch.randn(rows, dim, generator=g).to(T[table])
    for it, scale in ((torch.int64, math.sqrt(dim)), (torch.int32, -0.37)):
        ids = make_ids(n, rows, it, n)
        res, intact = guarded((n, dim), T[out])
        zq.zq_embed_lookup(w.cuda(), ids.cuda(), scale, res)
        assert same(res, expect_lookup(w.float(), ids, scale, T[out]))
        assert intact()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("table", ["int8", "fp32", "bf16", "fp16"])
def test_lookup_every_remainder(table, out):
    """Widths of every remainder: groups that start at any element, last groups
    of every length."""
    g = torch.Generator().manual_seed(5)
    ids = make_ids(37, 9, torch.int64, 6)
    for dim in list(range(1, 18)) + list(range(505, 522)):
        res, intact = guarded((37, dim), T[out])
        if table == "int8":
            codes = torch.randint(-128, 128, (9, dim), generator=g, dtype=torch.int8)
            scales = torch.rand(-(-9 * dim // 32), generator=g)
            w = torch.from_numpy(O.dequant_int8(codes.numpy().reshape(-1), scales.numpy(), 32)).view(9, dim)
            zq.zq_embed_lookup_int8(codes.cuda(), scales.cuda(), 32, ids.cuda(), 1.5, res)
        else:
            w = torch.randn(9, dim, generator=g).to(T[table])
            zq.zq_embed_lookup(w.cuda(), ids.cuda(), 1.5, res)
        assert same(res, expect_lookup(w.float(), ids, 1.5, T[out])) and intact(), dim


def test_lookup_special_values():
    """Infinities, NaN, signed zeros, subnormals and results past fp16's range."""
    v = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1e-42, -3e-39, 1e30, 70000.0, 65519.0, 1e-8, 6e-8])
    w = v.repeat(3).reshape(3, 12)
    ids = torch.tensor([2, 5, 0, -1, 2 ** 40, -(2 ** 63)])
    for out in T.values():
        for scale in (1.0, 3.0, 0.0, math.inf):
            res, intact = guarded((6, 12), out)
            zq.zq_embed_lookup(w.cuda(), ids.cuda(), scale, res)
            assert same(res, expect_lookup(w, ids, scale, out)) and intact()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,dim,n,block", [(1, 1, 1, 32), (40, 24, 50, 32), (77, 33, 41, 64), (50, 768, 60, 2048),
                                              (31, 1001, 20, 4096), (20, 4096, 9, 128), (300, 5, 300, 32)])
def test_lookup_int8(out, rows, dim, n, block):
    """Equal to the oracle's dequantization of the whole table, then the lookup."""
    rng = np.random.default_rng(rows + dim)
    codes = rng.integers(-128, 128, size=rows * dim).astype(np.int8)
    scales = (rng.random(-(-rows * dim // block)) * 1e-2).astype(np.float32)
    w = torch.from_numpy(O.dequant_int8(codes, scales, block)).reshape(rows, dim)
    for it in (torch.int64, torch.int32):
        ids = make_ids(n, rows, it, n)
        res, intact = guarded((n, dim), T[out])
        zq.zq_embed_lookup_int8(torch.from_numpy(codes).reshape(rows, dim).cuda(), torch.from_numpy(scales).cuda(),
                                block, ids.cuda(), 1.7, res)
        assert same(res, expect_lookup(w, ids, 1.7, T[out])) and intact()


def test_lookup_many_tokens():
    """Waves past the first workgroups, ids of two dimensions."""
    w = torch.randn(500, 136, device="cuda").bfloat16()
    ids = torch.randint(-3, 503, (70, 333), device="cuda")
    res = torch.empty(70, 333, 136, device="cuda")
    zq.zq_embed_lookup(w, ids, 2.0, res)
    assert same(res.reshape(-1, 136), expect_lookup(w.float().cpu(), ids, 2.0, torch.float32))


def check_grad(dout, ids, scale, old, got, mode, gt):
    """`got` against the sums in 64 bits (the bound in this file's header), on
    the device that dout is on."""
    rows, dim = old.shape
    dev = dout.device
    dout, ids, got, old = dout.double(), ids.to(dev).long().reshape(-1), got.to(dev), old.to(dev)
    there = (ids >= 0) & (ids < rows)
    zero = torch.zeros(rows, dim, dtype=torch.float64, device=dev)
    s = zero.index_add(0, ids[there], dout[there])
    a = zero.index_add(0, ids[there], dout[there].abs())
    count = torch.bincount(ids[there], minlength=rows).double()[:, None]
    base = zero if mode == zq.ZQ_GRAD_WRITE else old.double()
    scale = float(np.float32(scale))
    exact = base + scale * s
    bound = (count + 3) * 2.0 ** -24 * (abs(scale) * a + base.abs()) + TINY[gt]
    eps = torch.finfo(T[gt]).eps
    if gt != "fp32":
        # Half a step, or a whole one where the rounding is stochastic.
        step = eps if mode == zq.ZQ_GRAD_ADD_SR else eps / 2
        bound = bound + step * (exact.abs() + bound) + TINY[gt]
    err = (got.double() - exact).abs()
    bad = (err > bound).nonzero()
    assert bad.numel() == 0, (bad[0].tolist(), got[tuple(bad[0])].item(), exact[tuple(bad[0])].item(),
                              bound[tuple(bad[0])].item(), len(bad))
    untouched = count[:, 0] == 0
    exp = torch.zeros_like(old) if mode == zq.ZQ_GRAD_WRITE else old
    assert same(got[untouched], exp[untouched])


def run_grad(dout, ids, scale, old, mode, seed=0, base=0, stream=None):
    rows, dim = old.shape
    n = rows * dim
    buf = torch.empty(n + GUARD, dtype=old.dtype, device="cuda")
    buf[n:] = 7
    grad = buf[:n].view(rows, dim)
    grad.copy_(torch.full_like(old, math.nan) if mode == zq.ZQ_GRAD_WRITE else old)
    need = zq.embed_grad_workspace(ids.numel(), rows, dim)
    ws = torch.full((need + GUARD,), 0xAB, dtype=torch.uint8, device="cuda")
    zq.zq_embed_grad(dout.cuda(), ids.cuda(), scale, grad, mode, ws[:need], seed=seed, counter_base=base)
    assert bool((buf[n:] == 7).all()) and bool((ws[need:] == 0xAB).all())
    return grad


MODES = [("write", t) for t in T] + [("add", t) for t in T] + [("add_sr", "bf16")]
MODE = {"write": zq.ZQ_GRAD_WRITE, "add": zq.ZQ_GRAD_ADD, "add_sr": zq.ZQ_GRAD_ADD_SR}


@pytest.mark.parametrize("mode,gt", MODES)
@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,rows,dim,kind", [
    (1, 1, 1, "one"), (1, 5, 8, "mixed"), (33, 10, 24, "mixed"), (64, 3, 520, "mixed"), (65, 3, 17, "one"),
    (97, 1, 40, "one"), (200, 40, 136, "none"), (500, 30, 1001, "mixed"), (1025, 600, 72, "zipf")])
def test_grad(mode, gt, dt, n, rows, dim, kind):
    g = torch.Generator().manual_seed(n + rows + dim)
    dout = torch.randn(n, dim, generator=g).to(T[dt])
    old = torch.randn(rows, dim, generator=g).to(T[gt])
    ids = make_ids(n, rows, torch.int64 if n % 2 else torch.int32, n, kind)
    got = run_grad(dout, ids, 0.7, old, MODE[mode], seed=n * 1234567891011, base=rows * 3 + 5)
    check_grad(dout, ids, 0.7, old, got, MODE[mode], gt)


@pytest.mark.parametrize("mode,gt", [("write", "fp32"), ("write", "fp16"), ("add", "fp32"), ("add", "bf16"),
                                     ("add_sr", "bf16")])
@pytest.mark.parametrize("n,rows,dim", [(9000, 3000, 1544), (24000, 3000, 1545), (24000, 700, 2048),
                                        (40000, 3000, 1544), (36000, 40, 1001)])
def test_grad_of_many_tokens(mode, gt, n, rows, dim):
    """Chunks of 8, 16 and 32 tokens, several column groups, long and short runs."""
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    dout = torch.randn(n, dim, generator=g, device="cuda").bfloat16()
    old = torch.randn(rows, dim, generator=g, device="cuda").to(T[gt])
    ids = make_ids(n, rows, torch.int64, n)
    got = run_grad(dout, ids, 0.3, old, MODE[mode], seed=n, base=dim)
    check_grad(dout, ids, 0.3, old, got, MODE[mode], gt)


@pytest.mark.parametrize("mode,gt", MODES)
@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
def test_grad_every_remainder(mode, gt, dt):
    g = torch.Generator(device="cuda").manual_seed(7)
    ids = make_ids(150, 11, torch.int32, 8)
    for dim in list(range(1, 18)) + list(range(509, 522)):
        dout = torch.randn(150, dim, generator=g, device="cuda").to(T[dt])
        old = torch.randn(11, dim, generator=g, device="cuda").to(T[gt])
        got = run_grad(dout, ids, 0.7, old, MODE[mode], seed=dim, base=3 * dim)
        check_grad(dout, ids, 0.7, old, got, MODE[mode], gt)


SWEEP = np.random.default_rng(2024)


def draw():
    n = int(2 ** SWEEP.uniform(0, 14))
    return (n, int(2 ** SWEEP.uniform(0, 12)), int(2 ** SWEEP.uniform(0, 11 if n < 3000 else 8)),
            ["fp32", "bf16", "fp16"][SWEEP.integers(3)], *MODES[SWEEP.integers(len(MODES))],
            ["one", "zipf", "mixed", "none"][SWEEP.choice(4, p=[0.1, 0.4, 0.45, 0.05])], int(SWEEP.integers(1 << 40)))


@pytest.mark.parametrize("n,rows,dim,dt,mode,gt,kind,seed", [draw() for _ in range(96)])
def test_grad_random_sweep(n, rows, dim, dt, mode, gt, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dout = torch.randn(n, dim, generator=g, device="cuda").to(T[dt])
    old = torch.randn(rows, dim, generator=g, device="cuda").to(T[gt])
    ids = make_ids(n, rows, torch.int64 if seed % 2 else torch.int32, seed, kind)
    got = run_grad(dout, ids, -1.25, old, MODE[mode], seed=seed * 977, base=seed % 1000)
    check_grad(dout, ids, -1.25, old, got, MODE[mode], gt)


@pytest.mark.parametrize("n", [2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 128, 129, 160, 1000, 2048, 2049, 4096, 4097,
                               8192, 8193, 16384, 20000,
                               32768, 32769, 70000, 140000])
@pytest.mark.parametrize("kind", ["one", "zipf", "mixed", "runs"])
def test_grad_run_lengths(n, kind):
    """Runs that end at, before and after every chunk border, both sorts, and
    one run over everything; int values, so every sum is exact and the result
    has to be the sum itself."""
    rows, dim = 700, 16
    g = torch.Generator().manual_seed(n)
    if kind == "runs":
        ids, r = [], 0
        lengths = [1, 31, 32, 33, 63, 64, 65, 96, 97, 2, 128, 5]
        while len(ids) < n:
            ids += [r % rows] * lengths[r % len(lengths)]
            r += 1
        ids = torch.tensor(ids[:n])[torch.randperm(n, generator=g)]
    else:
        ids = make_ids(n, rows, torch.int64, n, kind)
    dout = torch.randint(-100, 101, (n, dim), generator=g).float()
    got = run_grad(dout, ids, 1.0, torch.zeros(rows, dim), zq.ZQ_GRAD_WRITE)
    there = (ids >= 0) & (ids < rows)
    exp = torch.zeros(rows, dim).index_add_(0, ids[there], dout[there])
    assert torch.equal(got.cpu(), exp)


@pytest.mark.parametrize("n,dim", [(64, 16), (65, 16), (300, 8), (5000, 520), (24000, 16), (40000, 1544), (300000, 16),
                                   (1 << 20, 16)])
@pytest.mark.parametrize("other", [0, 10])
def test_grad_error_of_long_runs(n, dim, other):
    """The header's bound for a row of m tokens, min(m - 1, 70 + m / 64) u / (1 -
    that u) times the sum of |dout| with u = 2^-24 (the write is exact with scale
    1), on positive values, whose partial sums are as large as they get; one row
    has all the tokens, or all but `other` % of them."""
    g = torch.Generator(device="cuda").manual_seed(n + other)
    rows = 5
    dout = torch.rand(n, dim, generator=g, device="cuda").add_(0.5)
    ids = torch.full((n,), 3, device="cuda")
    ids[torch.rand(n, generator=g, device="cuda") * 100 < other] = 1
    got = run_grad(dout, ids, 1.0, torch.zeros(rows, dim), zq.ZQ_GRAD_WRITE).double()
    for r in (1, 3):
        m = int((ids == r).sum())
        exact = dout[ids == r].double().sum(0)
        ku = min(max(m - 1, 0), 70 + m // 64) * 2.0 ** -24
        assert bool(((got[r] - exact).abs() <= ku / (1 - ku) * exact).all())


@pytest.mark.parametrize("rows", [1, 2, 255, 511, 512, 513, 50257, 262143, 262144, 300001, 500003, 2 ** 20,
                                  2 ** 27 + 5])
@pytest.mark.parametrize("n", [300, 9000])
def test_grad_vocabularies(rows, n):
    """Ranges of one row to 512 rows, one to four digits, both sorts; the largest and smallest row
    are named, and positions of equal ids keep their order (a sum of values that
    cancel only in that order)."""
    dim = 2
    ids = make_ids(n, rows, torch.int64, rows % 1000, "zipf")
    ids[:2] = torch.tensor([0, rows - 1])
    ids[7:200:3] = rows // 2
    dout = torch.randint(-9, 10, (n, dim)).float()
    order = (ids == rows // 2).nonzero()[:, 0]
    dout[order[0]], dout[order[1]], dout[order[2]] = 1.0, 2.0 ** 24, -(2.0 ** 24)
    grad = torch.full((rows, dim), 5.0, device="cuda")
    ws = torch.empty(zq.embed_grad_workspace(n, rows, dim), dtype=torch.uint8, device="cuda")
    zq.zq_embed_grad(dout.cuda(), ids.cuda(), 1.0, grad, zq.ZQ_GRAD_ADD, ws)
    named = ids.unique()
    other = ids != rows // 2
    exp = torch.zeros(rows, dim, device="cuda").index_add_(0, ids[other].cuda(), dout[other].cuda()).add_(5.0)
    # 1 + 2^24 rounds to 2^24, so the first three add up to 0, and the rest are
    # small integers: exact in any grouping.
    exp[rows // 2] = 5.0 + dout[order[3:]].sum(0).cuda()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[named.cuda()] = False
    assert bool((grad[keep] == 5.0).all())
    written = torch.full((rows, dim), math.nan, device="cuda")
    zq.zq_embed_grad(dout.cuda(), ids.cuda(), 1.0, written, zq.ZQ_GRAD_WRITE, ws)
    assert torch.equal(written, exp - 5.0)
    assert torch.equal(grad, exp)


@pytest.mark.parametrize("dim,base", [(8, 0), (16, 3), (17, 0), (40, 7), (521, 2 ** 35 + 6), (768, 5), (1001, 12)])
@pytest.mark.parametrize("n", [40, 300])
def test_grad_sr_bits(dim, base, n):
    """Sums that bf16 holds exactly: the result is the oracle's zq_sr_accumulate
    of the whole table, bit for bit (long runs too)."""
    rows = 9
    g = torch.Generator().manual_seed(dim + n)
    ids = make_ids(n, rows - 1, torch.int64, dim, "zipf")  # the last row stays unnamed
    dout = torch.zeros(n, dim)
    first = [int((ids == r).nonzero()[0]) for r in ids.unique()]
    dout[first] = torch.randint(-60, 61, (len(first), dim), generator=g).float() / 8
    old = torch.randn(rows, dim, generator=g).mul(3).bfloat16()
    seed = 0x123456789ABCDEF + n
    got = run_grad(dout.bfloat16(), ids, 0.5, old, zq.ZQ_GRAD_ADD_SR, seed=seed, base=base)
    src = torch.zeros(rows, dim).index_add_(0, ids, dout * 0.5).bfloat16()
    bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16).reshape(-1).copy()
    dst = bits(old)
    O.sr_accumulate(dst, bits(src), seed, base, False)
    assert np.array_equal(bits(got.cpu()), dst)


def test_grad_of_special_values():
    """NaN and infinities stay in their rows and columns; padded tokens' NaN
    stays out."""
    n, rows, dim = 150, 6, 24
    dout = torch.ones(n, dim)
    ids = torch.arange(n) % 5
    dout[0, 3], dout[1, 4], dout[6, 5], dout[11, 5] = math.nan, math.inf, math.inf, -math.inf
    ids[2] = -1
    dout[2] = math.nan
    for mode, gt in MODES:
        old = torch.zeros(rows, dim, dtype=T[gt])
        got = run_grad(dout, ids, 1.0, old, MODE[mode]).cpu().float()
        exp = torch.zeros(rows, dim).index_add_(0, ids[ids >= 0], dout[ids >= 0])
        assert torch.equal(got.isnan(), exp.isnan())
        fine = ~exp.isnan()
        assert torch.equal(got[fine], exp[fine])


def test_grad_of_no_tokens():
    for gt in T:
        for rows, dim in ((1, 1), (3, 7), (1000, 521)):
            buf = torch.full((rows * dim + GUARD,), 5.0, dtype=T[gt], device="cuda")
            grad = buf[:rows * dim].view(rows, dim)
            none = torch.empty(0, dtype=torch.int64, device="cuda")
            ws = torch.empty(0, dtype=torch.uint8, device="cuda")
            d = torch.empty(0, dim, device="cuda")
            zq.zq_embed_grad(d, none, 1.0, grad, zq.ZQ_GRAD_ADD, ws)
            assert bool((buf == 5).all())
            zq.zq_embed_grad(d, none, 1.0, grad, zq.ZQ_GRAD_WRITE, ws)
            assert bool((grad == 0).all()) and bool((buf[rows * dim:] == 5).all())


def test_grad_equals_differences_of_the_lookup():
    """The lookup is linear in the table: the difference of a loss between two
    tables is the gradient's product with the tables' difference."""
    rows, dim, n = 60, 40, 400
    g = torch.Generator().manual_seed(3)
    w = torch.randint(-8, 9, (rows, dim), generator=g).float()
    r = torch.randint(-8, 9, (n, dim), generator=g).float()
    ids = make_ids(n, rows, torch.int64, 4)
    grad = run_grad(r, ids, 4.0, w, zq.ZQ_GRAD_WRITE).cpu().double()

    def loss(table):
        out = torch.empty(n, dim, device="cuda")
        zq.zq_embed_lookup(table.cuda(), ids.cuda(), 4.0, out)
        return float((out.cpu().double() * r.double()).sum())

    for k in range(40):
        v, j = int(torch.randint(0, rows, (1,), generator=g)), int(torch.randint(0, dim, (1,), generator=g))
        up, down = w.clone(), w.clone()
        up[v, j] += 0.5
        down[v, j] -= 0.5
        assert loss(up) - loss(down) == float(grad[v, j])  # all values are small integers or halves


def test_grad_is_deterministic_and_independent_of_the_workspace():
    n, rows, dim = 12000, 400, 520
    dout = torch.randn(n, dim, device="cuda").bfloat16()
    ids = make_ids(n, rows, torch.int32, 1).cuda()
    got = []
    for fill in (0, 0xFF, 0x5A):
        grad = torch.empty(rows, dim, device="cuda")
        ws = torch.full((zq.embed_grad_workspace(n, rows, dim),), fill, dtype=torch.uint8, device="cuda")
        zq.zq_embed_grad(dout, ids, 1.0, grad, zq.ZQ_GRAD_WRITE, ws)
        got.append(grad.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_a_larger_buffer_and_an_offset_slice():
    """Aligned slices of larger buffers, more workspace than needed."""
    rows, dim, n = 20, 16, 70
    big = torch.randn(100, 16, device="cuda")
    ids = make_ids(n, rows, torch.int64, 8).cuda()
    dout = big[10:10 + n]
    grad = torch.zeros(50, 16, device="cuda")[4:24]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    zq.zq_embed_grad(dout, ids, 1.0, grad, zq.ZQ_GRAD_WRITE, ws)
    check_grad(dout, ids, 1.0, grad.clone(), grad, zq.ZQ_GRAD_WRITE, "fp32")
    with pytest.raises(ValueError, match="contiguous"):
        zq.zq_embed_lookup(big[:, :8], ids, 1.0, torch.empty(n, 8, device="cuda"))
    with pytest.raises(ValueError, match="workspace holds"):
        zq.zq_embed_grad(dout, ids, 1.0, grad, zq.ZQ_GRAD_WRITE, ws[:64])
    with pytest.raises(ValueError, match="out holds"):
        zq.zq_embed_lookup(big, ids, 1.0, torch.empty(n - 1, 16, device="cuda"))
    with pytest.raises(TypeError):
        zq.zq_embed_lookup(big, ids.float(), 1.0, torch.empty(n, 16, device="cuda"))
    with pytest.raises(zq.ZQError, match="DTYPE"):
        zq.zq_embed_grad(dout, ids, 1.0, grad, zq.ZQ_GRAD_ADD_SR, ws)


def test_offsets_past_2_to_32():
    """A bf16 table and gradient of more than 2^32 elements (rows on both sides
    of 2^31 and 2^32 elements), and an output of more than 2^32."""
    dim, rows = 4104, (1 << 20) + 3000
    w = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    at = sorted({0, 1, rows - 1} | {(e // dim) + k for e in (1 << 31, 1 << 32) for k in (-1, 0, 1)})
    vals = torch.randn(len(at), dim, device="cuda").bfloat16()
    w[torch.tensor(at, device="cuda")] = vals
    ids = torch.tensor(at * 3, device="cuda")
    out = torch.empty(len(ids), dim, dtype=torch.bfloat16, device="cuda")
    zq.zq_embed_lookup(w, ids, 1.0, out)
    assert torch.equal(out, vals.repeat(3, 1))
    ws = torch.empty(zq.embed_grad_workspace(len(ids), rows, dim), dtype=torch.uint8, device="cuda")
    zq.zq_embed_grad(out, ids, 1.0, w, zq.ZQ_GRAD_ADD, ws)  # w + 3 w
    exp = (vals.double() * 4).float().bfloat16()
    assert torch.equal(w[torch.tensor(at, device="cuda")], exp)
    zq.zq_embed_grad(out, ids, 1.0, w, zq.ZQ_GRAD_WRITE, ws)
    assert int(w.count_nonzero()) == int((vals.float() * 3).bfloat16().count_nonzero())
    del w
    n = (1 << 20) + 3000
    small = torch.randn(8, dim, device="cuda").bfloat16()
    ids = torch.randint(0, 8, (n,), device="cuda", dtype=torch.int32)
    out = torch.full((n, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    zq.zq_embed_lookup(small, ids, 1.0, out)
    for t in [0, n - 1] + [e // dim + k for e in (1 << 31, 1 << 32) for k in (-1, 0, 1)]:
        assert torch.equal(out[t], small[int(ids[t])])
    # The gradient of that many tokens: 131073 chunks, runs of 2^17 tokens.
    one = torch.ones(1, device="cuda", dtype=torch.bfloat16).expand(n, dim).contiguous()
    grad = torch.empty(8, dim, device="cuda")
    ws = torch.empty(zq.embed_grad_workspace(n, 8, dim), dtype=torch.uint8, device="cuda")
    zq.zq_embed_grad(one, ids, 1.0, grad, zq.ZQ_GRAD_WRITE, ws)
    assert torch.equal(grad, torch.bincount(ids, minlength=8).float()[:, None].expand(8, dim))
