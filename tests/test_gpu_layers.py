"""SwiGLU and linear gradients from int8 activations, and the vocabulary
projection's cross entropy, on the GPU, against their formulas in 64 bits.

Tolerances are sums of what each rounding may do (u = half a step of a 16-bit
type relative to the value: bf16 2^-8, fp16 2^-11):
  swiglu  h 2^-21 of itself (exponential, reciprocal, sum and two products of
          2^-23 or less each), gradients 2^-20 (two products and a sum more; the
          sum's terms stand in the bound with their sizes); then u, or 2^-24 for fp32
  a product of K terms  (K + 8) 2^-24 times the sum of the terms' sizes
  lse     what the logits are off by, and 2^-23 (64 + V / 2048 + |lse|) for the
          exponentials and sums
  q       u of itself, and p times what its exponent is off by
In fp16 a result below 2^-14 is off by up to 2^-25, q by 2^-25 before it is scaled
back.
"""
import math

import pytest
import torch

from weight_communication_zero_amd import zq

pytestmark = pytest.mark.gpu

T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
GUARD = 64
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


class Out:
    """An output of n elements, poisoned, with guard elements after it."""

    def __init__(self, shape, dtype, fill=None):
        n = math.prod(shape)
        self.buf = torch.full((n + GUARD,), 77 if fill is None else 0, dtype=dtype, device="cuda")
        if fill is not None:
            self.buf[:n] = fill.reshape(-1)
            self.buf[n:] = 77
        self.t = self.buf[:n].view(shape)
        self.n = n

    def check(self):
        assert bool((self.buf[self.n:] == 77).all()), "write past the end of an output"
        return self.t


def workspace(size):
    buf = torch.full((size + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
    return buf


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def quantized(x, block):
    """zq_quant_int8 of x and the 64-bit values that the blocks hold."""
    n = x.numel()
    codes = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(-(-n // block), device="cuda")
    zq.zq_quant_int8(x.contiguous(), block, codes, scales)
    return codes, scales, held(codes, scales, block)


def held(codes, scales, block):
    at = torch.arange(codes.numel(), device="cuda") // block
    return (codes.reshape(-1).float() * scales[at]).double().view(codes.shape)


def near(got, want, bound, what=""):
    got, want = got.double(), want.double()
    fine = want.isfinite()
    assert torch.equal(fine, got.isfinite()), what + ": another set of finite values"
    assert torch.equal(want.isnan(), got.isnan()), what + ": NaN elsewhere"
    inf = want.isinf()
    assert torch.equal(want[inf], got[inf]), what + ": infinities"
    off = (got - want).abs()[fine] - (bound if isinstance(bound, float) else bound.expand(want.shape)[fine])
    assert off.numel() == 0 or float(off.max()) <= 0, (what, float(off.max()), float((got - want).abs()[fine].max()))


def same(a, b):
    kind = {1: torch.int8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


# ---- SwiGLU ---------------------------------------------------------------

def sigmoid_pair(g):
    return torch.special.expit(g), torch.special.expit(-g)


def swiglu(gate, up, block):
    n = gate.numel()
    h = Out((n,), gate.dtype)
    gc, uc = Out((n,), torch.int8), Out((n,), torch.int8)
    gs, us = Out((-(-n // block),), torch.float32), Out((-(-n // block),), torch.float32)
    zq.zq_swiglu_int8(gate, up, block, h.t, gc.t, gs.t, uc.t, us.t)
    torch.cuda.synchronize()
    return tuple(x.check() for x in (h, gc, gs, uc, us))


def swiglu_grad(kept, block, dh, with_h):
    n = dh.numel()
    dg, du = Out((n,), dh.dtype), Out((n,), dh.dtype)
    h = Out((n,), dh.dtype) if with_h else None
    zq.zq_swiglu_grad_int8(*kept, block, dh, dg.t, du.t, h=h.t if h else None)
    torch.cuda.synchronize()
    return dg.check(), du.check(), h.check() if h else None


def check_grads(got, g, u, dh, what):
    dg, du, h = got
    s, r = sigmoid_pair(g)
    t = dh.dtype
    d = dh.double()
    size = (d * u * s).abs() * (1 + (g * r).abs())
    want = d * u * s * (1 + g * r)
    near(dg, want, 2.0 ** -20 * size + U[t] * want.abs() + FLOOR[t], what + " dgate")
    want = d * g * s
    near(du, want, (2.0 ** -20 + U[t]) * want.abs() + FLOOR[t], what + " dup")
    if h is not None:
        want = g * s * u
        near(h, want, (2.0 ** -20 + U[t]) * want.abs() + FLOOR[t], what + " h")


SIZES = [1, 7, 8, 31, 33, 511, 512, 513, 4095, 4097, 20011]


@pytest.mark.parametrize("dtype", sorted(T))
@pytest.mark.parametrize("block", [32, 64, 128, 256, 512, 1024, 2048, 4096])
def test_swiglu_and_its_gradient(dtype, block):
    t = T[dtype]
    for n in SIZES + [3 * block - 5]:
        gate, up = randn((n,), n, t, 3.0), randn((n,), n + 1, t)
        h, gc, gs, uc, us = swiglu(gate, up, block)
        for x, c, s in ((gate, gc, gs), (up, uc, us)):
            codes, scales, _ = quantized(x, block)
            same(c, codes)
            same(s, scales)
        g, u = gate.double(), up.double()
        want = g * torch.special.expit(g) * u
        near(h, want, (2.0 ** -21 + U[t]) * want.abs() + FLOOR[t], f"h n={n}")
        dh = randn((n,), n + 2, t, 0.1)
        kept = (gc, gs, uc, us)
        for with_h in (False, True):
            check_grads(swiglu_grad(kept, block, dh, with_h), held(gc, gs, block), held(uc, us, block), dh, f"n={n}")


@pytest.mark.parametrize("dtype", sorted(T))
def test_swiglu_far_gates_zeros_and_infinities(dtype):
    t = T[dtype]
    g = torch.tensor([0.0, -0.0, 1e-4, -1e-4, 10, -10, 60, -60, 87, -87, 89, -89, 300, -300, 6e4, -6e4], device="cuda")
    n = 64 * g.numel()
    gate = g.repeat(64).to(t)                       # blocks of 32 hold every gate twice
    up = randn((n,), 5, t)
    h, gc, gs, uc, us = swiglu(gate, up, 32)
    x = gate.double()
    want = x * torch.special.expit(x) * up.double()
    if t == torch.float16:  # rounding to binary16 gives infinity from 65520 (its largest value and half a step) up
        want = torch.where(want.abs() >= 65520, want.sign() * INF, want)
    # exp(-|g|) below 2^-126 is taken as 0: sizes up to 2^-126 |g u| may vanish.
    tiny = 2.0 ** -126 * (x * up.double()).abs()
    near(h, want, (2.0 ** -21 + U[t]) * want.abs() + FLOOR[t] + tiny, "h")
    # Kept gates up to +-300 in blocks of one size each.
    k = torch.randint(-127, 128, (n,), generator=gen(6), device="cuda", dtype=torch.int8)
    s = torch.logspace(-6, math.log10(300 / 127), n // 32, device="cuda")
    dh = randn((n,), 7, t)
    gv, uv = held(k, s, 32), held(uc, us, 32)
    dg, du, h = swiglu_grad((k, s, uc, us), 32, dh, True)
    sg, r = sigmoid_pair(gv)
    d = dh.double()
    tiny = 2.0 ** -126 * (1 + gv.abs()) ** 2 * (1 + (d * uv).abs()) * (1 + d.abs() + uv.abs())
    size = (d * uv * sg).abs() * (1 + (gv * r).abs())
    near(dg, d * uv * sg * (1 + gv * r), (2.0 ** -20 + U[t]) * size + FLOOR[t] + tiny, "dgate")
    near(du, d * gv * sg, (2.0 ** -20 + U[t]) * (d * gv * sg).abs() + FLOOR[t] + tiny, "dup")
    near(h, gv * sg * uv, (2.0 ** -20 + U[t]) * (gv * sg * uv).abs() + FLOOR[t] + tiny, "h")
    # An infinity or NaN touches its own product, and its own block's codes, alone.
    gate, up = randn((256,), 8, t), randn((256,), 9, t)
    want, gc0, gs0, uc0, us0 = (x.clone() for x in swiglu(gate, up, 64))
    gate[70], gate[71], up[200], gate[72] = INF, -INF, NAN, NAN
    h, gc, gs, uc, us = swiglu(gate, up, 64)
    rest = torch.ones(256, dtype=torch.bool, device="cuda")
    rest[[70, 71, 72, 200]] = False
    same(h[rest], want[rest])
    assert float(h[70]) == math.copysign(INF, float(up[70])) and bool(h[[71, 72, 200]].isnan().all())
    whole = torch.arange(256, device="cuda") // 64 != 1
    same(gc[whole], gc0[whole])
    same(us[:3], us0[:3])


def test_swiglu_inputs_may_be_one_buffer_and_lie_anywhere():
    buf = randn((3, 4104), 1, torch.bfloat16)
    gate, up = buf[0, 8:4104], buf[1, 8:4104]       # 16-byte aligned rows of a wider tensor
    h, *kept = swiglu(gate, up, 128)
    want = gate.double() * torch.special.expit(gate.double()) * up.double()
    near(h, want, (2.0 ** -21 + 2.0 ** -8) * want.abs() + 2.0 ** -133)
    h, gc, gs, uc, us = swiglu(gate, gate, 128)
    same(gc, uc)
    same(gs, us)


def test_swiglu_gradient_agrees_with_differences():
    n, block = 4096, 128
    _, _, gate = quantized(randn((n,), 1, std=2.0), block)   # values that their own blocks hold
    _, _, up = quantized(randn((n,), 2), block)
    gate, up = gate.float(), up.float()
    dh = randn((n,), 3)
    _, *kept = swiglu(gate, up, block)
    assert torch.equal(held(kept[0], kept[1], block).float(), gate)
    dg, du, _ = swiglu_grad(kept, block, dh, False)
    e = 2.0 ** -8
    for grad, plus, minus in ((dg, (gate + e, up), (gate - e, up)), (du, (gate, up + e), (gate, up - e))):
        a, b = swiglu(*plus, block)[0], swiglu(*minus, block)[0]
        step = ((plus[0] - minus[0]).double() + (plus[1] - minus[1]).double())
        diff = (a.double() - b.double()) / step * dh.double()
        # The third derivative of silu is below 0.6: e^2 / 6 of it; and two roundings of h, 2^-21 each, over 2 e.
        bound = dh.double().abs() * (up.double().abs() * 0.1 * e * e + (a.abs() + b.abs()).double() * 2.0 ** -21 / (2 * e))
        near(grad, diff, bound + 2.0 ** -20 * (1 + diff.abs()))


# ---- a linear layer's weight gradient -------------------------------------

def linear_grad(dy, codes, scales, block, grad, mode):
    (n, o), i = dy.shape, codes.shape[1]
    out = Out((o, i), grad if isinstance(grad, torch.dtype) else grad.dtype,
              None if isinstance(grad, torch.dtype) else grad)
    need = zq.linear_grad_workspace(n, o, i)
    ws = workspace(need)
    zq.zq_linear_grad_int8(dy, codes, scales, block, out.t, mode, ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    return out.check()


def linear_want(dy, codes, scales, block, old, t):
    x = held(codes, scales, block).float().to(dy.dtype).double()
    d = dy.double()
    want, size = d.t() @ x, d.abs().t() @ x.abs()
    bound = (dy.shape[0] + 8) * 2.0 ** -24 * size
    if old is not None:
        want = want + old.double()
        bound = bound + 2.0 ** -24 * want.abs()
    return want, bound + U[t] * want.abs() + FLOOR[t]


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 9), (63, 64, 72), (64, 128, 128), (65, 129, 7), (200, 300, 260),
          (1001, 321, 515), (130, 512, 1024), (5000, 40, 24)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_grad(dtype, shape):
    n, o, i = shape
    t = T[dtype]
    dy = randn((n, o), 1, t, 0.1)
    for k, block in enumerate((32, 256, 4096)):
        codes, scales, _ = quantized(randn((n, i), 2), block)
        for out in (t, torch.float32):
            want, bound = linear_want(dy, codes, scales, block, None, out)
            near(linear_grad(dy, codes, scales, block, out, zq.ZQ_GRAD_WRITE), want, bound, f"write {block} {out}")
        old = randn((o, i), 3 + k, out)
        want, bound = linear_want(dy, codes, scales, block, old, out)
        near(linear_grad(dy, codes, scales, block, old, zq.ZQ_GRAD_ADD), want, bound, f"add {block}")
    old = randn((o, i), 9, t)
    want, bound = linear_want(dy, codes, scales, block, old, t)
    near(linear_grad(dy, codes, scales, block, old, zq.ZQ_GRAD_ADD), want, bound, "add 16-bit")


def test_linear_grad_of_a_16_bit_type_other_than_the_products():
    dy = randn((77, 24), 1, torch.bfloat16)
    codes, scales, _ = quantized(randn((77, 40), 2), 64)
    want, bound = linear_want(dy, codes, scales, 64, None, torch.float16)
    near(linear_grad(dy, codes, scales, 64, torch.float16, zq.ZQ_GRAD_WRITE), want, bound)


@pytest.mark.parametrize("shape", [(8192, 256, 128), (8200, 2048, 2048), (4096, 1, 640)])
def test_linear_grad_long_sums_split_and_equal_bits(shape):
    n, o, i = shape
    dy = randn((n, o), 1, torch.bfloat16)
    codes, scales, _ = quantized(randn((n, i), 2), 128)
    a = linear_grad(dy, codes, scales, 128, torch.float32, zq.ZQ_GRAD_WRITE)
    want, bound = linear_want(dy, codes, scales, 128, None, torch.float32)
    near(a, want, bound)
    for _ in range(3):
        same(a, linear_grad(dy, codes, scales, 128, torch.float32, zq.ZQ_GRAD_WRITE))


def test_linear_grad_of_the_most_tokens():
    n, o, i = 1 << 20, 9, 16
    dy = randn((n, o), 1, torch.bfloat16)
    codes, scales, _ = quantized(randn((n, i), 2), 4096)
    want, bound = linear_want(dy, codes, scales, 4096, None, torch.float32)
    near(linear_grad(dy, codes, scales, 4096, torch.float32, zq.ZQ_GRAD_WRITE), want, bound)


def test_linear_grad_infinities_stay_in_their_row():
    """The last token's step of 64 is ragged: what fills it up must not meet an
    infinity of dy or a NaN."""
    n, o, i = 70, 130, 140
    dy = randn((n, o), 1, torch.bfloat16)
    codes, scales, _ = quantized(randn((n, i), 2), 32)
    dy[69, 7], dy[69, 100], dy[3, 50] = INF, NAN, -INF
    want, bound = linear_want(dy, codes, scales, 32, None, torch.float32)
    zero = (codes[[69, 3]] == 0)
    got = linear_grad(dy, codes, scales, 32, torch.float32, zq.ZQ_GRAD_WRITE)
    rows = torch.ones(o, dtype=torch.bool, device="cuda")
    rows[[7, 50, 100]] = False
    near(got[rows], want[rows], bound[rows])
    assert bool(got[100].isnan().all())
    for row, tok, sign in ((7, 0, 1), (50, 1, -1)):
        x = codes[[69, 3]][tok].double() * sign
        assert torch.equal(got[row].isnan(), zero[tok]) and bool((got[row][~zero[tok]] == x[~zero[tok]].sign() * INF).all())


# ---- cross entropy --------------------------------------------------------

def ce_inputs(n, d, rows, dtype, seed, pad=0, id_type=torch.int64, std=0.05):
    t = T[dtype]
    x, w = randn((n, d), seed, t), randn((rows, d), seed + 1, t, std)
    ids = torch.randint(0, rows, (n,), generator=gen(seed + 2), device="cuda")
    out = torch.rand(n, generator=gen(seed + 3), device="cuda") * 100 < pad
    none = torch.tensor([-1, rows, -100, 2 ** 31 - 1], device="cuda")[torch.arange(n, device="cuda") % 4]
    ids = torch.where(out, none, ids).to(id_type)
    x[out] = NAN                                              # padding may hold anything
    return x, w, ids, ~out


def ce_loss(x, w, ids, scale=1.0, piece=0, codes=None):
    n, (rows, d) = ids.numel(), w.shape
    loss, lse = Out((n,), torch.float32), Out((n,), torch.float32)
    need = zq.ce_loss_workspace(n, rows, d, piece)
    ws = workspace(need)
    if codes:
        zq.zq_ce_loss_int8(x, *codes, ids, scale, loss.t, lse.t, ws[:need], piece=piece)
    else:
        zq.zq_ce_loss(x, w, ids, scale, loss.t, lse.t, ws[:need], piece=piece)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    return loss.check(), lse.check()


def logits(x, w, scale):
    x, w = x.double(), w.double()
    z = x @ w.t() * scale
    off = (x.shape[1] + 8) * 2.0 ** -24 * abs(scale) * (x.abs() @ w.abs().t()) + 2.0 ** -23 * z.abs()
    return z, off


def check_loss(got, x, w, ids, there, scale):
    loss, lse = got
    rows = w.shape[0]
    assert not bool(loss[~there].view(torch.int32).any()) and not bool(lse[~there].view(torch.int32).any())
    z, off = logits(x[there], w, scale)
    want = torch.logsumexp(z, 1)
    bound = off.max(1).values + 2.0 ** -23 * (64 + rows / 2048 + want.abs())
    near(lse[there], want, bound, "lse")
    near(loss[there], want - z.gather(1, ids[there].long()[:, None])[:, 0], 2 * bound, "loss")


CE = [(1, 1, 1), (1, 64, 100), (2, 7, 2), (3, 65, 257), (17, 128, 1000), (64, 512, 640), (130, 192, 999),
      (300, 100, 5003), (257, 256, 256), (33, 768, 50257)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", CE)
def test_ce_loss(dtype, shape):
    n, d, rows = shape
    for pad, id_type, scale, piece in ((0, torch.int64, 1.0, 0), (30, torch.int32, 0.5, 256), (30, torch.int64, -2.0, 700)):
        x, w, ids, there = ce_inputs(n, d, rows, dtype, n + d, pad, id_type)
        check_loss(ce_loss(x, w, ids, scale, piece), x, w, ids, there, scale)


# Beyond 512 tokens the loss gathers those that count; from 1025 on the gathering takes 8 ids a thread, beyond 8192
# more than one round; 2^20 tokens are the most.
LONG = [(512, 64, 300), (513, 64, 300), (1024, 128, 65), (1025, 192, 777), (2050, 100, 515), (9000, 64, 130),
        (1 << 20, 8, 5)]


@pytest.mark.parametrize("pad", [0, 10, 60, 99])
@pytest.mark.parametrize("shape", LONG)
def test_ce_of_many_tokens(shape, pad):
    n, d, rows = shape
    x, w, ids, there = ce_inputs(n, d, rows, "bf16", n + pad, pad)
    got = ce_loss(x, w, ids)
    check_loss(got, x, w, ids, there, 1.0)
    lse = torch.where(there, got[1], NAN)
    dloss = torch.where(there, randn((n,), 9, std=30.0 / n), torch.full((n,), INF, device="cuda"))
    dx, bx, dw, bw = ce_want(x, w, ids, there, 1.0, lse, dloss)
    got = ce_grad(x, w, ids, 1.0, lse, dloss, torch.bfloat16)
    assert not bool(got[0][~there].view(torch.int16).any())
    near(got[0], dx, final(dx, bx, torch.bfloat16), "dx")
    near(got[1], dw, final(dw, bw, torch.bfloat16), "dw")


def test_ce_loss_of_tokens_that_are_all_left_out():
    x, w, ids, _ = ce_inputs(70, 64, 300, "bf16", 1, 101)
    loss, lse = ce_loss(x, w, ids)
    assert not bool(loss.any()) and not bool(lse.any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 100, 513])
def test_ce_loss_from_codes_equals_that_of_the_dequantized_values(dtype, dim):
    x, w, ids, there = ce_inputs(90, dim, 1111, dtype, 3, 10)
    for block in (32, 2048):
        codes, scales, _ = quantized(w, block)
        values = torch.empty_like(w)
        zq.zq_dequant_int8(codes, scales, block, values)
        for piece in (0, 512):
            a, b = ce_loss(x, w, ids, 1.0, piece, (codes, scales, block)), ce_loss(x, values, ids, 1.0, piece)
            same(a[0], b[0])
            same(a[1], b[1])
        check_loss(a, x, values, ids, there, 1.0)


def test_ce_loss_of_far_logits():
    x, w, ids, there = ce_inputs(40, 64, 500, "fp16", 1)
    w = (w.double() * 4000).half()                   # logits of thousands: no overflow, the others vanish
    check_loss(ce_loss(x, w, ids), x, w, ids, there, 1.0)
    check_loss(ce_loss(x, w * 0, ids), x, w * 0, ids, there, 1.0)    # log(rows) throughout


@pytest.mark.parametrize("piece", [0, 256])
def test_ce_loss_of_infinite_and_nan_logits(piece):
    x, w, ids, _ = ce_inputs(40, 64, 700, "bf16", 1)
    x = x.abs()
    w[5, 3], w[400, 9] = -INF, -INF                  # two logits of -inf for every token
    ids[0], ids[1] = 5, 400
    x[2, 0] = INF                                    # a token with infinities of both signs
    x[4, 1] = NAN
    w[650, 2] = INF                                  # +inf for every token
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    loss, lse = ce_loss(x, w, ids, 1.0, piece)
    near(lse, want, 0.0)
    near(loss, want - z.gather(1, ids[:, None])[:, 0], 0.0)
    w[650, 2] = 1.0
    x[2, 0] = 1.0
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    loss, lse = ce_loss(x, w, ids, 1.0, piece)
    near(lse, want, 1e-3)
    near(loss, want - z.gather(1, ids[:, None])[:, 0], 1e-3)
    w[:] = 1.0
    x[:] = 1.0
    w[:, 3] = -INF                                   # nothing but -inf: lse -inf, loss NaN
    loss, lse = ce_loss(x, w, ids, 1.0, piece)
    assert bool((lse == -INF).all()) and bool(loss.isnan().all())


def ce_grad(x, w, ids, scale, lse, dloss, dw, mode=zq.ZQ_GRAD_WRITE, piece=0, codes=None, with_dx=True):
    n, (rows, d) = ids.numel(), w.shape
    dx = Out((n, d), x.dtype) if with_dx else None
    out = None if dw is None else Out((rows, d), dw if isinstance(dw, torch.dtype) else dw.dtype,
                                      None if isinstance(dw, torch.dtype) else dw)
    need = zq.ce_grad_workspace(n, rows, d, piece)
    ws = workspace(need)
    head = (codes,) if codes else ((w,),)
    call = zq.zq_ce_grad_int8 if codes else zq.zq_ce_grad
    call(x, *head[0], ids, scale, lse, dloss, dx.t if dx else None, out.t if out else None, mode, ws[:need], piece=piece)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    return dx.check() if dx else None, out.check() if out else None


def ce_want(x, w, ids, there, scale, lse, dloss, u=None):
    """dx and dw in 64 bits, and what the roundings before the output's may do; u:
    q's relative rounding."""
    u, t = U[x.dtype] if u is None else u, x.dtype
    xs, ws, y = x[there].double(), w.double(), ids[there].long()
    z, off = logits(x[there], w, scale)
    g, l = dloss[there].double()[:, None], lse[there].double()[:, None]
    p = torch.exp(z - l)
    slack = p * (off + 2.0 ** -22 * (2 + (z - l).abs() + l.abs()))
    q = p.scatter_add(1, y[:, None], torch.full_like(l, -1.0))
    e = g.abs() * (u * (q.abs() + slack) + slack + 2.0 ** -23 * q.abs())
    if t == torch.float16 and g.numel():
        e = e + 2.0 ** -39 * float(g.abs().max()) * 2
    q = q * g
    k = 2.0 ** -24
    dx, dw = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), scale * (q.t() @ xs)
    bx = torch.zeros_like(dx)
    dx[there] = scale * (q @ ws)
    bx[there] = abs(scale) * (e @ ws.abs() + k * (w.shape[0] + 16) * ((q.abs() + e) @ ws.abs()))
    bw = abs(scale) * (e.t() @ xs.abs() + k * (len(xs) + 16) * ((q.abs() + e).t() @ xs.abs()))
    return dx, bx + 2.0 ** -23 * dx.abs(), dw, bw + 2.0 ** -23 * dw.abs()


def final(want, bound, t):
    return bound + U[t] * (want.abs() + bound) + FLOOR[t]


def exact_lse(x, w, ids, there, scale):
    z = x.double() @ w.double().t() * scale
    return torch.where(there, torch.logsumexp(z, 1), torch.full_like(z[:, 0], NAN)).float()   # NaN: not to be used


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", CE)
def test_ce_grad(dtype, shape):
    n, d, rows = shape
    t = T[dtype]
    for pad, id_type, scale, piece in ((0, torch.int64, 1.0, 0), (30, torch.int32, 0.5, 256), (30, torch.int64, -2.0, 700)):
        x, w, ids, there = ce_inputs(n, d, rows, dtype, n + d, pad, id_type)
        lse = exact_lse(x, w, ids, there, scale)
        dloss = torch.where(there, randn((n,), 9, std=30.0 / n), torch.full((n,), NAN, device="cuda"))
        dx, bx, dw, bw = ce_want(x, w, ids, there, scale, lse, dloss)
        got = ce_grad(x, w, ids, scale, lse, dloss, t, piece=piece)
        assert not bool(got[0][~there].view(torch.int16).any())
        near(got[0], dx, final(dx, bx, t), "dx")
        near(got[1], dw, final(dw, bw, t), "dw")
        got32 = ce_grad(x, w, ids, scale, lse, dloss, torch.float32, piece=piece, with_dx=False)
        near(got32[1], dw, final(dw, bw, torch.float32), "dw fp32")
        alone = ce_grad(x, w, ids, scale, lse, dloss, None, piece=piece)
        same(alone[0], got[0])
        old = randn((rows, d), 11, torch.float32)
        near(ce_grad(x, w, ids, scale, lse, dloss, old, zq.ZQ_GRAD_ADD, piece)[1], dw + old.double(),
             final(dw, bw, torch.float32) + 2.0 ** -23 * old.double().abs(), "dw added")
        old = randn((rows, d), 12, t)
        near(ce_grad(x, w, ids, scale, lse, dloss, old, zq.ZQ_GRAD_ADD, piece)[1], dw + old.double(),
             final(dw + old.double(), bw + 2.0 ** -23 * old.double().abs(), t), "dw added 16-bit")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 31, 64, 128])
def test_ce_grad_of_few_tokens_keeps_q_in_two_parts(n, dtype):
    """q's rounding is off by half a step of half a step; an fp32 dw shows it.  (A second
    part is below 2^-8 or 2^-11 of q and rounded by as much again.)"""
    x, w, ids, there = ce_inputs(n, 200, 1500, dtype, n, 20)
    lse = exact_lse(x, w, ids, there, 1.0)
    dloss = torch.where(there, randn((n,), 9), torch.full((n,), NAN, device="cuda"))
    dx, bx, dw, bw = ce_want(x, w, ids, there, 1.0, lse, dloss, u=U[T[dtype]] ** 2)
    for piece in (0, 512):
        got = ce_grad(x, w, ids, 1.0, lse, dloss, torch.float32, piece=piece)
        near(got[1], dw, final(dw, bw, torch.float32), "dw")
        near(got[0], dx, final(dx, bx, T[dtype]), "dx")


def test_ce_grad_of_tokens_that_are_all_left_out():
    x, w, ids, there = ce_inputs(70, 64, 300, "bf16", 1, 101)
    lse, dloss = torch.full((70,), NAN, device="cuda"), torch.full((70,), NAN, device="cuda")
    old = randn((300, 64), 1, torch.float32)
    for piece in (0, 256):
        dx, dw = ce_grad(x, w, ids, 1.0, lse, dloss, torch.bfloat16, piece=piece)
        assert not bool(dx.view(torch.int16).any()) and not bool((dw != 0).any())
        same(ce_grad(x, w, ids, 1.0, lse, dloss, old, zq.ZQ_GRAD_ADD, piece)[1], old)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 100, 513])
def test_ce_grad_from_codes_equals_that_of_the_dequantized_values(dtype, dim):
    x, w, ids, there = ce_inputs(90, dim, 1111, dtype, 3, 10)
    codes, scales, _ = quantized(w, 128)
    values = torch.empty_like(w)
    zq.zq_dequant_int8(codes, scales, 128, values)
    lse = exact_lse(x, values, ids, there, 1.0)
    dloss = randn((90,), 5)
    for piece in (0, 512):
        a = ce_grad(x, w, ids, 1.0, lse, dloss, T[dtype], piece=piece, codes=(codes, scales, 128))
        b = ce_grad(x, values, ids, 1.0, lse, dloss, T[dtype], piece=piece)
        same(a[0], b[0])
        same(a[1], b[1])


@pytest.mark.parametrize("std", [1e-12, 1e-3, 1e4])
def test_ce_grad_fp16_scales_the_probabilities(std):
    """Loss gradients from far below fp16's range to near its end."""
    x, w, ids, there = ce_inputs(100, 64, 400, "fp16", 3, 10)
    lse = exact_lse(x, w, ids, there, 1.0)
    dloss = randn((100,), 5, std=std)
    dx, bx, dw, bw = ce_want(x, w, ids, there, 1.0, lse, dloss)
    got = ce_grad(x, w, ids, 1.0, lse, dloss, torch.float32)
    near(got[1], dw, final(dw, bw, torch.float32), "dw")
    near(got[0], dx, final(dx, bx, torch.float16), "dx")


def test_ce_grad_of_zero_infinite_and_nan_loss_gradients():
    x, w, ids, there = ce_inputs(100, 64, 400, "fp16", 3)
    lse = exact_lse(x, w, ids, there, 1.0)
    dx, dw = ce_grad(x, w, ids, 1.0, lse, torch.zeros(100, device="cuda"), torch.float16)
    assert not bool((dx != 0).any()) and not bool((dw != 0).any())
    dloss = randn((100,), 5)
    clean = ce_grad(x, w, ids, 1.0, lse, dloss, torch.float16)[0].clone()
    dloss[7], dloss[9] = NAN, INF
    dx, dw = ce_grad(x, w, ids, 1.0, lse, dloss, torch.float16)
    rest = torch.ones(100, dtype=torch.bool, device="cuda")
    rest[[7, 9]] = False
    assert bool(dx[7].isnan().all()) and not bool(dx[9].isfinite().any()) and bool(dw.isnan().all())
    assert bool(dx[rest].isfinite().all())
    near(dx[rest], clean[rest], 2.0 ** -8 * clean[rest].double().abs() + 2.0 ** -14)


@pytest.mark.parametrize("n,d,rows", [(64, 64, 200), (33, 100, 77)])
def test_ce_gradient_agrees_with_differences(n, d, rows):
    """Central differences of zq_ce_loss along a random direction of signs.  x and w
    are multiples of their steps, so that both ends are exact in fp16."""
    ex, ew = 2.0 ** -6, 2.0 ** -9
    x = (randn((n, d), 1) / ex).round().clamp(-400, 400) * ex
    w = (randn((rows, d), 2) * 0.1 / ew).round() * ew
    x, w = x.half(), w.half()
    ids = torch.randint(0, rows, (n,), generator=gen(3), device="cuda")
    dloss = randn((n,), 4)
    lse = ce_loss(x, w, ids)[1].clone()
    dx, dw = ce_grad(x, w, ids, 1.0, lse, dloss, torch.float32)
    sx, sw = randn((n, d), 5).sign(), randn((rows, d), 6).sign()
    for grad, plus, minus, move, v in (
            (dx, ((x.float() + ex * sx).half(), w), ((x.float() - ex * sx).half(), w), ex * sx.double() @ w.double().t(), ex * sx),
            (dw, (x, (w.float() + ew * sw).half()), (x, (w.float() - ew * sw).half()), x.double() @ (ew * sw.double()).t(), ew * sw)):
        assert torch.equal(plus[0].float() + minus[0].float(), 2 * x.float())
        a, b = (ce_loss(*p, ids)[0].double() for p in (plus, minus))
        diff = ((a - b) / 2 * dloss.double()).sum()
        # Third order: the third cumulant of the logits' moves, below (their range)^3; and the losses' own error.
        third = (move.max(1).values - move.min(1).values) ** 3 / 6
        noise = 2.0 ** -23 * (64 + a.abs() + (d + 8) * 0.5 * (x.double().abs() @ w.double().abs().t()).max(1).values)
        bound = (dloss.double().abs() * (third + noise)).sum()
        along = (grad.double() * v.double()).sum()
        rounding = 2.0 ** -10 * (grad.double() * v.double()).abs().sum()  # dx's and q's
        assert abs(float(along - diff)) <= float(bound + rounding), (float(along), float(diff), float(bound + rounding))


def test_ce_equal_inputs_give_equal_bits():
    x, w, ids, there = ce_inputs(700, 256, 3001, "bf16", 3, 10)
    dloss = randn((700,), 5)
    first = None
    for _ in range(3):
        loss, lse = ce_loss(x, w, ids, 1.0, 1024)
        now = (loss, lse) + ce_grad(x, w, ids, 1.0, lse, dloss, torch.bfloat16, piece=1024)
        if first is None:
            first = now
        for a, b in zip(first, now):
            same(a, b)


@pytest.mark.parametrize("big", ["x", "w"])
def test_ce_beyond_4_gib(big):
    """Operands whose last rows start past 2^32 bytes."""
    n, d, rows = (140000, 16384, 64) if big == "x" else (64, 16384, 140000)
    t = torch.bfloat16
    x, w = (torch.empty(k, d, dtype=t, device="cuda") for k in (n, rows))
    for k, m in enumerate((x, w)):
        for i in range(0, m.shape[0], 10000):
            m[i:i + 10000] = randn(m[i:i + 10000].shape, 100 * k + i, t, 0.1)
    ids = torch.randint(0, rows, (n,), generator=gen(1), device="cuda")
    loss, lse = ce_loss(x, w, ids)
    at = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
    z = torch.cat([x[at].double() @ w[i:i + 10000].double().t() for i in range(0, rows, 10000)], 1)
    want = torch.logsumexp(z, 1)
    bound = 16400 * 2.0 ** -24 * 2.0 * 0.01 * 16384 + 2.0 ** -23 * (64 + rows / 2048 + 20)
    near(lse[at], want, bound)
    dloss = randn((n,), 2)
    dx, dw = ce_grad(x, w, ids, 1.0, lse, dloss, t)
    q = torch.exp(z - lse[at].double()[:, None])
    q[torch.arange(5, device="cuda"), ids[at]] -= 1
    q *= dloss[at].double()[:, None]
    want = sum(q[:, i:i + 10000] @ w[i:i + 10000].double() for i in range(0, rows, 10000))
    size = sum(q[:, i:i + 10000].abs() @ w[i:i + 10000].double().abs() for i in range(0, rows, 10000))
    near(dx[at], want, (2.0 ** -8 + 2 * bound) * size + 2.0 ** -8 * want.abs() + 2.0 ** -133)
    v = torch.tensor([0, rows // 2, rows - 1], device="cuda")
    want, size = torch.zeros(3, d, dtype=torch.float64, device="cuda"), torch.zeros(3, d, dtype=torch.float64, device="cuda")
    for i in range(0, n, 10000):
        xs = x[i:i + 10000].double()
        q = torch.exp(xs @ w[v].double().t() - lse[i:i + 10000].double()[:, None])
        q -= (ids[i:i + 10000, None] == v[None]).double()
        q *= dloss[i:i + 10000].double()[:, None]
        want += q.t() @ xs
        size += q.abs().t() @ xs.abs()
    near(dw[v], want, (2.0 ** -8 + 2 * bound) * size + 2.0 ** -8 * want.abs() + 2.0 ** -133)


# ---- together -------------------------------------------------------------

class Step:
    """A small model's training step made of the library's calls: lookup from qwZ
    codes, a gated layer, the head (the same table), and every gradient into one
    clipped list.  torch does the three plain projections."""

    def __init__(self, n=500, dim=128, ffn=320, rows=1003, block=128, seed=1):
        bf = torch.bfloat16
        self.shape = n, dim, ffn, rows
        self.block = block
        self.wg, self.wu = randn((ffn, dim), seed, bf, 0.1), randn((ffn, dim), seed + 1, bf, 0.1)
        self.wd = randn((dim, ffn), seed + 2, bf, 0.1)
        self.codes, self.scales, _ = quantized(randn((rows, dim), seed + 3, bf, 0.1), 2048)
        self.ids = torch.randint(-3, rows, (n,), generator=gen(seed + 4), device="cuda")
        self.next = torch.roll(self.ids, -1)
        self.dloss = torch.full((n,), 1.0 / n, device="cuda")

        def e(*s, dt=bf):
            return torch.zeros(*s, dtype=dt, device="cuda")

        i8, f32 = torch.int8, torch.float32
        self.x, self.gate, self.up, self.h, self.y = e(n, dim), e(n, ffn), e(n, ffn), e(n, ffn), e(n, dim)
        self.xk, self.xs = e(n, dim, dt=i8), e(-(-n * dim // block), dt=f32)
        self.kept = (e(n * ffn, dt=i8), e(-(-n * ffn // block), dt=f32), e(n * ffn, dt=i8), e(-(-n * ffn // block), dt=f32))
        self.hk, self.hs = e(n, ffn, dt=i8), e(-(-n * ffn // block), dt=f32)
        self.loss, self.lse = e(n, dt=f32), e(n, dt=f32)
        self.dy, self.dh, self.dg, self.du, self.dx = e(n, dim), e(n, ffn), e(n, ffn), e(n, ffn), e(n, dim)
        self.d_wg, self.d_wu, self.d_wd = e(ffn, dim, dt=f32), e(ffn, dim, dt=f32), e(dim, ffn, dt=f32)
        self.d_table = e(rows, dim, dt=f32)
        u8 = torch.uint8
        self.w1 = e(zq.ce_loss_workspace(n, rows, dim), dt=u8)
        self.w2 = e(zq.ce_grad_workspace(n, rows, dim), dt=u8)
        self.w3 = e(max(zq.linear_grad_workspace(n, ffn, dim), zq.linear_grad_workspace(n, dim, ffn)), dt=u8)
        self.w4 = e(zq.embed_grad_workspace(n, rows, dim), dt=u8)
        grads = (self.d_wg, self.d_wu, self.d_wd, self.d_table)
        self.table = zq.GradSegmentTable([(g, g) for g in grads])
        self.w5 = e(zq.grad_sumsq_workspace(4), dt=u8)
        self.sumsq, self.norm = e(1, dt=torch.float64), e(1, dt=f32)

    def run(self, clip=1e9):
        b = self.block
        zq.zq_embed_lookup_int8(self.codes, self.scales, 2048, self.ids, 1.0, self.x)
        zq.zq_quant_int8(self.x, b, self.xk, self.xs)
        torch.matmul(self.x, self.wg.t(), out=self.gate)
        torch.matmul(self.x, self.wu.t(), out=self.up)
        zq.zq_swiglu_int8(self.gate, self.up, b, self.h, *self.kept)
        torch.matmul(self.h, self.wd.t(), out=self.y)
        zq.zq_ce_loss_int8(self.y, self.codes, self.scales, 2048, self.next, 1.0, self.loss, self.lse, self.w1)
        zq.zq_ce_grad_int8(self.y, self.codes, self.scales, 2048, self.next, 1.0, self.lse, self.dloss, self.dy,
                           self.d_table, zq.ZQ_GRAD_WRITE, self.w2)
        torch.matmul(self.dy, self.wd, out=self.dh)
        zq.zq_swiglu_grad_int8(*self.kept, b, self.dh, self.dg, self.du, h=self.h)
        zq.zq_quant_int8(self.h, b, self.hk, self.hs)
        zq.zq_linear_grad_int8(self.dy, self.hk, self.hs, b, self.d_wd, zq.ZQ_GRAD_WRITE, self.w3)
        zq.zq_linear_grad_int8(self.dg, self.xk, self.xs, b, self.d_wg, zq.ZQ_GRAD_WRITE, self.w3)
        zq.zq_linear_grad_int8(self.du, self.xk, self.xs, b, self.d_wu, zq.ZQ_GRAD_WRITE, self.w3)
        torch.matmul(self.dg, self.wg, out=self.dx)
        self.dx.addmm_(self.du, self.wu)
        zq.zq_embed_grad(self.dx, self.ids, 1.0, self.d_table, zq.ZQ_GRAD_ADD, self.w4)
        zq.zq_grad_sumsq_batched(self.table, self.sumsq, self.w5)
        zq.zq_grad_clip_batched(self.table, self.sumsq, clip, norm=self.norm)

    def outputs(self):
        return [x.clone() for x in (self.loss, self.d_wg, self.d_wu, self.d_wd, self.d_table, self.norm)]


def test_a_training_step_of_these_calls():
    s = Step()
    s.run()
    n, dim, ffn, rows = s.shape
    table = held(s.codes, s.scales, 2048).requires_grad_()
    wg, wu, wd = (w.double().requires_grad_() for w in (s.wg, s.wu, s.wd))
    there = (s.ids >= 0)
    x = torch.where(there[:, None], table[s.ids.clamp(min=0)], 0.0)
    y = (torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())) @ wd.t()
    z = y @ table.t()
    counted = s.next >= 0
    loss = torch.where(counted, torch.logsumexp(z, 1) - z.gather(1, s.next.clamp(min=0)[:, None])[:, 0], 0.0)
    (loss / n).sum().backward()
    # bf16 activations (2^-8 each, over a handful of layers) and activations in 8 bits (a 1/254 of their block's
    # largest value, 3 to 4 times the typical one): a few percent of a gradient's norm.
    assert float((s.loss.double() - loss.detach()).abs().max()) < 0.1
    for got, want in ((s.d_wg, wg), (s.d_wu, wu), (s.d_wd, wd), (s.d_table, table)):
        assert float((got.double() - want.grad).norm() / want.grad.norm()) < 0.05
    want = torch.cat([w.grad.reshape(-1) for w in (wg, wu, wd, table)]).norm()
    assert abs(float(s.norm) / float(want) - 1) < 0.05


def test_a_captured_step_replays_to_the_eager_results():
    a, b = Step(seed=1), Step(seed=50)
    want = []
    for s in (a, b):
        s.run()
        want.append(s.outputs())
    side = torch.cuda.Stream()
    graphs = []
    for s in (a, b):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    eager = Step(seed=90)
    for _ in range(4):
        for s, g, w in zip((a, b), graphs, want):
            for x in s.outputs():
                x.zero_()
            s.loss.fill_(NAN)
            s.d_table.fill_(NAN)
            g.replay()
            eager.run()
            torch.cuda.synchronize()
            for x, y in zip(s.outputs(), w):
                same(x, y)


def test_two_graphs_may_share_a_workspace_in_turn():
    n, d, rows = 600, 128, 900
    ws = torch.empty(zq.ce_grad_workspace(n, rows, d, 256), dtype=torch.uint8, device="cuda")
    graphs, outs, want = [], [], []
    for k in range(2):
        x, w, ids, there = ce_inputs(n, d, rows, "bf16", 10 * k, 20)
        lse, dloss = exact_lse(x, w, ids, there, 1.0), randn((n,), k)
        dx, dw = torch.empty_like(x), torch.empty_like(w)

        def run():
            zq.zq_ce_grad(x, w, ids, 1.0, lse, dloss, dx, dw, zq.ZQ_GRAD_WRITE, ws, piece=256)

        run()
        want.append((dx.clone(), dw.clone()))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append((g, x, w, ids, lse, dloss))
        outs.append((dx, dw))
    for _ in range(3):
        for (g, *_rest), out, w in zip(graphs, outs, want):
            for o in out:
                o.fill_(NAN)
            g.replay()
            ws.fill_(0xFF)                           # what lies there between calls means nothing
            torch.cuda.synchronize()
            for o, v in zip(out, w):
                same(o, v)


def test_calls_on_several_streams_at_once():
    steps = [Step(seed=k) for k in (1, 20, 40)]
    want = []
    for s in steps:
        s.run()
        want.append(s.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for x, y in zip(s.outputs(), w):
                same(x, y)


def test_empty_calls():
    f, h, i8 = (torch.empty(0, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16, torch.int8))
    ids, ws = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    zq.zq_swiglu_int8(h, h, 32, h, i8, f, i8, f)
    zq.zq_swiglu_grad_int8(i8, f, i8, f, 32, h, h, h)
    w = randn((5, 9), 1, torch.bfloat16)
    zq.zq_ce_loss(h, w, ids, 1.0, f, f, ws)
    for t in T.values():
        for mode in (zq.ZQ_GRAD_WRITE, zq.ZQ_GRAD_ADD):
            old = randn((5, 9), 2, t)
            out = Out((5, 9), t, old)
            zq.zq_ce_grad(h, w, ids, 1.0, f, f, h, out.t, mode, ws)
            assert torch.equal(out.check(), old if mode == zq.ZQ_GRAD_ADD else torch.zeros_like(old))
            out = Out((5, 9), t, old)
            zq.zq_linear_grad_int8(h.view(0, 5), i8.view(0, 9), f, 32, out.t, mode, ws)
            assert torch.equal(out.check(), old if mode == zq.ZQ_GRAD_ADD else torch.zeros_like(old))


def test_another_device_or_a_foreign_tensor_is_refused():
    x, w, ids, _ = ce_inputs(4, 64, 10, "bf16", 1)
    f = torch.empty(4, device="cuda")
    ws = torch.empty(zq.ce_loss_workspace(4, 10, 64), dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError, match="w has dtype"):
        zq.zq_ce_loss(x, w.half(), ids, 1.0, f, f.clone(), ws)
    with pytest.raises(ValueError, match="workspace holds"):
        zq.zq_ce_loss(x, w, ids, 1.0, f, f.clone(), ws[:-1])
    with pytest.raises(zq.ZQError, match="overlap"):
        zq.zq_ce_loss(x, w, ids, 1.0, f, f, ws)
    with pytest.raises(ValueError, match="contiguous"):
        zq.zq_ce_loss(x, w.t().contiguous().t(), ids, 1.0, f, f.clone(), ws)
