"""SwiGLU from int8 activations where factors are far from 1, and over many elements,
on the GPU, against the formulas in 64 bits.

A gradient in binary32 has the sigmoid's error (2^-22 or less), two sums' and four
products' half steps of 2^-24: 2^-20 of the sizes together; then half a step of the
output's type.
"""
import pytest
import torch

from weight_communication_zero_amd import zq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def near(got, want, bound, what):
    assert bool(got.isfinite().all()), what + ": not finite"
    off = (got.double() - want).abs() - bound
    assert float(off.max()) <= 0, (what, float(off.max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_of_large_factors(dtype):
    """dh times up is past binary32's range, the gradients are not: gates from -30 to -87
    bring them back, and one of -120 leaves 0 or next to it."""
    n, block = 256, 32
    gates = [-30.0, -40.0, -50.0, -60.0, -70.0, -80.0, -85.0, -120.0]
    k = torch.full((n,), 127, dtype=torch.int8, device="cuda")
    k[1::2] = 100
    gs = torch.tensor(gates, device="cuda") / 127
    us = torch.full((n // block,), 1e20 / 127, device="cuda")
    dh = (torch.linspace(1, 9, n, device="cuda") * 1e20).to(dtype)
    dg, du, h = (torch.full_like(dh, 77.0) for _ in range(3))
    zq.zq_swiglu_grad_int8(k, gs, k, us, block, dh, dg, du, h=h)
    at = torch.arange(n, device="cuda") // block
    g, u = (k.float() * gs[at]).double(), (k.float() * us[at]).double()
    s, r = torch.special.expit(g), torch.special.expit(-g)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    d = dh.double()
    # What a sigmoid below 2^-126, taken as 0, leaves out.
    tiny = 2.0 ** -126 * (1 + g.abs())
    want = d * u * s * (1 + g * r)
    near(dg, want, 2.0 ** -20 * (d * u * s).abs() * (1 + (g * r).abs()) + half * want.abs() + tiny * d * u, "dgate")
    want = d * g * s
    near(du, want, (2.0 ** -20 + half) * want.abs() + tiny * d, "dup")
    want = g * s * u
    near(h, want, (2.0 ** -20 + half) * want.abs() + tiny * u, "h")


@pytest.mark.parametrize("n,block", [(389304, 2048), (1 << 22, 128)])
def test_many_fp32_codes_are_those_of_ieee_scales(n, block):
    """absmax / 127 and value / scale are IEEE quotients.  (A scale formed as a product with
    1 / 127 differs in the last place of 4 % of them, and then keeps another code for about
    one value in a million.)  64-bit quotients rounded to 32 bits are the IEEE ones: 53 bits
    are more than twice 24 and 2."""
    gen = torch.Generator(device="cuda").manual_seed(386)
    gate = torch.randn(n, generator=gen, device="cuda") * 1.5
    up, dh = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda") * 1e-2
    h, dg, du = (torch.empty(n, device="cuda") for _ in range(3))
    blocks = -(-n // block)
    kept = [torch.empty(n, dtype=torch.int8, device="cuda"), torch.empty(blocks, device="cuda"),
            torch.empty(n, dtype=torch.int8, device="cuda"), torch.empty(blocks, device="cuda")]
    zq.zq_swiglu_int8(gate, up, block, h, *kept)
    zq.zq_swiglu_grad_int8(*kept, block, dh, dg, du)
    held = []
    for x, codes, scales in ((gate, *kept[:2]), (up, *kept[2:])):
        v = torch.zeros(blocks * block, dtype=torch.float64, device="cuda")
        v[:n] = x
        v = v.view(-1, block)
        s = (v.abs().amax(1, keepdim=True) / torch.tensor(127.0, dtype=torch.float64, device="cuda")).float()
        k = (v / s.double()).float().double().round()
        assert torch.equal(scales, s[:, 0])
        assert torch.equal(codes.double(), k.view(-1)[:n])
        held.append((k * s.double()).float().double().view(-1)[:n])
    g, u = held
    s, r = torch.special.expit(g), torch.special.expit(-g)
    size = (dh.double() * u * s).abs() * (1 + (g * r).abs())
    near(dg, dh.double() * u * s * (1 + g * r), 2.0 ** -20 * size + 2.0 ** -149, "dgate")
    near(du, dh.double() * g * s, 2.0 ** -20 * (dh.double() * g * s).abs() + 2.0 ** -149, "dup")
