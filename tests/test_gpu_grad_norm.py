"""The global gradient norm and clipping on the GPU.

The sum of squares is compared with math.fsum of the exact squares (a square of
a binary32 value is exact in binary64): at these sizes no chain of additions is
longer than 2^12, so the relative error is below 2^-41.  The clip is compared
bit for bit with the formula applied to the device's own sum on the host
(binary64 square root, sum and quotient, one rounding to binary32, a binary32
product, one rounding to the type).
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from weight_communication_zero_amd import zq

pytestmark = pytest.mark.gpu

T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def tensors(sizes, dtype, seed, std=1e-3):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(dtype) for n in sizes]


def exact_sumsq(ts):
    return math.fsum(float(v) for t in ts for v in t.double().square().tolist())


def sumsq_of(gs, accumulate=None):
    q = torch.full((1,), math.nan if accumulate is None else accumulate, dtype=torch.float64, device="cuda")
    need = zq.grad_sumsq_workspace(len(gs))
    ws = torch.full((need + GUARD,), 0xAB, dtype=torch.uint8, device="cuda")
    zq.zq_grad_sumsq_batched([(g, None) for g in gs], q, ws[:need], accumulate=accumulate is not None)
    assert bool((ws[need:] == 0xAB).all())
    return q


def clip_factor(q, max_norm, eps):
    with np.errstate(all="ignore"):
        c = np.float64(np.float32(max_norm)) / (np.sqrt(np.float64(q)) + np.float64(np.float32(eps)))
    return np.float32(1.0) if c >= 1.0 else np.float32(c)


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


LISTS = {
    "empty": [], "zero": [0, 0], "one": [1], "odd": [3, 0, 17, 1023, 1024, 1025], "tile": [2047, 2048, 2049, 4096],
    "one_wg": [1024 * 64], "past_one_wg": [1024 * 64 + 1], "one_wg_16bit": [2048 * 64, 0], "past_16bit": [2048 * 64, 1],
    "128_segments": [65] * 128, "129_segments": [65] * 129, "300_segments": list(range(300)),
    "144_segments": [70] * 144, "145_segments": [70] * 145, "192_segments": [9] * 192, "193_segments": [9] * 193,
    "400_with_empty": [0, 33] * 200,
    "mid": [100003, 7, 65536, 99999, 1], "large_first": [3_000_001, 5, 9],
}


@pytest.mark.parametrize("dt", list(T))
@pytest.mark.parametrize("name", list(LISTS))
def test_sumsq(name, dt):
    ts = tensors(LISTS[name], T[dt], len(name))
    gs = [t.cuda() for t in ts]
    q = sumsq_of(gs)
    exact = exact_sumsq(ts)
    assert abs(float(q) - exact) <= 2.0 ** -41 * exact
    assert float(sumsq_of(gs)) == float(q)  # the same bits again
    added = float(sumsq_of(gs, accumulate=3.0))
    assert added == 3.0 + float(q)


def test_sumsq_of_values_whose_squares_leave_binary32():
    for v, dt in ((1e30, "fp32"), (1e-30, "fp32"), (2.0 ** -149, "fp32"), (3e38, "fp32"), (1e30, "bf16"),
                  (1e-38, "bf16"), (65504.0, "fp16"), (6e-8, "fp16")):
        t = torch.full((5000,), v, dtype=T[dt])
        q = float(sumsq_of([t.cuda()]))
        exact = 5000 * float(t[0]) ** 2
        assert exact > 0 and abs(q - exact) <= 2.0 ** -41 * exact


@pytest.mark.parametrize("at", [0, 1500, 4999])
def test_sumsq_of_infinities_and_nan(at):
    for dt in T.values():
        t = torch.ones(5000, dtype=dt)
        t[at] = -math.inf
        assert float(sumsq_of([t.cuda()])) == math.inf
        t[at] = math.nan
        assert math.isnan(float(sumsq_of([t.cuda()])))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_norm,eps", [(0.5, 1e-6), (1e9, 1e-6), (0.0, 1e-6), (0.1, 0.0), (1e-30, 0.5)])
@pytest.mark.parametrize("dt", list(T))
@pytest.mark.parametrize("name", ["one", "odd", "tile", "129_segments", "144_segments", "145_segments",
                                  "300_segments", "400_with_empty", "mid"])
def test_clip(name, dt, max_norm, eps, in_place):
    ts = tensors(LISTS[name], T[dt], 3, std=1.0)
    bufs = [torch.cat([t.cuda(), torch.full((GUARD,), 7.0, dtype=t.dtype, device="cuda")]) for t in ts]
    gs = [b[:t.numel()] for b, t in zip(bufs, ts)]
    if in_place:
        obufs, outs = bufs, gs
    else:
        obufs = [torch.full_like(b, 7.0) for b in bufs]
        outs = [b[:t.numel()] for b, t in zip(obufs, ts)]
    q = sumsq_of(gs)
    norm = torch.full((3,), -1.0, device="cuda")
    zq.zq_grad_clip_batched(zip(gs, outs), q, max_norm, eps, norm=norm[1:2])
    assert norm.tolist() == [-1.0, float(np.float32(np.sqrt(float(q)))), -1.0]
    c = torch.tensor(clip_factor(float(q), max_norm, eps))
    for t, o, ob, g in zip(ts, outs, obufs, gs):
        assert torch.equal(bits(o), bits((t.float() * c).to(t.dtype)))
        assert bool((ob[t.numel():] == 7).all())
        if not in_place:
            assert torch.equal(bits(g), bits(t))


@pytest.mark.parametrize("value", [math.inf, math.nan, 0.0])
def test_clip_by_a_norm_that_is_no_ordinary_number(value):
    """inf: finite values become 0 and infinities NaN; NaN: everything; 0: unchanged."""
    for dt in T.values():
        t = torch.tensor([1.0, -2.0, 0.0, math.inf, 3.0], dtype=dt)
        g, out = t.cuda(), torch.empty(5, dtype=dt, device="cuda")
        q = torch.full((1,), value, dtype=torch.float64, device="cuda")
        norm = torch.empty(1, device="cuda")
        zq.zq_grad_clip_batched([(g, out)], q, 1.0, norm=norm)
        exp = (t.float() * torch.tensor(clip_factor(value, 1.0, 1e-6))).to(dt)
        assert torch.equal(out.cpu().isnan(), exp.isnan())
        assert torch.equal(bits(out)[~exp.isnan()], bits(exp)[~exp.isnan()])
        assert torch.equal(norm.cpu().isnan(), torch.tensor([math.isnan(value)]))


def test_clip_without_segments_writes_the_norm():
    q = torch.full((1,), 9.0, dtype=torch.float64, device="cuda")
    norm = torch.zeros(1, device="cuda")
    zq.zq_grad_clip_batched([], q, 1.0, norm=norm)
    assert float(norm) == 3.0
    zq.zq_grad_clip_batched([], q, 1.0)  # and nothing without one


def test_two_dtypes_and_a_sum_over_ranks():
    """A bf16 list added to an fp32 list, and the sum of two ranks' sums: the
    clip sees the norm of all of it."""
    a, b = tensors([5000, 33], torch.float32, 1, 1.0), tensors([700], torch.bfloat16, 2, 1.0)
    q = sumsq_of([t.cuda() for t in a])
    ws = torch.empty(zq.grad_sumsq_workspace(1), dtype=torch.uint8, device="cuda")
    gb = [t.cuda() for t in b]
    zq.zq_grad_sumsq_batched([(t, None) for t in gb], q, ws, accumulate=True)
    exact = exact_sumsq(a + b)
    assert abs(float(q) - exact) <= 2.0 ** -40 * exact
    q = q + q  # two ranks with equal shards
    zq.zq_grad_clip_batched([(t, t) for t in gb], q, 1.0)
    c = torch.tensor(clip_factor(float(q), 1.0, 1e-6))
    assert torch.equal(bits(gb[0]), bits((b[0].float() * c).bfloat16()))


def test_offsets_past_2_to_32():
    n = (1 << 32) + 4099
    g = torch.full((n,), 0.5, dtype=torch.float16, device="cuda")
    q = sumsq_of([g])
    assert float(q) == n * 0.25  # every partial sum is exact
    g[-3:] = 4.0
    zq.zq_grad_clip_batched([(g, g)], q, 1024.0, 0.0)
    c = clip_factor(n * 0.25, 1024.0, 0.0)
    half = torch.tensor(c * np.float32(0.5)).half()
    assert bool((g[:-3] == half.cuda()).all())
    assert g[-3:].tolist() == [float(torch.tensor(c * np.float32(4.0)).half())] * 3


def test_refusals_of_the_binding():
    g = torch.zeros(64, device="cuda")
    q = torch.zeros(1, dtype=torch.float64, device="cuda")
    ws = torch.empty(zq.grad_sumsq_workspace(1), dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError, match="share one"):
        zq.GradSegmentTable([(g, None), (g.half(), None)])
    with pytest.raises(TypeError, match="out has dtype"):
        zq.GradSegmentTable([(g, g.half())])
    with pytest.raises(ValueError, match="out holds"):
        zq.GradSegmentTable([(g, g[:32])])
    with pytest.raises(ValueError, match="workspace holds"):
        zq.zq_grad_sumsq_batched([(g, None)], q, ws[:64])
    with pytest.raises(TypeError, match="sumsq has dtype"):
        zq.zq_grad_sumsq_batched([(g, None)], q.float(), ws)
    with pytest.raises(zq.ZQError, match="NULL"):
        zq.zq_grad_clip_batched([(g, None)], q, 1.0)
    with pytest.raises(zq.ZQError, match="ALIAS"):
        zq.zq_grad_clip_batched([(g[:32], g[16:48])], q, 1.0)
    with pytest.raises(zq.ZQError, match="SIZE"):
        zq.zq_grad_clip_batched([(g, g)], q, -1.0)


def step(s, tables):
    """The set as a training step uses it: qwZ codes of the table, lookup from
    them, the table's gradient (bf16 accumulator and fp32), EF quantize and
    reduce of the fp32 gradient, the norm over both and the clip."""
    zq.zq_quant_int8(s["w"], 128, s["c8"], s["s8"])
    zq.zq_embed_lookup_int8(s["c8"].view(ROWS, DIM), s["s8"], 128, s["ids"], 3.0, s["x"])
    zq.zq_embed_grad(s["x"], s["ids"], 3.0, s["acc"], zq.ZQ_GRAD_ADD_SR, s["ws"], seed=99, counter_base=5)
    zq.zq_embed_grad(s["x"], s["ids"], 3.0, s["dw"], zq.ZQ_GRAD_WRITE, s["ws"])
    zq.zq_quantize_ef_int4(s["dw"], s["ef"], 128, 0.9, 1.0, s["c4"], s["s4"])
    zq.zq_dequant_reduce([s["c4"]], [s["s4"]], ROWS * DIM, 128, 1.0, out=s["red"])
    zq.zq_grad_sumsq_batched(tables[0], s["q"], s["nws"])
    zq.zq_grad_sumsq_batched(tables[1], s["q"], s["nws"], accumulate=True)
    zq.zq_grad_clip_batched(tables[0], s["q"], 0.25, norm=s["norm"])
    zq.zq_grad_clip_batched(tables[1], s["q"], 0.25)


ROWS, DIM, NTOK = 96, 136, 333


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g, device="cuda")
    n = ROWS * DIM
    s = {"w": r(n).mul_(0.02).bfloat16(), "c8": torch.zeros(n, dtype=torch.int8, device="cuda"),
         "s8": torch.zeros(-(-n // 128), device="cuda"),
         "ids": torch.randint(-2, ROWS, (NTOK,), generator=g, device="cuda", dtype=torch.int32),
         "x": torch.zeros(NTOK, DIM, dtype=torch.bfloat16, device="cuda"), "acc": r(ROWS, DIM).bfloat16(),
         "dw": torch.zeros(ROWS, DIM, device="cuda"), "ef": torch.zeros(n, device="cuda"),
         "c4": torch.zeros(n // 2, dtype=torch.uint8, device="cuda"), "s4": torch.zeros(-(-n // 128), device="cuda"),
         "red": torch.zeros(n, device="cuda"), "q": torch.zeros(1, dtype=torch.float64, device="cuda"),
         "norm": torch.zeros(1, device="cuda"),
         "ws": torch.empty(zq.embed_grad_workspace(NTOK, ROWS, DIM), dtype=torch.uint8, device="cuda"),
         "nws": torch.empty(zq.grad_sumsq_workspace(1), dtype=torch.uint8, device="cuda")}
    s["clipped"] = torch.zeros(n, device="cuda")
    tables = [zq.GradSegmentTable([(s["red"], s["clipped"])]), zq.GradSegmentTable([(s["acc"], s["acc"])])]
    return s, tables


def test_a_step_of_all_of_them():
    s, tables = make(1)
    w, ids, acc = s["w"].cpu(), s["ids"].cpu().long(), s["acc"].cpu()
    step(s, tables)
    torch.cuda.synchronize()
    wb = w.view(torch.int16).numpy().view(np.uint16)
    c8, s8 = O.quant_int8(wb, 128)
    table = torch.from_numpy(O.dequant_int8(c8, s8, 128)).view(ROWS, DIM)
    there = ids >= 0
    x = torch.where(there[:, None], table[ids.clamp(min=0)] * 3.0, torch.zeros(())).bfloat16()
    assert torch.equal(s["x"].cpu(), x)
    exact = torch.zeros(ROWS, DIM, dtype=torch.float64).index_add_(0, ids[there], x[there].double() * 3)
    size = torch.zeros(ROWS, DIM, dtype=torch.float64).index_add_(0, ids[there], x[there].double().abs() * 3)
    bound = (torch.bincount(ids[there], minlength=ROWS).double()[:, None] + 3) * 2.0 ** -24 * size
    assert bool(((s["dw"].cpu().double() - exact).abs() <= bound).all())
    # From the kernel's own gradient on, the oracle gives the rest bit for bit.
    c4, s4 = O.quantize_ef_int4(s["dw"].cpu().numpy().reshape(-1), np.zeros(ROWS * DIM, np.float32), 128, 0.9, 1.0)
    red = O.dequant_reduce([c4], [s4], ROWS * DIM, 128, 1.0)
    red = torch.from_numpy(red[0] if isinstance(red, tuple) else red)
    assert torch.equal(s["red"].cpu(), red)
    before = (acc.double() + exact)
    n2 = float((red.double() ** 2).sum() + (before ** 2).sum())
    # The accumulator is within one bf16 step of `before`, 2^-7 relative at most.
    assert abs(float(s["norm"]) / math.sqrt(n2) - 1) < 2.0 ** -7
    c = torch.tensor(clip_factor(float(s["q"]), 0.25, 1e-6))
    assert torch.equal(s["clipped"].cpu(), red * c)
    both = (s["clipped"].double() ** 2).sum() + (s["acc"].double() ** 2).sum()
    assert float(both.sqrt()) <= 0.25 * (1 + 2.0 ** -8)


def test_two_graphs_that_share_a_workspace():
    """The step captured twice, on two buffer sets that share both workspaces,
    replayed in turn with eager work between: every replay equals the eager
    step."""
    eager, et = make(2)
    a, at = make(2)
    b, bt = make(3)
    eb, ebt = make(3)
    for k in ("ws", "nws"):
        b[k] = a[k]
    step(*make(9))  # loads every kernel before the capture
    torch.cuda.synchronize()
    graphs = []
    for s, t in ((a, at), (b, bt)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s, t)
        graphs.append(g)
    for i in range(3):
        for g, s, (e, t) in zip(graphs, (a, b), ((eager, et), (eb, ebt))):
            new = torch.randint(-2, ROWS, (NTOK,), device="cuda", dtype=torch.int32)
            for z in (s, e):
                z["ids"].copy_(new)
                z["w"].mul_(1.5)
            g.replay()
            step(e, t)
            torch.cuda.synchronize()
            for k in ("x", "acc", "dw", "ef", "red", "clipped", "q", "norm"):
                assert torch.equal(s[k], e[k]), (i, k)


def test_on_two_streams_at_once():
    """Two steps on two streams, each with its own workspaces."""
    sets = [make(20 + i) for i in range(2)]
    refs = [make(20 + i) for i in range(2)]
    for r in refs:
        step(*r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            step(*s)
    torch.cuda.synchronize()
    for (s, _), (r, _) in zip(sets, refs):
        for k in ("x", "acc", "dw", "red", "clipped", "q", "norm"):
            assert torch.equal(s[k], r[k]), k
