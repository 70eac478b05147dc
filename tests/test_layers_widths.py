"""The binding compares the widths of the layer calls' operands: a tensor with enough
elements but rows of another width is refused, on the host, before anything else is
looked at (CPU tensors of the right widths are refused as such)."""
import pytest
import torch

from weight_communication_zero_amd import zq

BF = torch.bfloat16
GPU = "must be a GPU tensor"


def ce_calls():
    f, ws, ids = torch.zeros(8), torch.zeros(64, dtype=torch.uint8), torch.zeros(8, dtype=torch.int64)
    w, codes = torch.zeros(10, 24, dtype=BF), torch.zeros(10, 24, dtype=torch.int8)
    dx, dw = torch.zeros(8, 24, dtype=BF), torch.zeros(10, 24)

    def loss(x):
        zq.zq_ce_loss(x, w, ids, 1.0, f, f, ws)

    def loss8(x):
        zq.zq_ce_loss_int8(x, codes, f, 32, ids, 1.0, f, f, ws)

    def grad(x, dx=dx, dw=dw):
        zq.zq_ce_grad(x, w, ids, 1.0, f, f, dx, dw, 0, ws)

    def grad8(x, dx=dx, dw=dw):
        zq.zq_ce_grad_int8(x, codes, f, 32, ids, 1.0, f, f, dx, dw, 0, ws)

    return loss, loss8, grad, grad8


def refusal(monkeypatch, call, *args, **kw):
    """What the call's width checks say (w and codes are CPU tensors here; their own
    refusal is left out)."""
    need = zq._need
    monkeypatch.setattr(zq, "_need", lambda name, t, n, d: need(name, t, n, d) if name == "x" else None)
    with pytest.raises(ValueError) as e:
        call(*args, **kw)
    return str(e.value)


@pytest.mark.parametrize("k", range(4))
def test_hidden_states_of_another_width(monkeypatch, k):
    call = ce_calls()[k]
    for shape in ((8, 32), (16, 12), (2, 8, 48), (8, 25), (1, 192), (5, 2, 20)):
        assert refusal(monkeypatch, call, torch.zeros(shape, dtype=BF)) == f"x has {shape[-1]} columns, the projection 24"
    for shape in ((8, 24), (192,), (2, 4, 24), (8, 4, 6), (9, 24)):
        assert GPU in refusal(monkeypatch, call, torch.zeros(shape, dtype=BF))


@pytest.mark.parametrize("k", (2, 3))
def test_gradients_of_another_width(monkeypatch, k):
    call, x = ce_calls()[k], torch.zeros(8, 24, dtype=BF)
    assert refusal(monkeypatch, call, x, dx=torch.zeros(8, 32, dtype=BF)) == "dx has 32 columns, the projection 24"
    assert refusal(monkeypatch, call, x, dw=torch.zeros(24, 10)) == "dw has 10 columns, the projection 24"
    for kw in ({"dx": None}, {"dw": None}, {"dx": torch.zeros(192, dtype=BF), "dw": torch.zeros(240)}):
        assert GPU in refusal(monkeypatch, call, x, **kw)


def test_kept_inputs_of_another_width():
    dy, grad, f = torch.zeros(8, 6, dtype=BF), torch.zeros(6, 24), torch.zeros(8)
    ws = torch.zeros(64, dtype=torch.uint8)
    for shape in ((8, 32), (24, 8), (8, 25)):
        with pytest.raises(ValueError, match=f"codes has {shape[1]} columns, grad 24"):
            zq.zq_linear_grad_int8(dy, torch.zeros(shape, dtype=torch.int8), f, 32, grad, 0, ws)
    for shape in ((8, 24), (192,), (2, 4, 24)):
        with pytest.raises(ValueError, match=GPU):
            zq.zq_linear_grad_int8(dy, torch.zeros(shape, dtype=torch.int8), f, 32, grad, 0, ws)
