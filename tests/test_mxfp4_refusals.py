"""Calls of the MXFP4 operators that are refused (on the host; nothing is launched)."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import gemv_int4_quantize_amd as w4


def _rows(n, k):
    p = (k + 127) // 128 * 128
    return w4.MXFP4Rows(torch.zeros(n, p // 2, dtype=torch.uint8), torch.zeros(n, p // 32, dtype=torch.uint8), n, k)


def _calls():
    """Each product with a tensor in the place that a derivative could be wanted of."""
    w, x, b = _rows(8, 64), torch.zeros(2, 64), torch.zeros(8)
    return {"mm_mxfp4": lambda t: w4.mm_mxfp4(t, w), "mm_mxfp4 bias": lambda t: w4.mm_mxfp4(x, w, bias=t),
            "mm_mxfp4_split": lambda t: w4.mm_mxfp4_split(t, w, [torch.zeros(2, 8)]),
            "mm_mxfp4_split bias": lambda t: w4.mm_mxfp4_split(_rows(2, 64), w, [torch.zeros(2, 8)], bias=t),
            "mm_mxfp4_t": lambda t: w4.mm_mxfp4_t(t, w), "sum_rows": lambda t: w4.mxfp4.sum_rows(t)}, {
            "mm_mxfp4": x, "mm_mxfp4 bias": b, "mm_mxfp4_split": x, "mm_mxfp4_split bias": b, "mm_mxfp4_t": torch.zeros(2, 8),
            "sum_rows": x}


@pytest.mark.parametrize("name", _calls()[0])
def test_no_derivative_is_lost(name):
    calls, inputs = _calls()
    call, t = calls[name], inputs[name]
    with pytest.raises(RuntimeError, match=f"{name.split()[0]} has no derivative"):
        call(t.clone().requires_grad_())
    with fwd.dual_level(), torch.no_grad():
        with pytest.raises(RuntimeError, match="no derivative"):
            call(fwd.make_dual(t, torch.ones_like(t)))
    # what loses nothing goes on, here to the check of devices
    with pytest.raises(ValueError, match="HIP device"):
        call(t)
    with torch.no_grad(), pytest.raises(ValueError, match="HIP device"):
        call(t.clone().requires_grad_())


@pytest.mark.parametrize("gate_up,down", [((4, 40, 64), (2, 64, 40)), ((2, 160, 64), (4, 64, 40)), ((4, 80, 64), (4, 40, 64)),
                                          ((1, 320, 64), (4, 64, 40)), ((4, 80, 64), (1, 256, 40)), ((8, 40, 64), (4, 64, 40))])
def test_experts_of_other_shapes(monkeypatch, gate_up, down):
    """Weights whose rows add up, but not expert by expert."""
    monkeypatch.setattr(w4.mxfp4, "quantize_mxfp4", lambda t: _rows(*t.shape))
    assert w4.MXFP4MoE.from_weight(torch.zeros(4, 80, 64), torch.zeros(4, 64, 40), 2).experts == 4
    with pytest.raises(ValueError, match="are wanted"):
        w4.MXFP4MoE.from_weight(torch.zeros(gate_up), torch.zeros(down), 1)


def test_logits_of_other_tokens(monkeypatch):
    """As many tokens, in another order of the leading sizes, are not the same tokens."""
    seen = []
    monkeypatch.setattr(w4.mxfp4, "moe_mxfp4", lambda x, z, *_: seen.append((x.shape, z.shape)) or x)
    layer = w4.MXFP4MoE(_rows(4 * 2 * 40, 64), _rows(4 * 64, 40), 2)
    for x, z in (((2, 3, 64), (3, 2, 4)), ((2, 3, 64), (1, 6, 4)), ((6, 1, 64), (2, 3, 4))):
        with pytest.raises(ValueError, match="same tokens"):
            layer(torch.zeros(x), torch.zeros(z))
    for x, z in (((2, 3, 64), (2, 3, 4)), ((2, 3, 64), (6, 4)), ((6, 64), (2, 3, 4)), ((64,), (4,)), ((64,), (1, 4)), ((6, 64), (6, 4))):
        assert layer(torch.zeros(x), torch.zeros(z)).shape == x
        t = 1 if len(x) == 1 else 6
        assert seen[-1] == ((t, 64), (t, 4))
