"""The 64-bit reference of the gated recurrence and the residual norm: gradients
against differences of the forward, and what the definitions say."""
import pytest
import torch

import recurrent_reference as R

F64 = torch.float64


def differences(f, t, at, h=1e-6):
    a, b = t.clone(), t.clone()
    a.view(-1)[at] += h
    b.view(-1)[at] -= h
    return float(f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("reset", [None, "random", "edges"])
@pytest.mark.parametrize("z", [False, True])
def test_recurrence_gradients_against_differences(z, reset):
    i = R.rec_inputs(3, F64, 2, 40, 3, z=z, reset=reset)

    def loss(**kw):
        v = dict(i, **kw)
        out, last, _ = R.rec_fwd(v["x"], v["r"], v["i"], v["A"], v["z"], v["h0"], v["reset"])
        return (out * i["dout"]).sum() + (last * i["dlast"]).sum()
    got, _ = R.rec_bwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["dout"], i["h0"], i["dlast"],
                       i["reset"])
    assert set(got) == {"dx", "dr", "di", "dA", "dh0"} | ({"dz"} if z else set())
    for name, g in got.items():
        t = i[name[1:]]
        for at in range(0, t.numel(), max(1, t.numel() // 11)):
            d = differences(lambda q: loss(**{name[1:]: q}), t, at)
            assert abs(d - float(g.reshape(-1)[at])) < 1e-7 * (1 + abs(d)), (name, at)


def test_recurrence_by_definition():
    i = R.rec_inputs(4, F64, 1, 30, 5, z=False, reset="edges")
    out, last, before = R.rec_fwd(i["x"], i["r"], i["i"], i["A"], None, i["h0"], i["reset"])
    assert torch.equal(out[:, -1], last) and torch.equal(before[:, 1:], out[:, :-1])
    cut = out.clone()
    # what lies before a flag does not reach what lies behind it
    j = dict(i, x=i["x"].clone(), h0=i["h0"] + 1)
    j["x"][:, :16] = 7.0
    out, _, _ = R.rec_fwd(j["x"], j["r"], j["i"], j["A"], None, j["h0"], j["reset"])
    assert torch.equal(out[:, 16:], cut[:, 16:]) and not torch.equal(out[:, :16], cut[:, :16])
    # a gate that is shut keeps the state and lets nothing in
    r = torch.full_like(i["r"], -800.0)
    out, last, _ = R.rec_fwd(i["x"], r, i["i"], i["A"], None, i["h0"], None)
    assert torch.equal(last, i["h0"])


@pytest.mark.parametrize("weight", [False, True])
def test_norm_gradients_against_differences(weight):
    i = R.norm_inputs(5, F64, F64, 3, 7, weight=weight)
    res = i["x"] + i["residual"]

    def loss(res, w):
        y = res / torch.sqrt(res.square().mean(-1, keepdim=True) + 1e-3)
        return ((y if w is None else y * w) * i["dout"]).sum() + (res * i["dres"]).sum()
    d, dw, _ = R.norm_bwd(res, i["weight"], i["dout"], i["dres"], 1e-3)
    for at in range(res.numel()):
        e = differences(lambda q: loss(q, i["weight"]), res, at)
        assert abs(e - float(d.reshape(-1)[at])) < 1e-7 * (1 + abs(e))
    if weight:
        for at in range(7):
            e = differences(lambda q: loss(res, q), i["weight"], at)
            assert abs(e - float(dw[at])) < 1e-7 * (1 + abs(e))
