"""Outputs of the recurrent block's operators that lie over an input, over one another or
over the workspace are refused, each over each (no GPU: nothing is launched)."""
import ctypes

import pytest

from scan_selective_fwd_amd import _lib

INVALID = 8
B, L, D, POOL = 2, 300, 96, 5
SEQ, STATE, CK = B * L * D * 2, B * D * 4, B * 5 * D * 4      # bytes
RECURRENCE = dict(x=SEQ, r=SEQ, i=SEQ, z=SEQ, A=D * 4, h0=STATE, reset=B * L)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def at(k):      # pointers that are never followed, 16 TiB apart
    return (k + 1) << 44


def pairs(outs, ins):
    return [(o, i) for o in outs for i in ins]


def places(inputs, outputs, out, over):
    """Pointers of all, `out` three times over `over`: at its start, its first bytes over the
    input's last, its last over the input's first."""
    p = {name: at(k) for k, name in enumerate([*inputs, *outputs])}
    for q in (p[over], p[over] + inputs[over] // 16 * 16 - 16, p[over] - outputs[out] + 16):
        yield {**p, out: q}


def shape(seqlen):
    return _lib.RecurrenceShape(batch=B, seqlen=seqlen, dim=D, x_batch_stride=seqlen * D,
                                x_token_stride=D, r_batch_stride=seqlen * D, r_token_stride=D,
                                i_batch_stride=seqlen * D, i_token_stride=D,
                                z_batch_stride=seqlen * D, z_token_stride=D, dtype=1)


FWD = dict(out=SEQ, last=STATE, ck=CK)


@pytest.mark.parametrize("out,over", [p for p in pairs(FWD, RECURRENCE) if p != ("last", "h0")])
def test_recurrence_forward(lib, out, over):
    for p in places(RECURRENCE, FWD, out, over):
        assert forward(lib, p) == INVALID


def forward(lib, p):
    return lib.mamba_gated_recurrence_fwd(
        ctypes.byref(shape(L)), p["x"], p["r"], p["i"], p["A"], p["z"], p["h0"], p["reset"],
        p["out"], p["last"], p["ck"], p.get("ws", at(60)), 1 << 40, None)


def rest(outs, out):
    return {k: v for k, v in outs.items() if k != out}


@pytest.mark.parametrize("out,over", [p for p in pairs(FWD, FWD) if p[0] != p[1]])
def test_recurrence_forward_among_outputs(lib, out, over):
    for p in places({**RECURRENCE, **rest(FWD, out)}, {out: FWD[out]}, out, over):
        assert forward(lib, p) == INVALID


@pytest.mark.parametrize("over", [*RECURRENCE, *FWD])
def test_recurrence_forward_workspace(lib, over):
    n = lib.mamba_gated_recurrence_fwd_workspace_size(ctypes.byref(shape(L)))
    for p in places({**RECURRENCE, **FWD}, {"ws": n // 16 * 16}, "ws", over):
        assert forward(lib, p) == INVALID


BWD_IN = dict(RECURRENCE, dout=SEQ, dlast=STATE, ck=CK)
BWD = dict(dx=SEQ, dr=SEQ, di=SEQ, dz=SEQ, dA=D * 4, dh0=STATE)


@pytest.mark.parametrize("out,over", pairs(BWD, BWD_IN))
def test_recurrence_backward(lib, out, over):
    for p in places(BWD_IN, BWD, out, over):
        assert backward(lib, p) == INVALID


def backward(lib, p):
    return lib.mamba_gated_recurrence_bwd(
        ctypes.byref(shape(L)), p["x"], p["r"], p["i"], p["A"], p["z"], p["h0"], p["reset"],
        p["dout"], p["dlast"], p["ck"], p["dx"], p["dr"], p["di"], p["dA"], p["dz"], p["dh0"],
        p.get("ws", at(60)), 1 << 40, None)


@pytest.mark.parametrize("out,over", [p for p in pairs(BWD, BWD) if p[0] != p[1]])
def test_recurrence_backward_among_outputs(lib, out, over):
    for p in places({**BWD_IN, **rest(BWD, out)}, {out: BWD[out]}, out, over):
        assert backward(lib, p) == INVALID


@pytest.mark.parametrize("over", [*BWD_IN, *BWD])
def test_recurrence_backward_workspace(lib, over):
    n = lib.mamba_gated_recurrence_bwd_workspace_size(ctypes.byref(shape(L)), 1)
    for p in places({**BWD_IN, **BWD}, {"ws": n // 16 * 16}, "ws", over):
        assert backward(lib, p) == INVALID


UPDATE_IN = dict(x=B * D * 2, r=B * D * 2, i=B * D * 2, z=B * D * 2, A=D * 4, slots=B * 4)
UPDATE = dict(out=B * D * 2, state=POOL * D * 4)


@pytest.mark.parametrize("out,over", pairs(UPDATE, UPDATE_IN) + [("out", "state")])
def test_recurrence_update(lib, out, over):
    ins = dict(UPDATE_IN, state=POOL * D * 4)
    for p in places(ins, {k: v for k, v in UPDATE.items() if k == out or k not in ins}, out, over):
        st = lib.mamba_gated_recurrence_update(ctypes.byref(shape(1)), p["state"], p["slots"], POOL,
                                               p["x"], p["r"], p["i"], p["A"], p["z"], p["out"],
                                               None)
        assert st == INVALID


ROWS = 6
N16, N32 = ROWS * D * 2, ROWS * D * 4
NORM_IN = dict(x=N16, res=N32, w=D * 4)
NORM = dict(out=N16, scale=ROWS * 4, keep=N32)


@pytest.mark.parametrize("out,over", pairs(NORM, NORM_IN))
@pytest.mark.parametrize("fp8", [False, True])
def test_norm_forward(lib, out, over, fp8):
    if out == "scale" and not fp8:
        return
    outs = dict(NORM, out=ROWS * D if fp8 else N16)
    for n, p in enumerate(places(NORM_IN, outs, out, over)):
        if (out, over, n) != ("keep", "res", 0):       # the stream in place
            assert norm(lib, p, fp8) == INVALID


def norm(lib, p, fp8):
    args = (p["x"], 0, D, p["res"], 0, D, p["w"], 1, ROWS, D, 1e-5, 1, 0, p["out"])
    return lib.mamba_residual_norm_fp8(*args, p["scale"], p["keep"], None) if fp8 else \
        lib.mamba_residual_norm_fwd(*args, p["keep"], None)


@pytest.mark.parametrize("out,over", [p for p in pairs(NORM, NORM) if p[0] != p[1]])
@pytest.mark.parametrize("fp8", [False, True])
def test_norm_forward_among_outputs(lib, out, over, fp8):
    if "scale" in (out, over) and not fp8:
        return
    outs = dict(NORM, out=ROWS * D if fp8 else N16)
    for p in places({**NORM_IN, **rest(outs, out)}, {out: outs[out]}, out, over):
        assert norm(lib, p, fp8) == INVALID


NORM_BWD_IN = dict(res=N32, w=D * 4, dout=N16, dres=N32)
NORM_BWD = dict(dx=N16, dresidual=N32, dw=D * 4)


@pytest.mark.parametrize("out,over", pairs(NORM_BWD, NORM_BWD_IN))
def test_norm_backward(lib, out, over):
    for p in places(NORM_BWD_IN, NORM_BWD, out, over):
        assert norm_backward(lib, p) == INVALID


def norm_backward(lib, p):
    return lib.mamba_residual_norm_bwd(p["res"], 0, D, p["w"], p["dout"], p["dres"], 1, ROWS, D,
                                       1e-5, 1, 0, p["dx"], p["dresidual"], p["dw"],
                                       p.get("ws", at(60)), 1 << 30, None)


@pytest.mark.parametrize("out,over", [p for p in pairs(NORM_BWD, NORM_BWD) if p[0] != p[1]])
def test_norm_backward_among_outputs(lib, out, over):
    for p in places({**NORM_BWD_IN, **rest(NORM_BWD, out)}, {out: NORM_BWD[out]}, out, over):
        assert norm_backward(lib, p) == INVALID


@pytest.mark.parametrize("over", [*NORM_BWD_IN, *NORM_BWD])
def test_norm_backward_workspace(lib, over):
    n = lib.mamba_residual_norm_bwd_workspace_size(ROWS, D)
    for p in places({**NORM_BWD_IN, **NORM_BWD}, {"ws": n // 16 * 16}, "ws", over):
        assert norm_backward(lib, p) == INVALID
