"""The residual norm where its statistics come near the ends of float32 or vanish."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
         "mixed": (torch.bfloat16, torch.float32)}


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def check_bwd(got, i, eps):
    d, dw, dw_abs = R.norm_bwd(i["residual"], i["weight"], i["dout"], i["dres"], eps)
    terms = R.norm_terms(i["residual"], i["weight"], i["dout"], i["dres"], eps)
    for k in ("dx", "dresidual"):
        R.check(k, got[k], d, terms)
    R.check("dweight", got["dweight"], dw, dw_abs)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [33, 256, 768, 1500])
@pytest.mark.parametrize("rows", [1, 5, 2050])
def test_backward_without_eps(ms, rows, dim, types):
    """No row is zero, so that every gradient is finite, also where the last pass over the
    rows leaves some of a block's teams without one."""
    t = TYPES[types]
    i = R.norm_inputs(21, *t, rows, dim)
    kind = dict(x=t[0], dout=t[0], residual=t[1], dres=t[1], weight=torch.float32)
    g = {k: v.to(kind[k]).cuda() for k, v in i.items()}
    check_bwd(ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], g["dres"], eps=0.0), i, 0.0)
