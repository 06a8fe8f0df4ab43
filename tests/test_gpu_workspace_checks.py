"""Every call that takes a workspace refuses one in host memory, or one that is not a
single piece, before it launches anything."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def calls():
    import scan_selective_fwd_amd as ms
    b, dim, N, L = 2, 24, 16, 600
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    u, delta, B, C = r(b, dim, L), r(b, dim, L), r(b, N, L), r(b, N, L)
    A = -torch.rand(dim, N, device="cuda") - 0.5
    yield "scan_fwd", lambda **k: ms.scan_fwd(u, delta, A, B, C, segments=3, **k)
    yield "scan_bwd", lambda **k: ms.scan_bwd(u, delta, A, B, C, None, None, None, u, **k)
    Ac = torch.complex(A, r(dim, N))
    Bc, Cc = torch.complex(B, r(b, N, L)), torch.complex(C, r(b, N, L))
    yield "scan_fwd_complex", lambda **k: ms.scan_fwd_complex(u, delta, Ac, Bc, Cc, segments=3, **k)
    yield "scan_bwd_complex", lambda **k: ms.scan_bwd_complex(u, delta, Ac, Bc, Cc, None, None,
                                                              None, u, **k)
    uh, dh, Bh = r(b, 90, 4, 16), r(b, 90, 4), r(b, 90, 1, 16)
    Ah = -torch.rand(4, device="cuda") - 0.5
    yield "heads_scan_fwd", lambda **k: ms.heads_scan_fwd(uh, dh, Ah, Bh, Bh, **k)
    yield "heads_scan_bwd", lambda **k: ms.heads_scan_bwd(uh, dh, Ah, Bh, Bh, None, None, uh, **k)
    x, w = r(b, 90, 24), r(24, 4)
    yield "conv1d_tokens_bwd", lambda **k: ms.conv1d_tokens_bwd(x, w, None, x, **k)
    yield "gated_norm_bwd", lambda **k: ms.gated_norm_bwd(x, x, None, x, **k)


@pytest.mark.parametrize("at", range(8))
def test_a_workspace_the_kernels_cannot_write_is_refused(at):
    name, call = list(calls())[at]
    n = 1 << 24
    ok = torch.empty(n, dtype=torch.uint8, device="cuda")
    call(workspace=ok)
    torch.cuda.synchronize()
    print(name, flush=True)
    with pytest.raises(ValueError):
        call(workspace=torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError):
        call(workspace=ok[:1].expand(n))
    with pytest.raises(TypeError):
        call(workspace=n)
