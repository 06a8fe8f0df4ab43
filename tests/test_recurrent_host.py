"""Host side of the recurrent block's operators (no GPU, nothing is launched): the
library refuses bad arguments with the documented status before any device
call, sizes its workspaces, and its kernels keep to the chip's registers."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from kernel_resources import kernel_resources
from scan_selective_fwd_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
BAD = 2 ** 64 - 1
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED, INVALID = 1, 2, 3, 4, 5, 6, 8


def at(k):      # pointers that are never followed, 16 TiB apart
    return (k + 1) << 44


X, R_, I_, A, Z, H0, OUT, LAST, CK, WS, DX, DR, DI, DA, DZ, DOUT = (at(k) for k in range(16))


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def shape(**kw):
    s = _lib.RecurrenceShape(batch=2, seqlen=300, dim=96, x_batch_stride=28800, x_token_stride=96,
                             r_batch_stride=57600, r_token_stride=192, i_batch_stride=57600,
                             i_token_stride=192, z_batch_stride=28800, z_token_stride=96, dtype=1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def fwd(lib, s, x=X, r=R_, a=A, z=None, h0=None, out=OUT, last=None, ck=None, ws=WS, wsb=1 << 40):
    return lib.mamba_gated_recurrence_fwd(ctypes.byref(s) if s is not None else None, x, r, I_, a,
                                          z, h0, None, out, last, ck, ws, wsb, None)


def bwd(lib, s, z=None, h0=None, dout=DOUT, ck=None, dx=DX, dz=None, dh0=None, ws=WS, wsb=1 << 40):
    return lib.mamba_gated_recurrence_bwd(ctypes.byref(s), X, R_, I_, A, z, h0, None, dout, None,
                                          ck, dx, DR, DI, DA, dz, dh0, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(dim=-1), SHAPE),
    (dict(x_token_stride=-1), SHAPE), (dict(i_batch_stride=-5), SHAPE), (dict(dtype=2), DTYPE),
    (dict(seqlen=2 ** 60), UNSUPPORTED), (dict(batch=2 ** 40), UNSUPPORTED),
    (dict(dim=2 ** 29), UNSUPPORTED), (dict(r_batch_stride=2 ** 62), UNSUPPORTED),
    (dict(z_token_stride=2 ** 61), UNSUPPORTED)])
def test_recurrence_shapes_are_refused(lib, change, status):
    s = shape(**change)
    assert fwd(lib, s) == status and bwd(lib, s) == status
    ref = ctypes.byref(s)
    assert lib.mamba_gated_recurrence_fwd_workspace_size(ref) == BAD
    assert lib.mamba_gated_recurrence_bwd_workspace_size(ref, 0) == BAD
    assert lib.mamba_gated_recurrence_checkpoint_size(ref) == BAD


def test_recurrence_pointers_and_workspaces_are_refused(lib):
    s = shape()
    ref = ctypes.byref(s)
    nf = lib.mamba_gated_recurrence_fwd_workspace_size(ref)
    n1 = lib.mamba_gated_recurrence_bwd_workspace_size(ref, 1)
    n0 = lib.mamba_gated_recurrence_bwd_workspace_size(ref, 0)
    assert 0 < nf < 2 ** 24 and 0 < n1 < n0 < 2 ** 24
    assert lib.mamba_gated_recurrence_checkpoint_size(ref) == 2 * 5 * 96 * 4
    assert fwd(lib, None) == NULL
    assert fwd(lib, s, x=None) == NULL and fwd(lib, s, out=None) == NULL and fwd(lib, s, a=None) == NULL
    assert fwd(lib, s, r=R_ + 1) == ALIGN and fwd(lib, s, a=A + 2) == ALIGN
    assert fwd(lib, s, last=LAST + 2) == ALIGN and fwd(lib, s, ck=CK + 1) == ALIGN
    assert fwd(lib, s, ws=WS + 8) == ALIGN
    assert fwd(lib, s, wsb=nf - 1) == WORKSPACE and fwd(lib, s, ws=None) == WORKSPACE
    assert fwd(lib, s, h0=H0, last=H0 + 4) == INVALID          # a part of h0
    for over in (X, X + 2 * 28800, R_ + 64):                   # out over an input
        assert fwd(lib, s, out=over) == INVALID
    assert fwd(lib, s, z=Z, out=Z) == INVALID
    assert bwd(lib, s, ck=CK, wsb=n1 - 1) == WORKSPACE and bwd(lib, s, wsb=n0 - 1) == WORKSPACE
    assert bwd(lib, s, dout=None) == NULL and bwd(lib, s, dx=None) == NULL
    assert bwd(lib, s, z=Z) == INVALID and bwd(lib, s, dz=DZ) == INVALID
    assert bwd(lib, s, dh0=DZ) == INVALID                      # of an absent input
    assert bwd(lib, s, dx=R_) == INVALID and bwd(lib, s, dx=DX + 1) == ALIGN


def test_short_sequences_need_no_workspace(lib):
    sizes = [lib.mamba_gated_recurrence_fwd_workspace_size(ctypes.byref(shape(seqlen=n)))
             for n in (1, 256, 257, 5000)]
    assert sizes[:2] == [0, 0] and 0 < sizes[2] < sizes[3]
    s = shape(seqlen=10, x_batch_stride=960)
    assert lib.mamba_gated_recurrence_bwd_workspace_size(ctypes.byref(s), 1) == 768   # dA's shares, 2 x 96


def test_recurrence_update_is_refused(lib):
    def go(s=None, state=LAST, slots=None, pool=4, x=X, out=OUT):
        s = s or shape(seqlen=1)
        return lib.mamba_gated_recurrence_update(ctypes.byref(s), state, slots, pool, x, R_, I_, A,
                                                 None, out, None)
    assert go(shape()) == SHAPE                                 # more than one step
    assert go(pool=1) == SHAPE and go(pool=0, slots=CK) == SHAPE
    assert go(state=None) == NULL and go(x=None) == NULL and go(out=None) == NULL
    assert go(state=LAST + 2) == ALIGN and go(slots=CK + 1, pool=1) == ALIGN
    assert go(out=X) == INVALID and go(pool=2 ** 60) == UNSUPPORTED


def test_norm_is_refused(lib):
    def go(x=X, sx=64, res=R_, sr=64, w=None, rows=4, dim=64, eps=1e-5, dt=1, rdt=1, out=OUT,
           keep=LAST, batch=2, sb=256):
        return lib.mamba_residual_norm_fwd(x, sb, sx, res, sb, sr, w, batch, rows, dim, eps, dt,
                                           rdt, out, keep, None)
    assert go(rows=0) == SHAPE and go(dim=0) == SHAPE and go(sx=-1) == SHAPE and go(sr=-1) == SHAPE
    assert go(eps=-1.0) == INVALID and go(eps=float("nan")) == INVALID
    assert go(dt=7) == DTYPE and go(dt=0, rdt=1) == DTYPE and go(rdt=3) == DTYPE
    assert go(x=None) == NULL and go(out=None) == NULL and go(keep=None) == NULL
    assert go(res=None) == INVALID                              # residual_out alone
    assert go(x=X + 1) == ALIGN and go(rdt=0, res=R_ + 2) == ALIGN and go(w=A + 2) == ALIGN
    assert go(rows=2 ** 60) == UNSUPPORTED and go(dim=2 ** 29) == UNSUPPORTED
    assert go(out=X) == INVALID and go(out=R_) == INVALID and go(keep=X) == INVALID
    assert go(keep=R_ + 16) == INVALID                          # a part of the stream
    assert go(keep=R_, sr=128) == INVALID                       # in place, rows apart
    assert go(keep=R_, sb=512) == INVALID                       # or batch rows apart
    assert go(batch=0) == SHAPE and go(sb=-1) == SHAPE and go(batch=2 ** 58) == UNSUPPORTED

    def fp8(scale=CK, out=OUT):
        return lib.mamba_residual_norm_fp8(X, 0, 64, R_, 0, 64, None, 1, 4, 64, 1e-5, 1, 1, out,
                                           scale, LAST, None)
    assert fp8(scale=None) == NULL and fp8(scale=CK + 1) == ALIGN and fp8(out=None) == NULL
    n = lib.mamba_residual_norm_bwd_workspace_size(4, 64)
    assert n == 1024 and lib.mamba_residual_norm_bwd_workspace_size(4, 0) == BAD

    def back(res=R_, w=None, dw=None, dres=None, dresidual=None, rdt=1, dx=DX, wsb=n):
        return lib.mamba_residual_norm_bwd(res, 0, 64, w, DOUT, dres, 1, 4, 64, 1e-5, 1, rdt, dx,
                                           dresidual, dw, WS, wsb, None)
    assert back(w=A) == INVALID and back(dw=DA) == INVALID
    assert back(dresidual=DZ) == INVALID                        # of one type: it is dx
    assert back(res=None) == NULL and back(dx=None) == NULL and back(wsb=n - 1) == WORKSPACE
    assert back(dx=DOUT) == INVALID and back(dx=R_) == INVALID and back(dres=CK + 1) == ALIGN


def test_the_binding_refuses_before_any_call():
    """On the CPU: no tensor of the wrong place, kind or type reaches the library."""
    import scan_selective_fwd_amd as ms
    x, a = torch.zeros(2, 5, 8), torch.zeros(8)
    for call in (lambda: ms.gated_recurrence_fwd(x, x, x, a),
                 lambda: ms.gated_recurrence_bwd(x, x, x, a, None, x),
                 lambda: ms.gated_recurrence_update(x[0], x[0], x[0], x[0], a),
                 lambda: ms.gated_recurrence(x, x, x, a),
                 lambda: ms.residual_norm_fwd(x, x, a), lambda: ms.residual_norm_fp8(x),
                 lambda: ms.residual_norm_bwd(x, a, x), lambda: ms.residual_norm(x, x, a)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: ms.gated_recurrence_fwd(None, x, x, a), lambda: ms.residual_norm_fwd(3.0),
                 lambda: ms.residual_norm_bwd(None, a, x)):
        with pytest.raises(TypeError):
            call()
    assert ms.gated_recurrence_checkpoint_shape(2, 129, 7) == (2, 3, 7)
    assert ms.gated_recurrence_fwd_workspace_bytes(1, 200, 64) == 0
    with pytest.raises(ms.MambaScanError):
        ms.gated_recurrence_bwd_workspace_bytes(1, 0, 64)
    with pytest.raises(ms.MambaScanError):
        ms.gated_recurrence_fwd_workspace_bytes(1, 2 ** 60, 64)


def test_rows_of_views_are_where_the_strides_say():
    """The norm's batch and row strides give each row of a view, and no element outside it:
    broadcast batches and rows, slices, steps, and views together with dense tensors."""
    from scan_selective_fwd_amd import recurrent as rec
    wide = torch.arange(4 * 6 * 11, dtype=torch.float32).view(4, 6, 11)
    views = [wide, wide[..., 2:7], wide[:, 1:4], wide[:, ::2], wide[:, 3:4], wide[1:2, 1:4],
             wide[:1].expand(4, 6, 11), wide[:1, 2:5].expand(4, 3, 11), wide[:1].expand(1, 6, 11),
             wide[:, :1].expand(4, 6, 11), wide[:1, :1].expand(4, 6, 11), wide[0], wide[0, 0],
             wide[0, :1].expand(5, 11), wide[..., :1], wide[:1, :, :1].expand(4, 6, 1), wide[::2],
             wide.view(2, 2, 6, 11), wide.view(4, 2, 3, 11)[:1].expand(3, 2, 3, 11)]
    for v in views:
        for other in (v.contiguous(), v):
            sizes, a, b = rec._planes(v, rec._row_strides(v, "v"), rec._row_strides(other, "other"))
            assert sizes[0] * sizes[1] * sizes[2] == v.numel()
            for t, (sb, sr) in ((v, a), (other, b)):
                last = (sizes[0] - 1) * sb + (sizes[1] - 1) * sr + sizes[2]
                assert t.storage_offset() + last <= t.untyped_storage().nbytes() // 4
                assert torch.equal(t.as_strided(sizes, (sb, sr, 1)).reshape(v.shape), t)
    for v in (wide.transpose(1, 2), wide.transpose(0, 1), wide[..., ::2], wide[0, 0, ::2]):
        try:
            sizes, a, _ = rec._planes(v, rec._row_strides(v, "v"), (None, 0))
        except ValueError:
            continue
        assert torch.equal(v.as_strided(sizes, (*a, 1)).reshape(v.shape), v)


def test_kernels_keep_their_registers():
    """Two blocks of 8 waves share a CU at 128 registers a lane; nothing spills."""
    res = kernel_resources(os.path.join(ROOT, "scan_selective_fwd_amd", "libmamba_scan.so"))
    tiles = {k: v for k, v in res.items() if re.search(r"rec_(fwd|bwd)_kernelI.*Lb1EEE", k)}
    assert len(tiles) == 12 + 8
    assert not {k: v for k, v in tiles.items() if v["vgpr"] > 128}
    rest = {k: v for k, v in res.items() if re.search(r"rec_(fwd|bwd|step|sum|clear)_kernel", k)}
    assert len(rest) == 2 * (12 + 8) + 4 + 2 and not [k for k, v in rest.items() if v["scratch"]]
    norms = {k: v for k, v in res.items() if "res_norm" in k}
    assert len(norms) > 60 and not [k for k, v in norms.items() if v["scratch"]]


@pytest.mark.skipif(shutil.which("g++") is None or
                    not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="no host C++ compiler or HIP headers")
def test_abi_layer_under_sanitizers(tmp_path):
    """recurrent_api.cpp with host stand-ins for the dispatchers, over small and
    extreme sizes; every finding is fatal."""
    exe = str(tmp_path / "recurrent_driver")
    csrc = os.path.join(ROOT, "scan_selective_fwd_amd", "csrc")
    san = "-fsanitize=" + "address,undefined"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", san, "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include",
                        f"-I{csrc}",
                        os.path.join(ROOT, "tests", "sanitize", "recurrent_driver.cpp"),
                        os.path.join(csrc, "recurrent_api.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=600)
    if r.returncode != 0 and "sanitize" in r.stderr and "cannot find" in r.stderr:
        pytest.skip("the host compiler has no sanitizer runtime")
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                                UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and "recurrent ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
