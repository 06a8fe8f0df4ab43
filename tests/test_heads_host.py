"""Host side of the multi-head operators (no GPU, nothing is launched): the
library refuses bad arguments with the documented status before any device
call, sizes its workspaces, and its kernels keep to the chip's registers."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from kernel_resources import kernel_resources
from scan_selective_fwd_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
P = 1 << 20            # a pointer that is never followed
BAD = 2 ** 64 - 1
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED, INVALID = 1, 2, 3, 4, 5, 6, 8


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def shape(**kw):
    s = _lib.HeadsShape(batch=2, seqlen=100, heads=4, headdim=64, groups=2, dstate=128,
                        u_batch_stride=25600, u_token_stride=256, delta_batch_stride=400,
                        delta_token_stride=4, B_batch_stride=25600, B_token_stride=256,
                        C_batch_stride=25600, C_token_stride=256, delta_softplus=1, disc=0,
                        dtype=1, segments=0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def fwd(lib, s, u=P, A=P, out=P, ws=P, wsb=1 << 62, last=None, **kw):
    return lib.mamba_heads_scan_fwd(ctypes.byref(s) if s is not None else None, u, P, A, P, P,
                                    None, kw.get("bias"), None, None, out, last, ws, wsb, None)


def bwd(lib, s, ws=P, wsb=1 << 62, dout=P, dD=None, dh0=None):
    return lib.mamba_heads_scan_bwd(ctypes.byref(s), P, P, P, P, P, None, None, None, None, dout,
                                    None, P, P, P, P, P, dD, None, dh0, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(heads=-1), SHAPE),
    (dict(groups=3), SHAPE), (dict(u_token_stride=-1), SHAPE), (dict(C_batch_stride=-5), SHAPE),
    (dict(dtype=2), DTYPE), (dict(disc=9), DTYPE), (dict(segments=-1), INVALID),
    (dict(headdim=129), UNSUPPORTED), (dict(dstate=257), UNSUPPORTED),
    (dict(seqlen=2 ** 62), UNSUPPORTED), (dict(batch=2 ** 40), UNSUPPORTED),
    (dict(u_batch_stride=2 ** 62), UNSUPPORTED), (dict(B_token_stride=2 ** 61), UNSUPPORTED)])
def test_scan_shapes_are_refused(lib, change, status):
    s = shape(**change)
    assert fwd(lib, s) == status
    assert bwd(lib, s) == status
    ref = ctypes.byref(s)
    assert lib.mamba_heads_scan_fwd_workspace_size(ref) == BAD
    assert lib.mamba_heads_scan_bwd_workspace_size(ref) == BAD


def test_scan_pointers_and_workspaces_are_refused(lib):
    s = shape()
    ref = ctypes.byref(s)
    nf, nb = lib.mamba_heads_scan_fwd_workspace_size(ref), lib.mamba_heads_scan_bwd_workspace_size(ref)
    assert 0 < nf < nb < 2 ** 32
    assert fwd(lib, None) == NULL
    assert fwd(lib, s, u=None) == NULL and fwd(lib, s, out=None) == NULL
    assert fwd(lib, s, u=P + 1) == ALIGN and fwd(lib, s, A=P + 2) == ALIGN
    assert fwd(lib, s, last=P + 2) == ALIGN and fwd(lib, s, bias=P + 1) == ALIGN
    assert fwd(lib, s, wsb=nf - 1) == WORKSPACE and fwd(lib, s, ws=None) == WORKSPACE
    assert fwd(lib, s, ws=P + 8) == ALIGN
    assert bwd(lib, s, wsb=nb - 1) == WORKSPACE and bwd(lib, s, ws=None) == WORKSPACE
    assert bwd(lib, s, dout=None) == NULL
    assert bwd(lib, s, dD=P) == INVALID and bwd(lib, s, dh0=P) == INVALID   # of absent inputs


def test_more_segments_take_more_workspace(lib):
    sizes = [lib.mamba_heads_scan_fwd_workspace_size(ctypes.byref(shape(seqlen=4096, segments=k)))
             for k in (1, 2, 8, 64, 5000)]
    assert sizes[0] < sizes[1] < sizes[2] < sizes[3] == sizes[4]   # one chunk a segment at most


def test_state_update_is_refused(lib):
    def go(s, state=P, slots=None, pool=2, out=P):
        return lib.mamba_heads_state_update(ctypes.byref(s), state, slots, pool, P, P, P, P, P,
                                            None, None, out, None)
    one = shape(seqlen=1)
    assert go(shape()) == SHAPE                    # more than one token
    assert go(one, pool=1) == SHAPE and go(one, pool=0, slots=P) == SHAPE
    assert go(one, state=None) == NULL and go(one, out=None) == NULL
    assert go(one, slots=P + 2) == ALIGN and go(one, pool=2 ** 60) == UNSUPPORTED


def test_conv_is_refused(lib):
    def fwd_(x=P, w=P, W=4, dt=1, b=2, d=64, L=100, out=P, win=None, wout=None, st=64):
        return lib.mamba_conv1d_tokens_fwd(x, L * d, st, w, None, win, None, W, dt, b, d, L, out,
                                           wout, None)
    assert fwd_(W=1) == UNSUPPORTED and fwd_(W=5) == UNSUPPORTED and fwd_(W=0) == SHAPE
    assert fwd_(dt=3) == DTYPE and fwd_(b=0) == SHAPE and fwd_(L=0) == SHAPE
    assert fwd_(x=None) == NULL and fwd_(w=None) == NULL and fwd_(out=None) == NULL
    assert fwd_(x=P + 1) == ALIGN and fwd_(st=-1) == SHAPE
    assert fwd_(win=P, wout=P) == INVALID          # the window may not be its own successor
    assert fwd_(L=2 ** 61) == UNSUPPORTED
    n = lib.mamba_conv1d_tokens_bwd_workspace_size(2, 64, 100, 4)
    assert 0 < n < 2 ** 20
    assert lib.mamba_conv1d_tokens_bwd_workspace_size(2, 0, 100, 4) == BAD

    def bwd_(ws=P, wsb=n, db=None, dwin=None):
        return lib.mamba_conv1d_tokens_bwd(P, 6400, 64, P, None, None, None, P, 4, 1, 2, 64, 100,
                                           P, P, db, dwin, ws, wsb, None)
    assert bwd_(wsb=n - 1) == WORKSPACE and bwd_(ws=None) == WORKSPACE
    assert bwd_(db=P) == INVALID and bwd_(dwin=P) == INVALID
    upd = lib.mamba_conv1d_tokens_update
    assert upd(P, 64, P, None, 1, P, None, 4, 1, 2, 64, P, None) == SHAPE     # pool < batch
    assert upd(P, 64, None, None, 2, P, None, 4, 1, 2, 64, P, None) == NULL


def test_norm_is_refused(lib):
    def go(x=P, rows=4, dim=64, groups=2, eps=1e-5, dt=1, out=P, sx=64):
        return lib.mamba_gated_norm_fwd(x, sx, None, 0, None, rows, dim, groups, eps, 1, dt, out,
                                        None)
    assert go(groups=3) == SHAPE and go(rows=0) == SHAPE and go(sx=-1) == SHAPE
    assert go(eps=-1.0) == INVALID and go(eps=float("nan")) == INVALID
    assert go(dt=7) == DTYPE and go(x=None) == NULL and go(out=None) == NULL
    assert go(x=P + 1) == ALIGN and go(rows=2 ** 60) == UNSUPPORTED
    n = lib.mamba_gated_norm_bwd_workspace_size(4, 64, 2)
    assert 0 < n < 2 ** 16 and lib.mamba_gated_norm_bwd_workspace_size(4, 64, 3) == BAD

    def bwd_(z=None, dz=None, w=None, dw=None, wsb=n):
        return lib.mamba_gated_norm_bwd(P, 64, z, 64, w, P, 4, 64, 2, 1e-5, 1, 1, P, dz, dw, P,
                                        wsb, None)
    assert bwd_(z=P) == INVALID and bwd_(dz=P) == INVALID and bwd_(dw=P) == INVALID
    assert bwd_(wsb=n - 1) == WORKSPACE


def test_kernels_keep_their_registers():
    """The passes of the usual sizes (dstate up to 128, bfloat16, rows on 16
    bytes) keep two waves a SIMD, and their loops no scratch: a reload of a
    spilled value waits for every load in flight before it."""
    res = kernel_resources(os.path.join(ROOT, "scan_selective_fwd_amd", "libmamba_scan.so"))
    name = re.compile(r"heads_(fwd|seg|states|chunk)_kernelI([ft])Li(\d)ELb([01])E")
    seen = {m.groups(): v for k, v in res.items() if (m := name.search(k))}
    assert len(seen) == 4 * 2 * 4 * 2
    hot = {k: v for k, v in seen.items() if k[1] == "t" and k[2] in "124" and k[3] == "1"}
    assert not {k: v for k, v in hot.items() if v["vgpr"] > 256}
    assert not {k: v for k, v in hot.items() if v["scratch"] > (64 if k[0] == "chunk" else 0)}
    rest = [v for k, v in res.items()
            if re.search(r"tokconv_|norm_(fwd|bwd)|heads_step|heads_scal|heads_.*carry", k)]
    assert len(rest) > 40 and not [v for v in rest if v["scratch"]]


@pytest.mark.skipif(shutil.which("g++") is None or
                    not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="no host C++ compiler or HIP headers")
def test_abi_layer_under_sanitizers(tmp_path):
    """heads_api.cpp with host stand-ins for the dispatchers, over small and
    extreme sizes; every finding is fatal."""
    exe = str(tmp_path / "heads_driver")
    csrc = os.path.join(ROOT, "scan_selective_fwd_amd", "csrc")
    san = "-fsanitize=" + "address,undefined"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", san, "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include",
                        f"-I{csrc}", os.path.join(ROOT, "tests", "sanitize", "heads_driver.cpp"),
                        os.path.join(csrc, "heads_api.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=600)
    if r.returncode != 0 and "sanitize" in r.stderr and "cannot find" in r.stderr:
        pytest.skip("the host compiler has no sanitizer runtime")
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                                UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and "heads ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
