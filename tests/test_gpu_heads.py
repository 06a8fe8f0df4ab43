"""The multi-head operators on the GPU against the 64-bit reference: sizes
around every tile border, both types and discretisations, packed rows, views,
pools of states, and what is refused."""
import pytest
import torch

import heads_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# (batch, L, heads, P, groups, N)
SIZES = [(1, 1, 1, 1, 1, 1), (2, 1, 3, 5, 1, 7), (1, 2, 2, 64, 1, 128), (1, 63, 2, 64, 1, 16),
         (2, 64, 4, 64, 2, 128), (1, 65, 2, 32, 1, 64), (3, 130, 6, 48, 3, 80),
         (1, 200, 2, 128, 1, 256), (1, 300, 1, 100, 1, 200), (2, 257, 8, 64, 8, 128),
         (1, 129, 3, 17, 1, 33), (2, 96, 4, 8, 2, 24)]
SEQ = ("u", "delta", "B", "C", "dout")


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def dev(i, dtype):
    """The inputs on the GPU, in the types the calls take."""
    return {k: None if v is None else
            v.cuda() if v.dtype == torch.uint8 else
            v.to(dtype if k in SEQ else torch.float32).cuda() for k, v in i.items()}


def ref_fwd(i, **kw):
    return R.scan_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                      i["h0"], i["reset"], **kw)[:2]


def run_fwd(ms, g, softplus=True, **kw):
    return ms.heads_scan_fwd(g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["delta_bias"],
                             g["h0"], reset=g["reset"], return_last_state=True,
                             delta_softplus=softplus, **kw)


def run_bwd(ms, g, dlast=True, softplus=True, **kw):
    return ms.heads_scan_bwd(g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["delta_bias"],
                             g["dout"], g["h0"], reset=g["reset"], delta_softplus=softplus,
                             dlast_state=g["dlast"] if dlast else None, **kw)


def check_bwd(got, i, dlast=True, **kw):
    ref, scale = R.scan_bwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                            i["dout"], i["h0"], i["dlast"] if dlast else None, i["reset"], **kw)
    assert set(got) == set(ref)
    for k in ref:
        R.check(k, got[k], ref[k], scale.get(k))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("disc", ["zoh", "euler"])
@pytest.mark.parametrize("size", SIZES)
def test_forward(ms, size, disc, dtype):
    i = R.scan_inputs(11, DT[dtype], *size, h0=size[1] % 2 == 0)
    g = dev(i, DT[dtype])
    out, last = run_fwd(ms, g, disc=disc)
    assert out.dtype == DT[dtype] and last.dtype == torch.float32
    ro, rl = ref_fwd(i, disc=disc)
    R.check("out", out, ro)
    R.check("last_state", last, rl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reset", ["random", "every", "edges"])
@pytest.mark.parametrize("size", [(2, 1, 3, 5, 1, 7), (2, 257, 4, 64, 2, 128), (3, 130, 6, 48, 3, 80),
                                  (1, 500, 2, 32, 1, 16)])
def test_packed_forward_and_backward(ms, size, reset, dtype):
    i = R.scan_inputs(12, DT[dtype], *size, h0=True, reset=reset)
    g = dev(i, DT[dtype])
    out, last = run_fwd(ms, g)
    ro, rl = ref_fwd(i)
    R.check("out", out, ro)
    R.check("last_state", last, rl)
    check_bwd(run_bwd(ms, g), i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("disc", ["zoh", "euler"])
@pytest.mark.parametrize("size", SIZES)
def test_backward(ms, size, disc, dtype):
    i = R.scan_inputs(13, DT[dtype], *size, h0=size[1] % 2 == 0)
    dlast = size[2] % 2 == 0
    check_bwd(run_bwd(ms, dev(i, DT[dtype]), dlast, disc=disc), i, dlast, disc=disc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("segments", [1, 2, 3, 7, 100])
def test_segments(ms, segments, dtype):
    i = R.scan_inputs(14, DT[dtype], 2, 700, 4, 64, 2, 64, h0=True, reset="random")
    g = dev(i, DT[dtype])
    out, last = run_fwd(ms, g, segments=segments)
    ro, rl = ref_fwd(i)
    R.check("out", out, ro)
    R.check("last_state", last, rl)
    check_bwd(run_bwd(ms, g, segments=segments), i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("segments", [8, 9, 10, 17])
def test_where_a_pass_of_its_own_joins_the_segments(ms, segments, dtype):
    """More segments than the output pass joins by itself, and as many."""
    q = 32 if dtype == "f32" else 64
    i = R.scan_inputs(41, DT[dtype], 2, q * segments - 5, 3, 40, 1, 48, h0=True, reset="edges")
    out, last = run_fwd(ms, dev(i, DT[dtype]), segments=segments)
    ro, rl = ref_fwd(i)
    R.check("out", out, ro)
    R.check("last_state", last, rl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strong_decays_keep_the_last_state(ms, dtype):
    """Decays whose sum over a chunk is far below zero.  What reaches the state is
    near its end, with weights near 1 whose exponents are differences of such
    sums: 4 units of the step's softplus, 2 of the exponent, 2 of product and sum,
    2 for the float32 rounding of the reference's inputs' sum, of 2^-24 each."""
    i = R.scan_inputs(42, DT[dtype], 2, 256, 4, 64, 1, 128)
    i["A"][:] = -16.0
    i["delta_bias"][:] = -1.5
    last = run_fwd(ms, dev(i, DT[dtype]), disc="euler")[1]
    want = ref_fwd(i, disc="euler")[1]
    e = (last.double().cpu() - want).norm() / want.norm()
    assert float(e) <= 10 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("disc", ["zoh", "euler"])
def test_growing_still_and_undecayed_heads(ms, disc, dtype):
    i = R.scan_inputs(15, DT[dtype], 2, 190, 6, 32, 1, 64, h0=True, A="mixed")
    g = dev(i, DT[dtype])
    out, last = run_fwd(ms, g, disc=disc)
    ro, rl = ref_fwd(i, disc=disc)
    R.check("out", out, ro)
    R.check("last_state", last, rl)
    check_bwd(run_bwd(ms, g, disc=disc), i, disc=disc)


def test_plain_steps_and_absent_options(ms):
    """softplus off, steps up to 3 (log decays to -48 a step), no D, no bias."""
    i = R.scan_inputs(16, torch.float32, 2, 150, 4, 32, 2, 32)
    i["delta"] = R.Inputs(17, torch.float32).uniform(0.0, 3.0, 2, 150, 4)
    i["D"] = i["delta_bias"] = None
    g = dev(i, torch.float32)
    out, last = run_fwd(ms, g, softplus=False)
    ro, rl = ref_fwd(i, softplus=False)
    R.check("out", out, ro)
    R.check("last_state", last, rl)
    check_bwd(run_bwd(ms, g, softplus=False), i, softplus=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1])
def test_views_of_joined_rows(ms, offset, dtype):
    """u, B, C as parts of one row (at an aligned and an odd offset), delta a
    slice, one batch row repeated with stride 0."""
    b, L, H, P, G, N = 2, 90, 4, 16, 2, 24
    i = R.scan_inputs(18, DT[dtype], b, L, H, P, G, N)
    for n in ("u", "delta", "B", "C"):
        i[n] = i[n][:1].expand(b, *i[n].shape[1:]).contiguous()
    g = dev(i, DT[dtype])
    row = torch.zeros(1, L, 200, dtype=DT[dtype], device="cuda")
    o = offset
    parts = {}
    for n, w, shape in (("u", H * P, (H, P)), ("B", G * N, (G, N)), ("C", G * N, (G, N)),
                        ("delta", H, (H,))):
        v = row[..., o:o + w].unflatten(-1, shape)
        v.copy_(g[n][:1])
        parts[n] = v.expand(b, *v.shape[1:])
        o += w
    v = dict(g, **parts)
    out, last = run_fwd(ms, v)
    ro, rl = ref_fwd(i)
    R.check("out", out, ro)
    R.check("last_state", last, rl)
    check_bwd(run_bwd(ms, v), i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_in_pieces_and_token_by_token(ms, dtype):
    """A prompt scanned whole, in two calls, and its last tokens one by one."""
    i = R.scan_inputs(19, DT[dtype], 2, 140, 4, 64, 1, 128)
    g = dev(i, DT[dtype])
    cut = lambda a, b: dict(g, **{n: g[n][:, a:b] for n in ("u", "delta", "B", "C")})  # noqa: E731
    ro, rl = ref_fwd(i)
    o1, h = run_fwd(ms, cut(0, 75))
    o2, h = run_fwd(ms, dict(cut(75, 130), h0=h))
    R.check("pieces", torch.cat([o1, o2], 1), ro[:, :130])
    for t in range(130, 140):
        o = ms.heads_state_update(h, g["u"][:, t], g["delta"][:, t], g["A"], g["B"][:, t],
                                  g["C"][:, t], g["D"], g["delta_bias"])
        R.check("token", o, ro[:, t])
    R.check("state", h, rl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_token_update_over_a_pool(ms, size, dtype):
    _, _, H, P, G, N = size
    b, pool = 5, 9
    i = R.scan_inputs(21, DT[dtype], b, 1, H, P, G, N, h0=True)
    g = dev(i, DT[dtype])
    states = R.Inputs(22, torch.float32).f32(pool, H, P, N)
    slots = torch.tensor([7, 0, -1, 3, pool], dtype=torch.int32)   # two rows left out
    live = [0, 1, 3]
    at = slots[live].long()
    i["h0"][live] = states[at]
    ro, rl = ref_fwd(i)
    st = states.float().cuda()
    out = ms.heads_state_update(st, g["u"][:, 0], g["delta"][:, 0], g["A"], g["B"][:, 0],
                                g["C"][:, 0], g["D"], g["delta_bias"], slots=slots.cuda())
    R.check("out", out[live], ro[live, 0])
    assert not out[[2, 4]].any()
    R.check("state", st[at.cuda()], rl[live])
    rest = [k for k in range(pool) if k not in at.tolist()]
    assert torch.equal(st[rest].cpu(), states[rest].float())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3.4e38])
@pytest.mark.parametrize("what", ["u", "B", "C", "delta"])
def test_non_finite_values_stay_in_their_sequence(ms, what, value):
    """Neither earlier rows nor the other packed sequences see them."""
    L, at, start = 200, 70, 90
    i = R.scan_inputs(23, torch.float32, 2, L, 2, 32, 1, 32, reset="random")
    i["reset"][:] = 0
    i["reset"][:, start] = 1
    for dtype in (torch.float32, torch.bfloat16):
        g = dev(i, dtype)
        clean, clean_last = run_fwd(ms, g)
        bad = dict(g)
        bad[what] = g[what].clone()
        bad[what][0, at] = value
        out, last = run_fwd(ms, bad)
        assert torch.equal(out[1], clean[1])
        assert torch.equal(out[0, :at], clean[0, :at])
        assert torch.equal(out[0, start:], clean[0, start:])
        assert torch.equal(last, clean_last)
        if what != "delta" and value != 3.4e38:
            assert not torch.isfinite(out[0, at]).any()


def test_a_non_finite_step_reaches_what_follows(ms):
    i = R.scan_inputs(24, torch.float32, 1, 200, 1, 32, 1, 32)
    g = dev(i, torch.float32)
    g["u"][0, 70, 0, 5] = float("nan")
    out, last = run_fwd(ms, g)
    assert torch.isnan(out[0, 70:, 0, 5]).all() and torch.isnan(last[0, 0, 5]).all()
    keep = [k for k in range(32) if k != 5]
    assert torch.isfinite(out[0][:, 0, keep]).all() and torch.isfinite(out[0, :70]).all()


def test_equal_inputs_give_equal_bits(ms):
    i = R.scan_inputs(25, torch.bfloat16, 2, 300, 8, 64, 2, 128, h0=True)
    g = dev(i, torch.bfloat16)
    a, b = run_bwd(ms, g), run_bwd(ms, g)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_another_stream_and_a_kept_workspace(ms):
    i = R.scan_inputs(26, torch.bfloat16, 2, 300, 4, 64, 1, 64)
    g = dev(i, torch.bfloat16)
    want = run_fwd(ms, g)
    wantb = run_bwd(ms, g)
    n = max(ms.heads_fwd_workspace_bytes(2, 300, 4, 64, 1, 64, torch.bfloat16),
            ms.heads_bwd_workspace_bytes(2, 300, 4, 64, 1, 64, torch.bfloat16), 1)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_fwd(ms, g, workspace=ws)
        gotb = run_bwd(ms, g, workspace=ws)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(gotb[k], wantb[k]) for k in wantb)


def test_scan_autograd(ms):
    i = R.scan_inputs(27, torch.float32, 2, 70, 4, 32, 2, 16, h0=True)
    g = dev(i, torch.float32)
    names = ("u", "delta", "A", "B", "C", "D", "delta_bias", "h0")
    v = {n: g[n].clone().requires_grad_(True) for n in names}
    out, last = ms.heads_scan(*(v[n] for n in names), return_last_state=True)
    ((out * g["dout"]).sum() + (last * g["dlast"]).sum()).backward()
    ref, scale = R.scan_bwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                            i["dout"], i["h0"], i["dlast"])
    for n in names:
        R.check(n, v[n].grad, ref["d" + n], scale.get("d" + n))


@pytest.mark.parametrize("disc", ["zoh", "euler"])
def test_scan_gradient_against_differences(ms, disc):
    """The kernels' own forward, in 32 bits, along random directions."""
    i = R.scan_inputs(28, torch.float32, 2, 90, 4, 32, 1, 32, h0=True)
    g = dev(i, torch.float32)
    got = run_bwd(ms, g, disc=disc)
    r = R.Inputs(29, torch.float32)
    for n in ("u", "delta", "A", "B", "C", "D", "delta_bias", "h0"):
        d = r.f32(*i[n].shape).float().cuda()
        eps = 1e-2 if n not in ("delta", "delta_bias", "A") else 2e-3
        loss = []
        for s in (1.0, -1.0):
            o, last = run_fwd(ms, dict(g, **{n: g[n] + s * eps * d}), disc=disc)
            loss.append(float((o.double() * g["dout"]).sum() + (last.double() * g["dlast"]).sum()))
        fd = (loss[0] - loss[1]) / (2 * eps)
        an = float((got["d" + n].double() * d).sum())
        # float32 outputs of norm ~1e3 rounded at 2^-24, against eps; the third derivative
        size = float(got["d" + n].double().norm())
        assert abs(fd - an) <= 2e-2 * size + 0.05, (n, fd, an, size)


def test_refusals(ms):
    i = R.scan_inputs(30, torch.float32, 2, 20, 4, 16, 2, 16, h0=True)
    g = dev(i, torch.float32)

    def bad(exc, **kw):
        with pytest.raises(exc):
            run_fwd(ms, dict(g, **kw))

    bad(ValueError, u=g["u"].cpu())
    bad(ValueError, u=g["u"][..., ::2])
    bad(ValueError, u=g["u"][0])
    bad(TypeError, u=g["u"].half())
    bad(TypeError, B=g["B"].bfloat16())
    bad(ValueError, delta=g["delta"][:, :-1])
    bad(ValueError, A=g["A"][:3])
    bad(TypeError, h0=g["h0"].bfloat16())
    bad(ValueError, h0=g["h0"].transpose(2, 3))
    bad(ms.MambaScanError, B=g["B"].new_zeros(2, 20, 3, 16), C=g["C"].new_zeros(2, 20, 3, 16))
    bad(ms.MambaScanError, B=g["B"].new_zeros(2, 20, 1, 300), C=g["C"].new_zeros(2, 20, 1, 300),
        h0=None)
    bad(ms.MambaScanError, u=g["u"].new_zeros(2, 20, 4, 130), h0=None)
    bad(ms.MambaScanError, **{n: g[n][:, :0] for n in ("u", "delta", "B", "C")}, reset=None)
    with pytest.raises(ValueError):
        run_fwd(ms, g, disc="other")
    with pytest.raises(ms.MambaScanError):
        run_fwd(ms, g, segments=-1)
    st = g["h0"].clone()
    one = [g[n][:, 0] for n in ("u", "delta")] + [g["A"]] + [g[n][:, 0] for n in ("B", "C")]
    with pytest.raises(ms.MambaScanError):     # more rows than states, and no slots
        ms.heads_state_update(st[:1], *one)
    with pytest.raises(TypeError):
        ms.heads_state_update(st, *one, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert torch.equal(st, g["h0"])


# --------------------------------------------------------------------------- convolution

CONV = [(1, 1, 1, 2), (2, 2, 7, 4), (1, 5, 64, 3), (2, 16, 24, 4), (3, 65, 40, 4), (1, 130, 520, 4),
        (2, 333, 33, 2), (1, 64, 1032, 3)]     # (batch, L, dim, W)


def conv_inputs(seed, dtype, batch, L, dim, W, window, reset):
    r = R.Inputs(seed, dtype)
    return dict(x=r.seq(batch, L, dim), w=r.f32(dim, W, scale=0.5), b=r.f32(dim, scale=0.5),
                window=r.seq(batch, W - 1, dim) if window else None,
                reset=None if reset is None else r.flags(batch, L, reset),
                dout=r.seq(batch, L, dim))


def conv_dev(i, dtype):
    return {k: None if v is None else v.cuda() if v.dtype == torch.uint8 else
            v.to(dtype if k in ("x", "window", "dout") else torch.float32).cuda()
            for k, v in i.items()}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reset", [None, "random", "every", "edges"])
@pytest.mark.parametrize("size", CONV)
def test_conv_forward_and_backward(ms, size, reset, dtype):
    i = conv_inputs(31, DT[dtype], *size, window=size[1] % 2 == 1, reset=reset)
    g = conv_dev(i, DT[dtype])
    out, win = ms.conv1d_tokens_fwd(g["x"], g["w"], g["b"], window=g["window"], reset=g["reset"],
                                    return_window=True)
    ro, rw = R.conv_fwd(i["x"], i["w"], i["b"], i["window"], i["reset"])
    R.check("out", out, ro)
    assert torch.equal(win.double().cpu(), rw)
    got = ms.conv1d_tokens_bwd(g["x"], g["w"], g["b"], g["dout"], window=g["window"],
                               reset=g["reset"])
    want = R.autograd(lambda x, w, b, win: R.conv_fwd(x, w, b, win, i["reset"])[0],
                      [i["x"], i["w"], i["b"], i["window"]], i["dout"])
    pre_terms = i["dout"].square().sum((0, 1)).sqrt()
    for n, r in zip(("dx", "dw", "db", "dwindow"), want):
        if r is None:
            assert n not in got
            continue
        scale = {"dw": pre_terms.unsqueeze(1).expand_as(i["w"]), "db": pre_terms}.get(n)
        R.check(n, got[n], r, scale)


def test_conv_of_a_view_and_without_bias(ms):
    i = conv_inputs(32, torch.bfloat16, 2, 50, 48, 4, True, None)
    g = conv_dev(i, torch.bfloat16)
    wide = torch.randn(2, 50, 100, device="cuda").bfloat16()
    for o in (8, 5):
        v = wide[..., o:o + 48]
        v.copy_(g["x"])
        out = ms.conv1d_tokens_fwd(v, g["w"], None, window=g["window"])
        R.check("out", out, R.conv_fwd(i["x"], i["w"], None, i["window"])[0])
        got = ms.conv1d_tokens_bwd(v, g["w"], None, g["dout"], window=g["window"])
        assert set(got) == {"dx", "dw", "dwindow"}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,W", [(1, 2), (7, 4), (64, 3), (520, 4), (1792, 4)])
def test_conv_token_by_token_over_a_pool(ms, dim, W, dtype):
    b, pool = 4, 6
    i = conv_inputs(33, DT[dtype], b, 7, dim, W, True, None)
    g = conv_dev(i, DT[dtype])
    ro, rw = R.conv_fwd(i["x"], i["w"], i["b"], i["window"])
    slots = torch.tensor([5, 2, 0, 3], dtype=torch.int32, device="cuda")
    wins = torch.full((pool, W - 1, dim), 9.0, dtype=DT[dtype], device="cuda")
    wins[slots.long()] = g["window"]
    for t in range(7):
        out = ms.conv1d_tokens_update(g["x"][:, t], wins, g["w"], g["b"], slots=slots)
        R.check("out", out, ro[:, t])
    assert torch.equal(wins[slots.long()].double().cpu(), rw)
    assert (wins[[1, 4]] == 9.0).all()
    before = wins.clone()
    slots[1], slots[2] = -1, pool
    out = ms.conv1d_tokens_update(g["x"][:, 0], wins, g["w"], g["b"], slots=slots)
    assert not out[1:3].any() and out[[0, 3]].any()
    assert torch.equal(wins[[2, 0]], before[[2, 0]])


def test_conv_keeps_non_finite_values_in_their_sequence(ms):
    for dtype in (torch.float32, torch.bfloat16):
        i = conv_inputs(34, dtype, 1, 60, 64, 4, False, "random")
        i["reset"][:] = 0
        i["reset"][0, 30] = 1
        g = conv_dev(i, dtype)
        kw = dict(reset=g["reset"])
        clean = ms.conv1d_tokens_fwd(g["x"], g["w"], g["b"], **kw)
        cleanb = ms.conv1d_tokens_bwd(g["x"], g["w"], g["b"], g["dout"], **kw)
        for at in (29, 30):
            x = g["x"].clone()
            x[0, at] = float("nan")
            out = ms.conv1d_tokens_fwd(x, g["w"], g["b"], **kw)
            got = ms.conv1d_tokens_bwd(x, g["w"], g["b"], g["dout"], **kw)
            other = slice(30, 60) if at == 29 else slice(0, 30)
            assert torch.equal(out[0, other], clean[0, other])
            assert torch.equal(got["dx"][0, other], cleanb["dx"][0, other])
            assert torch.isnan(out[0, at]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [24, 21])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_reaches_no_further_than_its_width(ms, W, dim, dtype):
    """An infinity or NaN reaches the W tokens that weigh it and no other, either way."""
    i = conv_inputs(36, DT[dtype], 2, 70, dim, W, True, None)
    g = conv_dev(i, DT[dtype])
    clean = ms.conv1d_tokens_fwd(g["x"], g["w"], g["b"], window=g["window"])
    cleanb = ms.conv1d_tokens_bwd(g["x"], g["w"], g["b"], g["dout"], window=g["window"])
    for at in (0, 14, 31, 69):
        x, dout = g["x"].clone(), g["dout"].clone()
        x[0, at] = float("inf") if at % 2 else float("nan")
        dout[0, at] = x[0, at]
        out = ms.conv1d_tokens_fwd(x, g["w"], g["b"], window=g["window"])
        got = ms.conv1d_tokens_bwd(g["x"], g["w"], g["b"], dout, window=g["window"])
        reach = torch.arange(70, device="cuda")
        near = (reach >= at) & (reach < at + W)
        assert torch.equal(out[0, ~near], clean[0, ~near]) and torch.equal(out[1], clean[1])
        near = (reach <= at) & (reach > at - W)
        assert torch.equal(got["dx"][0, ~near], cleanb["dx"][0, ~near])
        assert torch.equal(got["dx"][1], cleanb["dx"][1])
        near = torch.arange(1 - W, 0, device="cuda") > at - W
        assert torch.equal(got["dwindow"][0, ~near], cleanb["dwindow"][0, ~near])


def test_conv_autograd_and_refusals(ms):
    i = conv_inputs(35, torch.float32, 2, 40, 24, 4, True, None)
    g = conv_dev(i, torch.float32)
    v = {n: g[n].clone().requires_grad_(True) for n in ("x", "w", "b", "window")}
    (ms.conv1d_tokens(v["x"], v["w"], v["b"], window=v["window"]) * g["dout"]).sum().backward()
    got = ms.conv1d_tokens_bwd(g["x"], g["w"], g["b"], g["dout"], window=g["window"])
    assert all(torch.equal(v[n].grad, got["d" + n]) for n in v)
    with pytest.raises(ms.MambaScanError):
        ms.conv1d_tokens_fwd(g["x"], g["w"].new_zeros(24, 5))
    with pytest.raises(ms.MambaScanError):
        ms.conv1d_tokens_fwd(g["x"][:, :0], g["w"])
    with pytest.raises(ValueError):
        ms.conv1d_tokens_fwd(g["x"].transpose(1, 2), g["w"].new_zeros(40, 4))
    with pytest.raises(ValueError):
        ms.conv1d_tokens_fwd(g["x"], g["w"], window=g["window"][:, :2])
    with pytest.raises(TypeError):
        ms.conv1d_tokens_fwd(g["x"].double(), g["w"])


# --------------------------------------------------------------------------- norm

NORM = [(1, 1, 1), (3, 7, 1), (5, 64, 2), (70, 512, 1), (9, 1536, 1), (6, 5120, 8), (3, 2056, 1),
        (2, 8192, 1), (2, 9000, 1), (4, 10240, 1), (3, 36, 4), (1100, 24, 3)]   # (rows, dim, groups)


def norm_inputs(seed, dtype, rows, dim):
    r = R.Inputs(seed, dtype)
    return dict(x=r.seq(rows, dim), z=r.seq(rows, dim), w=1 + r.f32(dim, scale=0.2),
                dout=r.seq(rows, dim))


def norm_dev(i, dtype):
    return {k: v.to(torch.float32 if k == "w" else dtype).cuda() for k, v in i.items()}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["first", "last", "none"])
@pytest.mark.parametrize("size", NORM)
def test_norm_forward_and_backward(ms, size, gate, dtype):
    rows, dim, groups = size
    i = norm_inputs(41, DT[dtype], rows, dim)
    i["x"][0] = 0.0          # a row without anything: eps alone
    g = norm_dev(i, DT[dtype])
    z = None if gate == "none" else g["z"]
    kw = dict(groups=groups, gate_first=gate != "last")
    out = ms.gated_norm_fwd(g["x"], z, g["w"], **kw)
    fn = lambda x, z, w: R.norm_fwd(x, z, w, groups, 1e-5, gate != "last")  # noqa: E731
    rz = None if z is None else i["z"]
    R.check("out", out, fn(i["x"], rz, i["w"]))
    got = ms.gated_norm_bwd(g["x"], z, g["w"], g["dout"], **kw)
    want = R.autograd(fn, [i["x"], rz, i["w"]], i["dout"])
    terms = i["dout"].square().sum(0).sqrt()
    for n, r in zip(("dx", "dz", "dweight"), want):
        if r is None:
            assert n not in got
            continue
        if n == "dx":      # the empty row's gradient is 1/sqrt(eps) times the others'
            R.check("dx", got[n][1:], r[1:]) if rows > 1 else None
            R.check("dx0", got[n][:1], r[:1])
        else:
            R.check(n, got[n], r, terms if n == "dweight" else None)


def test_norm_of_views_without_weight_and_of_more_dimensions(ms):
    r = torch.randn(2, 10, 100, device="cuda")
    for o in (0, 3):
        x, z = r[..., o:o + 40], r[..., 44 + o:84 + o]
        out = ms.gated_norm_fwd(x, z, None, groups=2)
        assert out.shape == x.shape
        R.check("out", out, R.norm_fwd(x.double().cpu(), z.double().cpu(), None, 2, 1e-5, True))
        assert set(ms.gated_norm_bwd(x, z, None, torch.ones_like(out), groups=2)) == {"dx", "dz"}


def test_norm_autograd_and_refusals(ms):
    i = norm_inputs(42, torch.float32, 6, 64)
    g = norm_dev(i, torch.float32)
    v = {n: g[n].clone().requires_grad_(True) for n in ("x", "z", "w")}
    (ms.gated_norm(v["x"], v["z"], v["w"], groups=4) * g["dout"]).sum().backward()
    got = ms.gated_norm_bwd(g["x"], g["z"], g["w"], g["dout"], groups=4)
    assert torch.equal(v["x"].grad, got["dx"]) and torch.equal(v["w"].grad, got["dweight"])
    with pytest.raises(ms.MambaScanError):
        ms.gated_norm_fwd(g["x"], g["z"], g["w"], groups=5)
    with pytest.raises(ms.MambaScanError):
        ms.gated_norm_fwd(g["x"], g["z"], g["w"], eps=-1.0)
    with pytest.raises(ms.MambaScanError):
        ms.gated_norm_fwd(g["x"][:0], g["z"][:0], g["w"])
    with pytest.raises(ValueError):
        ms.gated_norm_fwd(g["x"], g["z"][:3], g["w"])
    with pytest.raises(ValueError):
        ms.gated_norm_fwd(g["x"].t(), None, None)
    with pytest.raises(TypeError):
        ms.gated_norm_fwd(g["x"], g["z"].bfloat16(), g["w"])


# --------------------------------------------------------------------------- capture

def test_captured_calls_replay(ms):
    """The whole mixer's calls in one graph, replayed over changed inputs."""
    i = R.scan_inputs(51, torch.bfloat16, 2, 200, 4, 64, 1, 64)
    g = dev(i, torch.bfloat16)
    dim = 4 * 64
    w = torch.randn(dim, 4, device="cuda") * 0.5
    z = torch.randn(2, 200, dim, device="cuda").bfloat16()
    nw = torch.ones(dim, device="cuda")
    st = torch.zeros(2, 4, 64, 64, device="cuda")
    win = torch.zeros(2, 3, dim, device="cuda").bfloat16()
    x = g["u"].flatten(2).contiguous()

    def calls():
        c = ms.conv1d_tokens_fwd(x, w)
        out = ms.heads_scan_fwd(c.unflatten(-1, (4, 64)), g["delta"], g["A"], g["B"], g["C"],
                                g["D"], g["delta_bias"])
        y = ms.gated_norm_fwd(out.flatten(2), z, nw)
        d = ms.gated_norm_bwd(out.flatten(2), z, nw, y)
        b = ms.heads_scan_bwd(c.unflatten(-1, (4, 64)), g["delta"], g["A"], g["B"], g["C"],
                              g["D"], g["delta_bias"], d["dx"].unflatten(-1, (4, 64)))
        e = ms.conv1d_tokens_bwd(x, w, None, b["du"].flatten(2))
        t = ms.conv1d_tokens_update(x[:, 0], win, w)
        o = ms.heads_state_update(st, t.unflatten(-1, (4, 64)), g["delta"][:, 0], g["A"],
                                  g["B"][:, 0], g["C"][:, 0], g["D"], g["delta_bias"])
        return [y, o, e["dx"], e["dw"], d["dweight"], st, win] + [b[k] for k in sorted(b)]

    def fresh(k):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)).bfloat16())
        st.zero_()
        win.zero_()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for k in range(3):
        fresh(k)
        want = [t.clone() for t in calls()]
        for t in outs:
            if t is not st and t is not win:
                t.fill_(7)
        fresh(k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
