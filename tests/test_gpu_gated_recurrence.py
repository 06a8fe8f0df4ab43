"""The gated linear recurrence on the GPU against the 64-bit reference: lengths and
widths around every tile border, both types, packed rows, views, pools of
states, saturated gates, values that are not finite, and what is refused."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SEQ = ("x", "r", "i", "z", "dout")
# (batch, L, dim)
SIZES = [(1, 1, 1), (3, 1, 130), (1, 2, 64), (2, 15, 3), (1, 16, 128), (2, 17, 65), (1, 63, 127),
         (2, 64, 256), (1, 65, 129), (3, 127, 66), (1, 128, 1000), (2, 129, 514), (1, 200, 1536),
         (2, 513, 130), (1, 1025, 192), (2, 2311, 70), (1, 4500, 34)]


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def dev(i, dtype):
    return {k: None if v is None else v.cuda() if v.dtype == torch.uint8 else
            v.to(dtype if k in SEQ else torch.float32).cuda() for k, v in i.items()}


def run_fwd(ms, g, **kw):
    return ms.gated_recurrence_fwd(g["x"], g["r"], g["i"], g["A"], g["z"], g["h0"],
                                   reset=g["reset"], return_last_state=True, **kw)


def run_bwd(ms, g, dlast=True, **kw):
    return ms.gated_recurrence_bwd(g["x"], g["r"], g["i"], g["A"], g["z"], g["dout"], g["h0"],
                                   dlast_state=g["dlast"] if dlast else None, reset=g["reset"],
                                   **kw)


def check_fwd(got, i):
    out, last, _ = R.rec_fwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["h0"], i["reset"])
    R.check("out", got[0], out)
    R.check("last_state", got[1], last)


def check_bwd(got, i, dlast=True):
    ref, scale = R.rec_bwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["dout"], i["h0"],
                           i["dlast"] if dlast else None, i["reset"])
    assert set(got) == set(ref)
    for k in ref:
        R.check(k, got[k], ref[k], scale.get(k))


def kept(ms, g):
    b, L, d = g["x"].shape
    c = torch.full(ms.gated_recurrence_checkpoint_shape(b, L, d), float("nan"), device="cuda")
    run_fwd(ms, g, checkpoints=c)
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_forward(ms, size, z, dtype):
    i = R.rec_inputs(1, DT[dtype], *size, z=z, h0=size[1] % 2 == 1)
    got = run_fwd(ms, dev(i, DT[dtype]))
    assert got[0].dtype == DT[dtype] and got[1].dtype == torch.float32
    check_fwd(got, i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_backward(ms, size, z, dtype):
    i = R.rec_inputs(2, DT[dtype], *size, z=z, h0=size[1] % 2 == 1)
    g = dev(i, DT[dtype])
    got = run_bwd(ms, g)
    assert all(v.dtype == (DT[dtype] if k in ("dx", "dr", "di", "dz") else torch.float32)
               for k, v in got.items())
    check_bwd(got, i)
    with_kept = run_bwd(ms, g, checkpoints=kept(ms, g))
    for k in got:      # the checkpoints are the states that it forms itself
        assert torch.equal(got[k], with_kept[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reset", ["random", "every", "edges"])
@pytest.mark.parametrize("size", [(2, 1, 5), (2, 129, 64), (3, 300, 130), (2, 2311, 33)])
def test_packed(ms, size, reset, dtype):
    i = R.rec_inputs(3, DT[dtype], *size, reset=reset)
    g = dev(i, DT[dtype])
    check_fwd(run_fwd(ms, g), i)
    check_bwd(run_bwd(ms, g, checkpoints=kept(ms, g)), i)
    check_bwd(run_bwd(ms, g, dlast=False), i, dlast=False)
    flags = g["reset"].bool()
    assert torch.equal(run_fwd(ms, dict(g, reset=flags))[0], run_fwd(ms, g)[0])


@pytest.mark.parametrize("size", [(2, 70, 6), (1, 300, 128), (2, 2100, 40)])
def test_checkpoints_are_the_states(ms, size):
    i = R.rec_inputs(4, torch.float32, *size)
    _, _, before = R.rec_fwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["h0"])
    R.check("checkpoints", kept(ms, dev(i, torch.float32)), before[:, ::64])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,off", [(64, 0), (64, 1), (130, 2), (33, 3), (256, 8)])
def test_views_of_wider_rows(ms, dim, off, dtype):
    """x, r, i, z as parts of one row a token, at any offset."""
    i = R.rec_inputs(5, DT[dtype], 2, 150, dim)
    g = dev(i, DT[dtype])
    wide = torch.randn(2, 150, 4 * dim + 3 * off + 7, device="cuda").to(DT[dtype])
    v = dict(g)
    for k, name in enumerate("xriz"):
        at = off + k * dim + (k * off if k < 3 else 2 * off)
        wide[..., at:at + dim] = g[name]
        v[name] = wide[..., at:at + dim]
    before = wide.clone()
    assert all(torch.equal(a, b) for a, b in zip(run_fwd(ms, v), run_fwd(ms, g)))
    a, b = run_bwd(ms, v), run_bwd(ms, g)
    assert all(torch.equal(a[k], b[k]) for k in a) and torch.equal(wide, before)
    # one row for every batch row, and one token for every token
    one = dict(g, x=g["x"][:1].expand(2, 150, dim), r=g["r"][:, :1].expand(2, 150, dim))
    dense = dict(one, x=one["x"].contiguous(), r=one["r"].contiguous())
    assert torch.equal(run_fwd(ms, one)[0], run_fwd(ms, dense)[0])
    a, b = run_bwd(ms, one), run_bwd(ms, dense)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_a_prompt_in_pieces_and_single_tokens(ms):
    """Whole, in pieces through last_state (in place, too), and token by token."""
    i = R.rec_inputs(6, torch.float32, 2, 400, 192)
    g = dev(i, torch.float32)
    whole, last = run_fwd(ms, g)
    part = lambda a, b: {k: v[:, a:b] if k in ("x", "r", "i", "z") else v  # noqa: E731
                         for k, v in g.items()}
    state, outs = g["h0"].clone(), []
    for a, b in ((0, 1), (1, 200), (200, 390)):
        p = dict(part(a, b), h0=state)
        o, s = run_fwd(ms, p, last_state=state)
        assert s.data_ptr() == state.data_ptr()
        outs.append(o)
    for t in range(390, 400):
        p = part(t, t + 1)
        outs.append(ms.gated_recurrence_update(state, *(p[k][:, 0] for k in "xri"), g["A"],
                                               p["z"][:, 0])[:, None])
    R.check("out", torch.cat(outs, 1), whole)
    R.check("state", state, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1), (5, 3), (3, 64), (7, 130), (256, 515), (2, 4096)])
def test_update(ms, size, dtype):
    batch, dim = size
    i = R.rec_inputs(7, DT[dtype], batch, 1, dim)
    g = dev(i, DT[dtype])
    out, last, _ = R.rec_fwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["h0"])
    pool = torch.randn(2 * batch + 3, dim, device="cuda")
    slots = torch.randperm(2 * batch + 3, device="cuda")[:batch].to(torch.int32)
    pool[slots.long()] = g["h0"]
    others = pool.clone()
    got = ms.gated_recurrence_update(pool, *(g[k][:, 0] for k in "xri"), g["A"], g["z"][:, 0],
                                     slots=slots)
    R.check("out", got, out[:, 0])
    R.check("state", pool[slots.long()], last)
    others[slots.long()] = pool[slots.long()]
    assert torch.equal(pool, others)
    # without slots row b steps state b; without z out is the state; rows may be views
    state = g["h0"].clone()
    wide = torch.cat([g["r"][:, 0], g["i"][:, 0]], 1)
    got = ms.gated_recurrence_update(state, g["x"][:, 0], wide[:, :dim], wide[:, dim:], g["A"])
    assert torch.equal(state, pool[slots.long()])
    assert torch.equal(got, state.to(DT[dtype]))
    # a slot outside the pool: its row is zero and no state moves
    bad = slots.clone()
    bad[0], before = -1, pool.clone()
    got = ms.gated_recurrence_update(pool, *(g[k][:, 0] for k in "xri"), g["A"], slots=bad)
    assert not got[0].any() and torch.equal(pool[slots[0].long()], before[slots[0].long()])
    bad[0] = len(pool)
    got = ms.gated_recurrence_update(pool, *(g[k][:, 0] for k in "xri"), g["A"], slots=bad)
    assert not got[0].any() and torch.equal(pool[slots[0].long()], before[slots[0].long()])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_saturated_gates(ms, dtype):
    """Gates from shut to open: decays from 1 - 1e-18 to nothing, and A from 0 to -1e6."""
    i = R.rec_inputs(8, DT[dtype], 2, 200, 128)
    i["r"] = R.stored(i["r"] * 30, DT[dtype])
    i["i"] = R.stored(i["i"] * 30, DT[dtype])
    i["A"][:8] = torch.tensor([-1e-30, -1e-6, -1e-3, -50, -1e3, -1e6, -80, -104.0],
                              dtype=torch.float64)
    g = dev(i, DT[dtype])
    check_fwd(run_fwd(ms, g), i)
    got = run_bwd(ms, g)
    ref, scale = R.rec_bwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["dout"], i["h0"], i["dlast"])
    for k in ref:    # dA by channel: that of A = -1e-30 is 1e13 times the others'
        if k == "dA":
            assert ((got[k].double().cpu() - ref[k]).abs() <= 2e-5 * scale[k] + 1e-30).all()
        else:
            R.check(k, got[k], ref[k])
    g["A"][:3] = 0.0     # keeps its state, nothing enters
    out, last = run_fwd(ms, dict(g, z=None))
    assert torch.equal(last[:, :3], g["h0"][:, :3])
    assert torch.equal(out[:, :, :3], g["h0"][:, None, :3].expand(2, 200, 3).to(DT[dtype]))
    got = run_bwd(ms, g)
    assert all(torch.isfinite(got[k]).all() for k in ("dx", "dr", "di", "dz", "dh0"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["x", "r", "i", "h0"])
def test_non_finite_values_stay_in_their_sequence(ms, name, value, dtype):
    """A value that is not finite reaches no other channel and no other sequence's
    rows; in the forward, nothing before it."""
    L, at, flag = 1300, 700, 1100
    i = R.rec_inputs(9, DT[dtype], 2, L, 66)
    i["reset"] = torch.zeros(2, L, dtype=torch.uint8)
    i["reset"][0, flag] = 1
    i["reset"][0, 400] = 1
    g = dev(i, DT[dtype])
    clean_out, clean_last = run_fwd(ms, g)
    clean = run_bwd(ms, g)
    bad = dict(g)
    bad[name] = g[name].clone()
    if name == "h0":
        bad[name][0, 5] = value
        hit = slice(0, 400)
    else:
        bad[name][0, at, 5] = value
        hit = slice(at, flag)
    out, last = run_fwd(ms, bad)
    same = torch.ones_like(out, dtype=torch.bool)
    same[0, hit, 5] = False
    assert torch.equal(out[same], clean_out[same]) and torch.equal(last, clean_last)
    if name in ("x", "h0") or value != value:
        assert not torch.isfinite(out[0, hit.start, 5])
    got = run_bwd(ms, bad)
    for k in ("dx", "dr", "di", "dz"):
        same = torch.ones_like(out, dtype=torch.bool)
        same[0, 400 if name != "h0" else 0:flag if name != "h0" else 400, 5] = False
        assert torch.equal(got[k][same], clean[k][same]), k
    keep = torch.arange(66, device="cuda") != 5
    assert torch.equal(got["dA"][keep], clean["dA"][keep])
    assert torch.equal(got["dh0"][:, keep], clean["dh0"][:, keep])


def test_gradients_through_autograd(ms):
    i = R.rec_inputs(10, torch.float32, 2, 333, 70, reset="random")
    g = dev(i, torch.float32)
    names = ("x", "r", "i", "A", "z", "h0")
    leaf = {k: g[k].clone().requires_grad_(True) for k in names}
    out, last = ms.gated_recurrence(*(leaf[k] for k in names), reset=g["reset"],
                                    return_last_state=True)
    grads = torch.autograd.grad([out, last], [leaf[k] for k in names], [g["dout"], g["dlast"]])
    check_bwd({"d" + k: v for k, v in zip(names, grads)}, i)
    # through the last state alone, and with flags as truth values
    _, last = ms.gated_recurrence(*(leaf[k] for k in names), reset=g["reset"].bool(),
                                  return_last_state=True)
    grads = torch.autograd.grad(last, [leaf[k] for k in names], g["dlast"])
    check_bwd({"d" + k: v for k, v in zip(names, grads)}, dict(i, dout=i["dout"] * 0))
    loss = ms.gated_recurrence(*(leaf[k] for k in names)).square().sum()
    (d,) = torch.autograd.grad(loss, leaf["x"], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(d.square().sum() + leaf["x"].sum(), leaf["x"])


def test_gradients_against_differences(ms):
    """Along random directions: central differences of the forward in float32.  The
    loss's rounding is about 1e-6 of its terms' root sum of squares, over a step of
    2 2^-6; the difference's own error is of the order of 2^-12 of the third
    derivative."""
    i = R.rec_inputs(11, torch.float32, 2, 150, 64)
    g = dev(i, torch.float32)
    got = run_bwd(ms, g, dlast=False)
    h = 2.0 ** -6

    def loss(k, v):
        return float((run_fwd(ms, dict(g, **{k: v}))[0].double() * g["dout"].double()).sum())
    for k in ("x", "r", "i", "z", "A", "h0"):
        u = torch.randn(g[k].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        u = u * g["A"].abs() if k == "A" else u
        want = (loss(k, g[k] + h * u) - loss(k, g[k] - h * u)) / (2 * h)
        have = float((got["d" + k].double() * u.double()).sum())
        size = float((got["d" + k].double() * u.double()).norm())
        assert abs(want - have) < 2e-2 * size + 1e-3 * abs(have), (k, want, have, size)


@pytest.mark.parametrize("size", [(1, 130, 64), (2, 2311, 70)])
def test_outputs_are_overwritten_and_equal_calls_give_equal_bits(ms, size):
    i = R.rec_inputs(12, torch.bfloat16, *size)
    g = dev(i, torch.bfloat16)
    b, L, d = size
    guard = 64

    def padded(shape, dtype):
        n = torch.Size(shape).numel()
        flat = torch.full((n + 2 * guard,), float("nan"), dtype=dtype, device="cuda")
        return flat, flat[guard:guard + n].view(shape)
    out_, out = padded((b, L, d), torch.bfloat16)
    last_, last = padded((b, d), torch.float32)
    ck_, ck = padded(ms.gated_recurrence_checkpoint_shape(b, L, d), torch.float32)
    nw = ms.gated_recurrence_fwd_workspace_bytes(b, L, d, torch.bfloat16)
    ws = torch.full((nw + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    run_fwd(ms, g, out=out, last_state=last, checkpoints=ck, workspace=ws)
    assert (ws[nw:] == 0xA5).all()
    for flat, t in ((out_, out), (last_, last), (ck_, ck)):
        assert torch.isfinite(t).all() and not torch.isfinite(flat[:guard]).any()
        assert not torch.isfinite(flat[-guard:]).any()
    first = [out.clone(), last.clone(), ck.clone()]
    grads = run_bwd(ms, g, checkpoints=ck)
    for _ in range(3):
        again = run_fwd(ms, g, checkpoints=ck, workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        assert torch.equal(ck, first[2])
        more = run_bwd(ms, g, checkpoints=ck)
        assert all(torch.equal(more[k], grads[k]) for k in grads)
    nw = ms.gated_recurrence_bwd_workspace_bytes(b, L, d, torch.bfloat16, with_checkpoints=False)
    ws = torch.full((nw + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    more = run_bwd(ms, g, workspace=ws)
    assert (ws[nw:] == 0xA5).all() and all(torch.equal(more[k], grads[k]) for k in grads)


def test_refusals(ms):
    g = dev(R.rec_inputs(13, torch.float32, 2, 20, 8), torch.float32)
    run = lambda **kw: run_fwd(ms, dict(g, **kw))  # noqa: E731
    for bad in (dict(x=g["x"].cpu()), dict(r=g["r"][:, :19]), dict(A=g["A"][:7]),
                dict(h0=g["h0"][:1]), dict(x=g["x"].transpose(1, 2)),
                dict(z=g["z"][..., ::2].expand(2, 20, 4)), dict(reset=torch.zeros(2, 19,
                     dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            run(**bad)
    for bad in (dict(r=g["r"].bfloat16()), dict(A=g["A"].double()), dict(i=None),
                dict(x=g["x"].half())):
        with pytest.raises(TypeError):
            run(**bad)
    with pytest.raises(ValueError):
        run_fwd(ms, g, checkpoints=torch.empty(2, 2, 8, device="cuda"))
    with pytest.raises(ValueError):
        run_fwd(ms, g, workspace=torch.empty(1 << 20, device="cpu"))
    with pytest.raises(TypeError):
        run_bwd(ms, dict(g, dout=None))
    empty = {k: v[:, :0] if k in SEQ else v for k, v in g.items()}
    with pytest.raises(ms.MambaScanError):
        run_fwd(ms, empty)
    with pytest.raises(ms.MambaScanError):      # a part of h0
        both = torch.zeros(24, device="cuda")
        run_fwd(ms, dict(g, h0=both[:16].view(2, 8)), last_state=both[8:24].view(2, 8))
    with pytest.raises(ms.MambaScanError):      # out over an input
        run_fwd(ms, g, out=g["x"])
    with pytest.raises(ValueError):
        ms.gated_recurrence_update(g["h0"], g["x"][:, 0], g["r"][:, 0], g["i"][:1, 0], g["A"])
    with pytest.raises(ms.MambaScanError):      # fewer states than rows
        ms.gated_recurrence_update(g["h0"][:1], g["x"][:, 0], g["r"][:, 0], g["i"][:, 0], g["A"])
    with pytest.raises(TypeError):
        ms.gated_recurrence_update(g["h0"], g["x"][:, 0], g["r"][:, 0], g["i"][:, 0], g["A"],
                                   slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
