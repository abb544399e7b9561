"""The operators of ttt_ops.h against their formulas in 64 bits (tests/ops_ref.py), within the
bounds derived there, at the sizes, layouts and masks where they can go wrong."""
import math

import pytest
import torch

from tests import ops_ref as ref

pytestmark = pytest.mark.gpu
DT = ref.DT


def _ops():
    from weight_sequence_mixing_b200 import token_ops
    return token_ops


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float32)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------- rope
# B, H, N, pairs, d, pairing, dtype, layout of x ("heads": [B,H,N,d], "tokens": [B,N,H,d],
# "slice": columns of a wider [B,N,3Hd] buffer, "odd": one element past 16-byte alignment)
ROPE = [
    (1, 1, 1, (4,), 8, "halves", "bf16", "heads"),
    (8, 6, 1, (16, 16), 64, "halves", "bf16", "heads"),
    (2, 3, 37, (16, 16), 64, "halves", "bf16", "tokens"),
    (2, 3, 37, (16, 16), 64, "interleaved", "bf16", "slice"),
    (1, 2, 129, (32, 80, 80), 512, "interleaved", "bf16", "tokens"),
    (1, 2, 65, (32, 80, 80), 512, "halves", "bf16", "heads"),
    (3, 5, 41, (8, 12, 12), 80, "halves", "f32", "heads"),
    (3, 5, 41, (8, 12, 12), 80, "interleaved", "f32", "tokens"),
    (2, 2, 19, (7, 11), 38, "halves", "bf16", "heads"),
    (2, 2, 19, (7, 11), 37, "interleaved", "f32", "odd"),
    (2, 16, 33, (8,), 20, "halves", "bf16", "tokens"),
    (1, 3, 23, (1, 1, 1, 1), 9, "interleaved", "bf16", "odd"),
    (1, 40, 3, (64,), 128, "halves", "f32", "slice"),
    (2, 1, 300, (128, 128), 512, "halves", "f32", "heads"),
]


def _layout(x, layout):
    """x [B,H,N,d] on the GPU with the same values and other strides."""
    B, H, N, d = x.shape
    if layout == "tokens":
        return x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    if layout == "slice":
        wide = torch.full((B, N, 3, H, d), math.nan, dtype=x.dtype, device="cuda")
        wide[:, :, 1] = x.transpose(1, 2).cuda()
        return wide[:, :, 1].transpose(1, 2)
    if layout == "odd":
        flat = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        flat[1:] = x.reshape(-1).cuda()
        return flat[1:].view(B, H, N, d)
    return x.cuda()


def _positions(gen, B, N, axes, kind):
    if kind == "f32":
        return (torch.rand((N, axes), generator=gen) * 300 - 50).float()
    top = 2 ** 31 - 1 if kind == "far" else 1_100_000
    shape = (B, N, axes) if kind == "each" else (N, axes)
    return torch.randint(-1000, top, shape, generator=gen, dtype=torch.int64).to(torch.int32)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("positions", ["shared", "each", "f32", "far"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_rope(case, positions, inverse):
    B, H, N, pairs, d, pairing, dtype, layout = case
    gen = _gen(7)
    x = _randn(gen, B, H, N, d).to(DT[dtype])
    pos = _positions(gen, B, N, len(pairs), positions)
    base = [100.0 * 7 ** i for i in range(len(pairs))]
    op = _ops().RotaryPositions(dict(d=d, pairs=pairs, base=base, pairing=pairing, dtype=dtype))
    xd = _layout(x, layout)
    y = (op.backward if inverse else op.forward)(xd, pos.cuda())
    want, err = ref.rope(x.double(), pos, pairs, base, pairing, inverse)
    assert y.is_contiguous()
    ref.check("y", y, want, ref.rounded(want, err, DT[dtype]))
    # the copied channels are the same bits
    assert torch.equal(y[..., 2 * sum(pairs):].cpu(), x[..., 2 * sum(pairs):])
    # in the input's place, and into a given tensor with other strides: the same values
    other = torch.empty((B, N, H, d), dtype=DT[dtype], device="cuda").transpose(1, 2)
    assert (op.backward if inverse else op.forward)(xd, pos.cuda(), out=other) is other
    assert torch.equal(other, y)
    (op.backward if inverse else op.forward)(xd, pos.cuda(), out=xd)
    assert torch.equal(xd, y)


def test_rope_backward_is_the_gradient_of_forward():
    """<dy, rope(x)> is linear in x: its difference along a direction is <rope.backward(dy), direction>."""
    gen = _gen(3)
    x, v, dy = (_randn(gen, 2, 3, 29, 80) for _ in range(3))
    pos = _positions(gen, 2, 29, 3, "shared")
    op = _ops().RotaryPositions(dict(d=80, pairs=(8, 12, 12), dtype="f32"))
    f = lambda t: (op.forward(t.cuda(), pos.cuda()).double().cpu() * dy.double()).sum()  # noqa: E731
    got = (op.backward(dy.cuda(), pos.cuda()).double().cpu() * v.double()).sum()
    step = 0.5
    want = (f(x + step * v) - f(x - step * v)) / (2 * step)
    # each value of x +- step v and of either rotation is off by at most 2^-20 (|x_p| + |x_q|); summed against dy
    size = 2 * (x.abs() + v.abs()).double().sum() * 2.0 ** -20 * float(dy.abs().max()) * 3
    assert abs(got - want) <= size


@pytest.mark.parametrize("kind", [torch.int32, torch.float32])
def test_rope_fp32_keeps_the_digits_of_small_sines(kind):
    """Angles next to every quarter of a turn, of which only the fp32 value of the rest is rounded: p radians for
    the integers p nearest to multiples of pi / 2, and turns of far positions."""
    near = [0, 1, 3, 11, 22, 33, 44, 344, 355, 366, 377, 710, 51819, 52174, 103993, 104348, 208341, 312689, 833719, 1146408,
            4272943, 5419351]
    near = [p * s for p in near for s in (1, -1)]
    pos = torch.tensor(near, dtype=torch.float64).to(kind)[:, None].contiguous()
    x = torch.zeros(1, 1, len(near), 4)
    x[..., 0] = 1.0  # its pair's cosine and sine
    op = _ops().RotaryPositions(dict(d=4, pairs=(2,), base=10000.0, dtype="f32"))
    y = op.forward(x.cuda(), pos.cuda()).cpu()[0, 0].double()
    cos, sin = torch.cos(pos[:, 0].double()), torch.sin(pos[:, 0].double())
    # integers: the frequency is exact to 2^-64 turns, so the angle to |p| 2^-61.3 radians; fp32 positions: it is
    # rounded to 64 bits and so is their product, each 2^-53 of the angle (p radians) at most.  Then relative: the rest's rounding 2^-24, the sine's polynomial 3e-9, its
    # small terms a tenth of a half step and its last sum one; the cosine's last sum one, and three tenths of one
    # before it.  Below 2.5 half steps, and one for the product with 1 and the sum with 0.
    off = pos[:, 0].double().abs() * (2.0 ** -61.3 if kind == torch.int32 else 2.0 ** -52)
    ref.check("cos", y[:, 0], cos, off + 3.5 * ref.E32 * cos.abs())
    ref.check("sin", y[:, 2], sin, off + 3.5 * ref.E32 * sin.abs())


def test_rope_rows_beyond_32_bit_offsets():
    """The last rows of a tensor of more than 2^31 elements, read and written at 64-bit offsets."""
    N, d = (1 << 25) + 3, 72
    x = torch.empty((1, 1, N, d), dtype=torch.bfloat16, device="cuda")
    x.fill_(0.5)
    gen = _gen(5)
    tail = _randn(gen, 1, 1, 5, d).to(torch.bfloat16)
    x[:, :, -5:] = tail.cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].contiguous()
    op = _ops().RotaryPositions(dict(d=d, pairs=(32,), dtype="bf16"))
    y = op.forward(x, pos)
    want, err = ref.rope(tail.double(), pos[-5:].cpu(), (32,), 10000.0, "halves")
    ref.check("tail", y[:, :, -5:], want, ref.rounded(want, err, torch.bfloat16))


# ------------------------------------------------------------------------- scan
# B, L, D, gate, inp, dtype, state, ragged, packed (g and x columns of one buffer)
SCAN = [
    (1, 1, 1, "value", "plain", "f32", True, False, False),
    (8, 1, 384, "sigmoid", "complement", "bf16", True, False, False),
    (2, 2, 64, "exp", "plain", "bf16", False, False, True),
    (3, 37, 70, "sigmoid", "plain", "bf16", True, True, False),
    (2, 64, 128, "exp", "complement", "bf16", True, False, True),
    (2, 255, 33, "value", "complement", "f32", True, True, False),
    (5, 256, 64, "sigmoid", "complement", "bf16", False, True, True),
    (2, 257, 66, "exp", "plain", "f32", True, False, True),
    (1, 513, 8, "sigmoid", "complement", "f32", True, False, False),
    (4, 1030, 72, "sigmoid", "complement", "bf16", True, True, True),
    (1, 2111, 136, "exp", "complement", "bf16", True, False, False),
    (2, 1500, 17, "value", "plain", "bf16", True, True, False),
    (1, 3001, 64, "value", "plain", "f32", False, False, False),
    (70, 40, 24, "sigmoid", "complement", "f32", True, True, False),
]


def _scan_inputs(case, seed=11):
    B, L, D, gate, inp, dtype, state, ragged, packed = case
    gen = _gen(seed)
    z = _randn(gen, B, L, D)
    g = z + 2 if gate == "sigmoid" else -0.3 * torch.nn.functional.softplus(z) if gate == "exp" else \
        1 - 0.3 * torch.sigmoid(z)
    # some gates shut, open and (for values and exponentials) beyond one
    flat = g.view(-1)
    flat[::97] = {"sigmoid": -80.0, "exp": -120.0, "value": 0.0}[gate]
    flat[5::101] = {"sigmoid": 80.0, "exp": 0.0, "value": 1.0}[gate]
    if gate != "sigmoid":
        flat[7::103] = {"exp": 0.05, "value": -1.04}[gate]
    d = dict(g=g, x=_randn(gen, B, L, D), dh=_randn(gen, B, L, D))
    d = {k: v.to(DT[dtype]) for k, v in d.items()}
    d["h0"] = _randn(gen, B, D) if state else None
    d["dh_last"] = _randn(gen, B, D) if state else None
    d["lengths"] = None
    if ragged:
        n = torch.randint(1, L + 1, (B,), generator=gen)
        n[0], n[-1] = L, 0
        if B > 2:
            n[1] = 1
        d["lengths"] = n.to(torch.int32)
    return d


def _put(t, packed=None):
    """On the GPU; packed: as a column range of a wider buffer, NaN beside it."""
    if t is None:
        return None
    if packed is None:
        return t.cuda()
    B, L, D = t.shape
    wide = torch.full((B, L, 2 * D + 1), math.nan, dtype=t.dtype, device="cuda")
    part = wide[..., packed * D:(packed + 1) * D]
    part.copy_(t)
    return part


def _run_scan(case, d, **kw):
    B, L, D, gate, inp, dtype, state, ragged, packed = case
    op = _ops().GatedScan(dict(D=D, gate=gate, inp=inp, dtype=dtype))
    g, x = _put(d["g"], 0 if packed else None), _put(d["x"], 1 if packed else None)
    saved = op.new_saved(B, L)
    saved.fill_(255)  # NaN
    opt = {k: _put(d[k]) for k in ("h0", "lengths")}
    h, h_last = op.forward(g, x, saved=saved, **opt)
    dg, dx, dh0 = op.backward(_put(d["dh"]), g, x, saved, dh_last=_put(d["dh_last"]), lengths=opt["lengths"])
    op.check_status()
    return dict(h=h, h_last=h_last, dg=dg, dx=dx, dh0=dh0)


def _check_scan(case, d, got):
    B, L, D, gate, inp, dtype, state, ragged, packed = case
    want, err = ref.scan(d["g"].double(), d["x"].double(), gate, inp, None if d["h0"] is None else d["h0"].double(),
                         d["lengths"], d["dh"].double(), None if d["dh_last"] is None else d["dh_last"].double())
    for k, v in want.items():
        t = torch.float32 if k in ("h_last", "dh0") else DT[dtype]
        assert got[k].dtype == t
        live = ~torch.isnan(v)
        ref.check(k, got[k].cpu()[live], v[live], ref.rounded(v[live], err[k][live], t))
        assert (got[k].cpu()[~live] == 0).all(), k  # rows behind the end of tensors made by the call


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(map(str, c)))
def test_scan(case):
    d = _scan_inputs(case)
    got = _run_scan(case, d)
    _check_scan(case, d, got)
    # nothing depends on timing
    again = _run_scan(case, d)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("gate", ["value", "sigmoid", "exp"])
@pytest.mark.parametrize("inp", ["plain", "complement"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_every_gate_input_and_type(gate, inp, dtype):
    case = (2, 301, 40, gate, inp, dtype, True, False, False)
    d = _scan_inputs(case, 23)
    _check_scan(case, d, _run_scan(case, d))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 63), ("f32", 40)])
def test_scan_rows_behind_the_end_are_neither_read_nor_written(dtype, D):
    case = (4, 700, D, "sigmoid", "complement", dtype, True, True, False)
    d = _scan_inputs(case)
    d["lengths"] = torch.tensor([700, 0, 513, 1], dtype=torch.int32)
    behind = torch.arange(700)[None, :] >= d["lengths"][:, None]
    for k in ("g", "x", "dh"):
        d[k][behind] = math.nan
    op = _ops().GatedScan(dict(D=D, gate="sigmoid", inp="complement", dtype=dtype))
    g, x, dh, n = d["g"].cuda(), d["x"].cuda(), d["dh"].cuda(), d["lengths"].cuda()
    mark = lambda: torch.full_like(x, 77.0)  # noqa: E731
    saved, h, dg, dx = op.new_saved(4, 700), mark(), mark(), mark()
    _, h_last = op.forward(g, x, h0=d["h0"].cuda(), lengths=n, saved=saved, out=h)
    _, _, dh0 = op.backward(dh, g, x, saved, dh_last=d["dh_last"].cuda(), lengths=n, dg=dg, dx=dx)
    op.check_status()
    for t in (h, dg, dx):
        assert (t.cpu()[behind] == 77.0).all()
        assert torch.isfinite(t.cpu()[~behind]).all()
    # an empty sequence hands its state and its gradient through
    assert torch.equal(h_last[1].cpu(), d["h0"][1]) and torch.equal(dh0[1].cpu(), d["dh_last"][1])
    # lengths out of range are clamped
    wild = torch.tensor([2 ** 31 - 1, -5, 513, 1], dtype=torch.int32, device="cuda")
    h2 = mark()
    d2, last2 = op.forward(torch.nan_to_num(g), torch.nan_to_num(x), h0=d["h0"].cuda(), lengths=wild, out=h2)
    assert torch.equal(h2, h) and torch.equal(last2, h_last)


def test_scan_of_no_tokens_hands_the_state_through():
    op = _ops().GatedScan(dict(D=24, gate="exp", inp="plain", dtype="bf16"))
    e = torch.empty((3, 0, 24), dtype=torch.bfloat16, device="cuda")
    h0, dl = torch.randn(3, 24, device="cuda"), torch.randn(3, 24, device="cuda")
    saved = op.new_saved(3, 0)
    h, last = op.forward(e, e, h0=h0, saved=saved)
    assert h.shape == (3, 0, 24) and torch.equal(last, h0)
    assert torch.equal(op.forward(e, e)[1], torch.zeros_like(h0))
    dg, dx, dh0 = op.backward(e, e, e, saved, dh_last=dl)
    assert dg.shape == dx.shape == (3, 0, 24) and torch.equal(dh0, dl)
    op.check_status()


def test_scan_backward_of_no_tokens_reads_nothing_that_was_not_kept():
    """Many more states than the smallest buffer holds (new_saved gives 16 bytes for no tokens)."""
    B, D = 64, 4096
    op = _ops().GatedScan(dict(D=D, gate="sigmoid", inp="complement", dtype="f32"))
    e, dl = torch.empty((B, 0, D), device="cuda"), torch.randn(B, D, device="cuda")
    saved = op.new_saved(B, 0)
    assert saved.numel() == 16
    dg, dx, dh0 = op.backward(e, e, e, saved, dh_last=dl)
    op.check_status()
    assert dg.shape == dx.shape == (B, 0, D) and torch.equal(dh0, dl)


@pytest.mark.parametrize("dtype,D,parts", [("bf16", 72, (300, 1, 1, 517, 44)), ("f32", 33, (256, 257, 3))])
def test_scan_in_parts_with_the_state_handed_on(dtype, D, parts):
    """The state written in the place of the one read, call after call, against one call over all tokens."""
    case = (2, sum(parts), D, "sigmoid", "complement", dtype, True, False, False)
    d = _scan_inputs(case)
    op = _ops().GatedScan(dict(D=D, gate="sigmoid", inp="complement", dtype=dtype))
    state, at, got = d["h0"].cuda().clone(), 0, []
    for n in parts:
        g, x = d["g"][:, at:at + n].cuda(), d["x"][:, at:at + n].cuda()
        h, last = op.forward(g, x, h0=state, h_last=state)
        assert last is state
        got.append(h)
        at += n
    op.check_status()
    want, err = ref.scan(d["g"].double(), d["x"].double(), "sigmoid", "complement", d["h0"].double())
    ref.check("h", torch.cat(got, 1), want["h"], ref.rounded(want["h"], err["h"], DT[dtype]))
    ref.check("state", state, want["h_last"], ref.rounded(want["h_last"], err["h_last"], torch.float32))


def test_scan_infinities_and_nan_stay_in_their_channel_and_batch_entry():
    case = (3, 600, 64, "sigmoid", "plain", "bf16", True, False, False)
    d = _scan_inputs(case)
    clean = _run_scan(case, d)
    d["x"][1, 300, 5], d["x"][1, 100, 9], d["h0"][2, 7] = math.inf, math.nan, math.nan
    got = _run_scan(case, d)
    same = torch.ones(3, 64, dtype=torch.bool)
    same[1, 5] = same[1, 9] = same[2, 7] = False
    for k in ("h", "dx"):
        assert torch.equal(got[k].cpu().transpose(1, 2)[same], clean[k].cpu().transpose(1, 2)[same]), k
    h = got["h"].cpu()
    assert torch.isinf(h[1, 300, 5]) and torch.isnan(h[1, 100:, 9]).all() and torch.isfinite(h[1, :100, 9]).all()
    assert torch.equal(h[1, :300, 5], clean["h"].cpu()[1, :300, 5])


@pytest.mark.parametrize("L", [1, 16, 130, 600])
@pytest.mark.parametrize("inp", ["plain", "complement"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_sigmoid_gates_that_are_shut_or_open(dtype, inp, L):
    """Gates about the borders of the exponential's range: e^-g is infinite from -88.7 on, 1 / (1 + e^-g)
    below the normal range from -87.3 on (subnormal results are zero: 2^-126 off), e^-g so from 87.3 on."""
    edges = (-math.inf, -200.0, -104.0, -89.0, -88.5, -88.0, -87.5, -87.0, -86.5, -42.0, -41.5, -30.0, 0.0, 15.0, 30.0,
             87.0, 88.0, 89.0, 104.0, math.inf)
    case = (2, L, len(edges) + 1, "sigmoid", inp, dtype, True, False, False)
    d = _scan_inputs(case, 37)
    at = torch.arange(L)
    for c, e in enumerate(edges):  # a channel for each: at one token in three, at every one in the second entry
        d["g"][0, at % 3 == c % 3, c] = e
        d["g"][1, :, c] = e
    got = _run_scan(case, d)
    g, x, dh = d["g"].double(), d["x"].double(), d["dh"].double()
    # infinite gates as finite ones that are as shut or open in 64 bits, so that no bound meets infinity times zero
    want, err = ref.scan(g.clamp(-1e4, 1e4), x, "sigmoid", inp, d["h0"].double(), None, dh, d["dh_last"].double())
    # a gate below the normal range counts as zero: 2^-126 of the state or the gradient that it scales
    flush = 2.0 ** -126 * 8 * (1 + max(float(want[k].abs().max()) for k in want) ** 2)
    # bf16 takes 2^y with y = -g log2 e rounded to 32 bits: y is off by |y| 2^-24, so e^-g by |g| log2(e) 2^-24 ln 2
    # = |g| half steps, relative.  Every error that the reference counts has the gate's 12 half steps as its unit, of
    # which this makes 12 + |g| (past 104, e^-|g| is below all of fp32)
    more = torch.ones(len(edges) + 1, dtype=torch.float64)
    if dtype == "bf16":
        more[:-1] += torch.tensor([min(abs(e), 104.0) for e in edges]).double() * ref.E32 / ref.STEP
    for k, v in want.items():
        t = torch.float32 if k in ("h_last", "dh0") else DT[dtype]
        ref.check(k, got[k], v, ref.rounded(v, err[k] * more, t) + flush)


@pytest.mark.parametrize("L", [9, 300])
@pytest.mark.parametrize("gate", ["value", "sigmoid", "exp"])
@pytest.mark.parametrize("inp", ["plain", "complement"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_nan_gates_give_nan_where_the_formula_does(dtype, inp, gate, L):
    """A NaN gate at one token: that token's and later states, the gradients of that token's gate and input
    (with the complement) and of earlier ones."""
    case = (2, L, 6, gate, inp, dtype, True, False, False)
    d = _scan_inputs(case, 41)
    t = L // 2
    d["g"][1, t, 3] = math.nan
    got = {k: torch.isnan(v.cpu()) for k, v in _run_scan(case, d).items()}
    at = torch.arange(L)
    want = {k: torch.zeros_like(v) for k, v in got.items()}
    want["h"][1, t:, 3] = want["h_last"][1, 3] = want["dh0"][1, 3] = True
    want["dx"][1, :, 3] = (at <= t) if inp == "complement" else (at < t)
    want["dg"][1, :, 3] = True  # lam before the token, h behind it, the slope at it (value: h_{t-1} lam there)
    if gate == "value":
        want["dg"][1, t, 3] = False
    for k in want:
        assert torch.equal(got[k], want[k]), (k, torch.nonzero(got[k] != want[k])[:4].tolist())


def test_scan_gradients_against_differences():
    """h is linear in x and in h0, and a polynomial in value gates: central differences of the fp32 kernel's
    <dh, h> + <dh_last, h_last> against its gradients, and the same step in 64 bits for the gates."""
    case = (2, 300, 24, "value", "complement", "f32", True, False, False)
    d = _scan_inputs(case)
    got = {k: v.double().cpu() for k, v in _run_scan(case, d).items()}
    op = _ops().GatedScan(dict(D=24, gate="value", inp="complement", dtype="f32"))

    def loss(g, x, h0):
        h, last = op.forward(g.cuda(), x.cuda(), h0=h0.cuda())
        return (h.double().cpu() * d["dh"].double()).sum() + (last.double().cpu() * d["dh_last"].double()).sum()

    def loss64(g, x, h0):
        o, _ = ref.scan(g.double(), x.double(), "value", "complement", h0.double())
        return (o["h"] * d["dh"].double()).sum() + (o["h_last"] * d["dh_last"].double()).sum()

    _, err = ref.scan(d["g"].double(), d["x"].double(), "value", "complement", d["h0"].double(), None,
                      d["dh"].double(), d["dh_last"].double())
    noise = float((err["h"] * d["dh"].double().abs()).sum() + (err["h_last"] * d["dh_last"].double().abs()).sum())
    gen = _gen(9)
    for name, key, step in (("g", "dg", 2.0 ** -10), ("x", "dx", 0.5), ("h0", "dh0", 0.5)):
        v = _randn(gen, *d[name].shape)
        hi, lo = (dict(g=d["g"], x=d["x"], h0=d["h0"]) for _ in range(2))
        hi[name], lo[name] = d[name] + step * v, d[name] - step * v
        exact = (hi[name].double() - lo[name].double()) / (2 * step)  # the step that was taken
        diff = (loss(**hi) - loss(**lo)) / (2 * step)
        grad = (got[key] * exact).sum()
        # each loss is off by `noise` (up to twice that where inputs grew by the step), the gradient by its bound;
        # what the gates' difference keeps of its third order is the same in 64 bits
        third = abs((loss64(**hi) - loss64(**lo)) / (2 * step) - _dot64(d, key, exact)) if name == "g" else 0.0
        bound = 2 * 2 * noise / (2 * step) + float((err[key] * exact.abs()).sum()) + float(third) + \
            float((got[key].abs() * exact.abs()).sum()) * ref.E32
        assert abs(diff - grad) <= bound, (name, diff, grad, bound)


def _dot64(d, key, v):
    o, _ = ref.scan(d["g"].double(), d["x"].double(), "value", "complement", d["h0"].double(), None, d["dh"].double(),
                    d["dh_last"].double())
    return (o[key] * v).sum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,wide", [(70, 144), (72, 144), (33, 64), (1, 8), (9, 9), (131, 131), (193, 195), (127, 256)])
def test_scan_rows_of_any_width_and_stride(dtype, D, wide):
    """Channels that are no whole number of a tile's columns, in rows that start on 16 bytes, on 4 or on 2."""
    case = (2, 600, D, "exp", "complement", dtype, True, True, False)
    d = _scan_inputs(case)
    for at in (0, wide - D):
        strided = {}
        for k in ("g", "x", "dh"):
            rows = torch.full((2, 600, wide), math.nan, dtype=DT[dtype], device="cuda")
            strided[k] = rows[..., at:at + D]
            strided[k].copy_(d[k])
        op = _ops().GatedScan(dict(D=D, gate="exp", inp="complement", dtype=dtype))
        saved, n = op.new_saved(2, 600), d["lengths"].cuda()
        out = [torch.full((2, 600, wide), 7.0, dtype=DT[dtype], device="cuda") for _ in range(3)]
        h, dg, dx = (t[..., at:at + D] for t in out)
        _, last = op.forward(strided["g"], strided["x"], h0=d["h0"].cuda(), lengths=n, saved=saved, out=h)
        _, _, dh0 = op.backward(strided["dh"], strided["g"], strided["x"], saved, dh_last=d["dh_last"].cuda(), lengths=n,
                                dg=dg, dx=dx)
        op.check_status()
        beside = torch.ones(wide, dtype=torch.bool)
        beside[at:at + D] = False
        assert all((t.cpu()[..., beside] == 7.0).all() for t in out)
        behind = torch.arange(600)[None, :] >= d["lengths"][:, None]
        for t in (h, dg, dx):
            assert (t.cpu()[behind] == 7.0).all()
            t[behind.cuda()] = 0.0
        _check_scan(case, d, dict(h=h, h_last=last, dg=dg, dx=dx, dh0=dh0))


def test_scans_on_two_streams_at_once_and_a_broadcast_input():
    """Long chains of tiles on two streams side by side, the gates broadcast over the batch (stride 0)."""
    op = _ops().GatedScan(dict(D=96, gate="sigmoid", inp="plain", dtype="bf16"))
    gen = _gen(8)
    g = (_randn(gen, 1, 20000, 96) + 3).bfloat16().cuda().expand(3, -1, -1)
    x = _randn(gen, 3, 20000, 96).bfloat16().cuda()
    want = op.forward(g.contiguous(), x)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[op.forward(g, x, stream=s) for _ in range(6)] for s in streams]
    op.check_status()
    for h, last in (r for rs in got for r in rs):
        assert torch.equal(h, want[0]) and torch.equal(last, want[1])


@pytest.mark.parametrize("dtype,L", [("bf16", 900), ("f32", 900), ("bf16", 3), ("bf16", 1)])
def test_scan_with_one_decay_for_all_tokens(dtype, L):
    """A gate per channel, broadcast over batch and tokens (strides 0): values and gradients of every token.  The
    decay's own gradient is their sum, for the caller to take: dg has no place in the decay's row."""
    from weight_sequence_mixing_b200.binding import TTTError
    case = (3, L, 72, "sigmoid", "complement", dtype, True, L > 3, False)
    d = _scan_inputs(case)
    decay = d["g"][0, 0].clone()
    d["g"] = decay.expand(3, L, 72).contiguous()
    op = _ops().GatedScan(dict(D=72, gate="sigmoid", inp="complement", dtype=dtype))
    g, x, dh = decay.cuda().expand(3, L, 72), d["x"].cuda(), d["dh"].cuda()
    saved, n = op.new_saved(3, L), None if d["lengths"] is None else d["lengths"].cuda()

    def run():
        h, last = op.forward(g, x, h0=d["h0"].cuda(), lengths=n, saved=saved)
        dg, dx, dh0 = op.backward(dh, g, x, saved, dh_last=d["dh_last"].cuda(), lengths=n)
        op.check_status()
        return dict(h=h, h_last=last, dg=dg, dx=dx, dh0=dh0)
    got, again = run(), run()
    _check_scan(case, d, got)
    assert all(torch.equal(got[k], again[k]) for k in got)
    with pytest.raises(TTTError):
        op.backward(dh, g, x, saved, dg=torch.zeros(72, dtype=g.dtype, device="cuda").expand(3, L, 72))


def test_many_short_sequences():
    """More batch entries than a grid has rows: one new token and a few of each."""
    B, D = 70001, 6
    gen = _gen(12)
    x = _randn(gen, B, 3, D).bfloat16()
    op = _ops().GatedScan(dict(D=D, gate="value", inp="plain", dtype="bf16"))
    g = torch.full_like(x, 0.5).cuda()
    n = torch.arange(B, dtype=torch.int32) % 4
    h, last = op.forward(g, x.cuda(), lengths=n.cuda())
    want = torch.zeros(B, D)
    for t in range(3):
        want = torch.where((t < n)[:, None], 0.5 * want + x[:, t].float(), want)
    assert torch.equal(last.cpu(), want)
    assert (h.cpu()[torch.arange(3)[None] >= n[:, None]] == 0).all()
    rope = _ops().RotaryPositions(dict(d=6, pairs=(3,), dtype="bf16"))
    pos = torch.arange(3 * B, dtype=torch.int32).view(B, 3, 1)
    y = rope.forward(x.view(B, 1, 3, D).cuda(), pos.cuda())
    want, err = ref.rope(x.view(B, 1, 3, D).double(), pos, (3,), 10000.0, "halves")
    ref.check("y", y, want, ref.rounded(want, err, torch.bfloat16))


def test_scan_longer_than_32_bit_offsets():
    """A scan whose tensors hold more than 2^31 elements: its last rows."""
    L, D = (1 << 19) + 77, 4104
    op = _ops().GatedScan(dict(D=D, gate="value", inp="plain", dtype="bf16"))
    g = torch.zeros((1, L, D), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((1, L, D), dtype=torch.bfloat16, device="cuda")
    g[:, -3:], g[:, -600:-500] = 0.5, 1.0
    h, last = op.forward(g, x)
    op.check_status()
    assert torch.equal(h[0, -3:, 0].float().cpu(), torch.tensor([1.5, 1.75, 1.875]))
    assert (h[0, -3:] == h[0, -3:, :1]).all() and (last == 1.875).all()
    assert (h[0, -501] == 101.0).all() and (h[0, -700:-600] == 1.0).all()


def test_scan_clear_of_as_many_sequences_as_there_can_be():
    """2^31 - 1 sequences of one token and channel, one in a million of them with a token of its own."""
    from weight_sequence_mixing_b200.binding import LIB
    import ctypes
    B = 2 ** 31 - 1
    op = _ops().GatedScan(dict(D=1, gate="value", inp="plain", dtype="bf16"))
    y = torch.ones(B, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    n[::1_000_003] = 1
    n[-1] = 1
    status = LIB.ttt_scan_clear(op._handle, B, 1, n.data_ptr(), y.data_ptr(), (ctypes.c_int64 * 3)(1, 0, 1),
                                torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()
    assert (y[::1_000_003] == 1).all() and y[-1] == 1
    assert sum(int(torch.count_nonzero(part)) for part in y.split(1 << 28)) == len(range(0, B, 1_000_003)) + 1


@pytest.mark.parametrize("dtype,D,wide", [("bf16", 128, 128), ("bf16", 128, 130), ("bf16", 65, 65), ("f32", 33, 33)],
                         ids=["tma", "copies_of_4", "odd_rows", "fp32_copies"])
def test_scan_wait_that_runs_out_sets_the_status_and_ends(dtype, D, wide):
    """The first tile is left out: what waits for its state gives up, in every form of the loads, and the
    next call on the same buffers is right."""
    import ctypes
    from weight_sequence_mixing_b200.binding import LIB, TTT_ERR_TIMEOUT, TTTError
    case = (3, 9 * 256 + 40, D, "sigmoid", "complement", dtype, False, False, False)
    d = _scan_inputs(case)
    B, L = case[:2]
    rows = [torch.zeros((B, L, wide), dtype=DT[dtype], device="cuda") for _ in range(3)]
    g, x, h = (t[..., :D] for t in rows)
    g.copy_(d["g"]), x.copy_(d["x"])
    op = _ops().GatedScan(dict(D=D, gate="sigmoid", inp="complement", dtype=dtype))
    need = LIB.ttt_scan_workspace_size(op._handle, B, L)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s = (ctypes.c_int64 * 3)(L * wide, 0, wide)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    st = LIB.ttt_selftest_scan_timeout(op._handle, B, L, g.data_ptr(), s, x.data_ptr(), s, h.data_ptr(), s, ws.data_ptr(),
                                       need, op._status.data_ptr(), 20, torch.cuda.current_stream().cuda_stream)
    end.record()
    assert st == 0
    with pytest.raises(TTTError) as e:
        op.check_status()
    assert e.value.status == TTT_ERR_TIMEOUT
    assert 20 <= begin.elapsed_time(end) < 2000
    op.check_status()  # told once
    got, last = op.forward(g, x, out=h)
    op.check_status()
    want, err = ref.scan(d["g"].double(), d["x"].double(), "sigmoid", "complement")
    ref.check("h", got, want["h"], ref.rounded(want["h"], err["h"], DT[dtype]))
    ref.check("h_last", last, want["h_last"], ref.rounded(want["h_last"], err["h_last"], torch.float32))


# ------------------------------------------------------------------------- norm
# B, N, C, G, act, dtype, layout ("tokens": [B,N,C]; "heads": [B,G,N,C/G]; "slice"; "odd")
NORM = [
    (1, 1, 8, 2, "none", "f32", "tokens"),
    (1, 1, 64, 64, "silu", "bf16", "tokens"),
    (2, 2, 6, 6, "gelu", "f32", "tokens"),
    (1, 196, 64, 8, "silu", "bf16", "tokens"),
    (3, 100, 96, 32, "gelu", "f32", "tokens"),
    (2, 77, 384, 6, "silu", "bf16", "heads"),
    (2, 300, 128, 32, "silu", "bf16", "tokens"),
    (2, 513, 30, 2, "gelu", "bf16", "tokens"),
    (2, 129, 35, 5, "silu", "f32", "heads"),
    (2, 200, 64, 4, "silu", "bf16", "slice"),
    (2, 200, 64, 4, "none", "f32", "odd"),
    (1, 2100, 256, 1, "silu", "bf16", "tokens"),
    (1, 40, 2048, 16, "silu", "f32", "tokens"),
    (9, 33, 24, 3, "gelu", "bf16", "heads"),
    (1, 5, 1032, 8, "none", "bf16", "tokens"),
    # groups too large for one block: vectors of one group, of two, of several, groups over two blocks of
    # channels, more channels than a block has, rows of a block that stay empty, narrow vectors
    (2, 4100, 96, 6, "silu", "bf16", "tokens"),
    (1, 8200, 128, 32, "silu", "bf16", "tokens"),
    (1, 9001, 96, 32, "gelu", "f32", "tokens"),
    (1, 7000, 96, 32, "none", "bf16", "tokens"),
    (1, 400, 4128, 3, "silu", "bf16", "tokens"),
    (1, 300, 4100, 2, "gelu", "f32", "tokens"),
    (2, 1100, 384, 3, "silu", "bf16", "heads"),
    (3, 2050, 90, 5, "silu", "bf16", "tokens"),
    (2, 3333, 35, 1, "none", "bf16", "heads"),
    (1, 2500, 132, 2, "silu", "f32", "slice"),
    (2, 3000, 40, 2, "gelu", "bf16", "odd"),
]


def _norm_inputs(case, seed=5):
    B, N, C, G, act, dtype, layout = case
    gen = _gen(seed)
    x = (_randn(gen, B, N, C) * 1.5 + 0.5).to(DT[dtype])
    w, b, dy = 1 + 0.2 * _randn(gen, C), 0.2 * _randn(gen, C), _randn(gen, B, N, C).to(DT[dtype])
    if layout == "heads":
        xd = x.view(B, N, G, C // G).transpose(1, 2).contiguous().cuda()
    elif layout == "slice":
        wide = torch.full((B, N, 3 * C), math.nan, dtype=DT[dtype], device="cuda")
        xd = wide[..., C:2 * C]
        xd.copy_(x)
    elif layout == "odd":
        xd = torch.empty(B * N * C + 1, dtype=DT[dtype], device="cuda")[1:].view(B, N, C)
        xd.copy_(x)
    else:
        xd = x.cuda()
    return x, xd, w, b, dy


def _tokens(t, B, N, C):
    return t.transpose(1, 2).reshape(B, N, C) if t.dim() == 4 else t


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)))
def test_norm(case, weights):
    B, N, C, G, act, dtype, layout = case
    x, xd, w, b, dy = _norm_inputs(case)
    if not weights:
        w = b = None
    op = _ops().GroupNorm(dict(C=C, groups=G, act=act, eps=1e-5, dtype=dtype))
    wd, bd, dyd = (None if t is None else t.cuda() for t in (w, b, dy))
    stats = op.new_stats(B)
    y = op.forward(xd, wd, bd, stats=stats)
    dx, dw, db = op.backward(dyd, xd, wd, bd, stats)
    op.check_status()
    d64 = lambda t: None if t is None else t.double()  # noqa: E731
    want, err = ref.norm(x.double(), G, d64(w), d64(b), act, float(torch.tensor(1e-5)), dy.double())
    got = dict(y=y, mean=stats[..., 0], rstd=stats[..., 1], dx=_tokens(dx, B, N, C), dweight=dw, dbias=db)
    assert dx.shape == xd.shape and y.shape == (B, N, C)
    for k, v in got.items():
        ref.check(k, v, want[k], ref.rounded(want[k], err[k], DT[dtype] if k in ("y", "dx") else torch.float32))
    again = op.backward(dyd, xd, wd, bd, stats)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    assert torch.equal(op.forward(xd, wd, bd), y)
    # in the input's place
    if layout != "heads":
        inplace = dyd.clone()
        op.backward(inplace, xd, wd, bd, stats, dx=inplace)
        assert torch.equal(inplace, dx)
        op.forward(xd, wd, bd, out=xd)
        assert torch.equal(xd, y)


@pytest.mark.parametrize("dtype,offset", [("f32", 1000.0), ("f32", -3.0e4), ("bf16", 256.0)])
def test_norm_of_a_group_far_from_zero(dtype, offset):
    """The variance of values whose mean is many times their spread, the first value of all an outlier."""
    B, N, C, G = 2, 640, 48, 3
    x = (_randn(_gen(2), B, N, C) + offset).to(DT[dtype])
    x[:, 0, 0] = -offset
    op = _ops().GroupNorm(dict(C=C, groups=G, act="none", eps=1e-5, dtype=dtype))
    stats = op.new_stats(B)
    y = op.forward(x.cuda(), stats=stats)
    want, err = ref.norm(x.double(), G, None, None, "none", float(torch.tensor(1e-5)))
    # the variance is as exact as sums of squares about a nearby mean can be: far from what E[x^2] - mean^2 gives
    for k, v in dict(y=y, mean=stats[..., 0], rstd=stats[..., 1]).items():
        ref.check(k, v, want[k], ref.rounded(want[k], err[k], DT[dtype] if k == "y" else torch.float32))


@pytest.mark.parametrize("case", [(2, 100, 96, 32, "gelu", "f32", "tokens"), (2, 4100, 96, 6, "silu", "bf16", "tokens")],
                         ids=["one_block_a_group", "two_kernels"])
def test_norm_small_tensors_at_any_place_of_a_buffer(case):
    """Statistics, weights and their gradients one fp32 value past the alignment of a buffer."""
    B, N, C, G, act, dtype, layout = case
    x, xd, w, b, dy = _norm_inputs(case)
    op = _ops().GroupNorm(dict(C=C, groups=G, act=act, dtype=dtype))
    odd = lambda *shape: torch.empty(1 + math.prod(shape), device="cuda")[1:].view(shape)  # noqa: E731
    stats = op.new_stats(B)
    want = [op.forward(xd, w.cuda(), b.cuda(), stats=stats), *op.backward(dy.cuda(), xd, w.cuda(), b.cuda(), stats)]
    wd, bd, st, dw, db = odd(C).copy_(w), odd(C).copy_(b), odd(B, G, 2), odd(C), odd(C)
    assert all(t.data_ptr() % 8 == 4 for t in (wd, bd, st, dw, db))
    got = [op.forward(xd, wd, bd, stats=st), *op.backward(dy.cuda(), xd, wd, bd, st, dweight=dw, dbias=db)]
    assert torch.equal(st, stats) and all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,N", [(64, 20), (1, 40)], ids=["one_block_a_group", "two_kernels"])
def test_norm_gelu_keeps_its_digits_in_the_tail(dtype, G, N):
    """With a weight of zero z is the bias itself: z Phi(z) and, through dbias of a single dy, its slope, from
    -13 (where they are next to the least normal number) on, relative to the values."""
    C = 1024
    z = torch.linspace(-13.0, 9.0, C)
    op = _ops().GroupNorm(dict(C=C, groups=G, act="gelu", dtype=dtype))
    x = _randn(_gen(8), 1, N, C).to(DT[dtype]).cuda()
    w, b, stats = torch.zeros(C, device="cuda"), z.cuda(), op.new_stats(1)
    y = op.forward(x, w, b, stats=stats)
    dy = torch.zeros((1, N, C), dtype=DT[dtype], device="cuda")
    dy[0, N // 2] = 1.0
    _, _, slope = op.backward(dy, x, w, b, stats)
    z = z.double()
    cdf, pdf = 0.5 * torch.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # the exponent z^2 log2(e) / 2 <= 122 is rounded twice, its constant once: 1.5 2^-23 of it at most, times ln 2
    # 1.5e-5 in its exponential (erfc's argument, squared, is the same); the exponential itself, a reciprocal and the
    # polynomial 1.2e-6 more: in all below 2^-15
    off = 2.0 ** -15
    want = (z * cdf).expand(1, N, C)
    ref.check("y", y, want, ref.rounded(want, off * want.abs(), DT[dtype]))
    want = cdf + z * pdf
    ref.check("slope", slope, want, ref.rounded(want, off * (cdf + z.abs() * pdf), torch.float32))


def test_norm_nan_stays_in_its_group_and_batch_entry():
    case = (3, 150, 64, 4, "silu", "bf16", "tokens")
    x, xd, w, b, dy = _norm_inputs(case)
    op = _ops().GroupNorm(dict(C=64, groups=4, act="silu", dtype="bf16"))
    clean = op.forward(xd, w.cuda(), b.cuda())
    xd[1, 70, 20] = math.nan
    y = op.forward(xd, w.cuda(), b.cuda())
    hit = torch.zeros(3, 150, 64, dtype=torch.bool)
    hit[1, :, 16:32] = True
    assert torch.equal(y.cpu()[~hit], clean.cpu()[~hit]) and torch.isnan(y.cpu()[hit]).all()


def test_norm_of_equal_values_is_the_bias():
    op = _ops().GroupNorm(dict(C=64, groups=4, act="none", eps=1e-5, dtype="bf16"))
    x = torch.full((2, 300, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    b = torch.randn(64, device="cuda").bfloat16().float()
    y = op.forward(x, None, b)
    assert torch.equal(y.float(), b.expand(2, 300, 64))


def test_norm_gradients_against_differences():
    case = (2, 60, 24, 4, "gelu", "f32", "tokens")
    x, xd, w, b, dy = _norm_inputs(case)
    op = _ops().GroupNorm(dict(C=24, groups=4, act="gelu", dtype="f32"))
    stats = op.new_stats(2)
    op.forward(xd, w.cuda(), b.cuda(), stats=stats)
    grads = dict(zip(("x", "w", "b"), (t.double().cpu() for t in op.backward(dy.cuda(), xd, w.cuda(), b.cuda(), stats))))
    loss = lambda x, w, b: (op.forward(x.cuda(), w.cuda(), b.cuda()).double().cpu() * dy.double()).sum()  # noqa: E731
    eps = float(torch.tensor(1e-5))
    loss64 = lambda x, w, b: (ref.norm(x.double(), 4, w.double(), b.double(), "gelu", eps)[0]["y"] *  # noqa: E731
                              dy.double()).sum()
    want, err = ref.norm(x.double(), 4, w.double(), b.double(), "gelu", eps, dy.double())
    noise = float((ref.rounded(want["y"], err["y"], torch.float32) * dy.double().abs()).sum())
    gen = _gen(4)
    for name, key in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        v = _randn(gen, *dict(x=x, w=w, b=b)[name].shape)
        step = 2.0 ** -7
        hi, lo = dict(x=x, w=w, b=b), dict(x=x, w=w, b=b)
        hi[name], lo[name] = hi[name] + step * v, lo[name] - step * v
        exact = (hi[name].double() - lo[name].double()) / (2 * step)
        diff = (loss(**hi) - loss(**lo)) / (2 * step)
        third = abs((loss64(**hi) - loss64(**lo)) / (2 * step) - (want[key] * exact).sum())
        bound = 2 * 2 * noise / (2 * step) + float((ref.rounded(want[key], err[key], torch.float32) * exact.abs()).sum()) + \
            float(third)
        assert abs(diff - (grads[name] * exact).sum()) <= bound, name


# ---------------------------------------------------------- streams, graphs, refusals
def _three_ops():
    """(call, reset) of each operator's forward and backward on the same inputs."""
    ops = _ops()
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    pos = torch.arange(700, dtype=torch.int32, device="cuda")[:, None].contiguous()
    rope = ops.RotaryPositions(dict(d=64, pairs=(32,), dtype="bf16"))
    scan = ops.GatedScan(dict(D=128, gate="sigmoid", inp="complement", dtype="bf16"))
    norm = ops.GroupNorm(dict(C=128, groups=2, act="silu", dtype="bf16"))
    q, g, x, dh = r(2, 2, 700, 64), r(2, 700, 128), r(2, 700, 128), r(2, 700, 128)
    w, b = torch.rand(128, device="cuda"), torch.rand(128, device="cuda")

    def step(stream=None):
        y = rope.forward(q, pos, stream=stream)
        z = rope.backward(y, pos, stream=stream)
        saved, stats = scan.new_saved(2, 700, stream=stream), norm.new_stats(2, stream=stream)
        o = norm.forward(z, w, b, stats=stats, stream=stream)
        h, last = scan.forward(g, o, saved=saved, stream=stream)
        dg, dx, dh0 = scan.backward(dh, g, o, saved, stream=stream)
        dz, dw, db = norm.backward(dx, z, w, b, stats, stream=stream)
        return [y, z, o, h, last, dg, dx, dh0, dz, dw, db]

    return step, (scan, norm), (q, g, x, dh)


def test_ops_on_another_stream_and_in_two_graphs_that_replay_at_once():
    step, status, inputs = _three_ops()
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for rep in range(3):
        for o in outs:
            for t in o:
                t.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o)), rep
    # a graph reads its inputs anew
    inputs[0].mul_(0.5)
    want = [t.clone() for t in step()]
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs[0]))
    for op in status:
        op.check_status()


def test_refusals_of_the_binding():
    from weight_sequence_mixing_b200.binding import TTTError
    ops = _ops()
    rope = ops.RotaryPositions(dict(d=64, pairs=(16, 16), dtype="bf16"))
    x = torch.zeros((2, 3, 5, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[..., :32]), dict(x=x[0]), dict(x=x.cpu()), dict(pos=pos.long()),
                dict(pos=pos[:4]), dict(pos=pos.cpu()), dict(pos=torch.zeros((5, 4), dtype=torch.int32, device="cuda")[:, ::2]),
                dict(x=torch.zeros((2, 3, 64, 5), dtype=torch.bfloat16, device="cuda").transpose(2, 3)),
                dict(out=x[:, :, :4]), dict(out=x.float())):
        with pytest.raises(ValueError):
            rope.forward(**dict(dict(x=x, pos=pos), **bad))
    with pytest.raises(TTTError):  # batch entries and heads of the output in one place
        rope.forward(x, pos, out=torch.zeros_like(x).as_strided((2, 3, 5, 64), (0, 0, 64, 1)))
    with pytest.raises(ValueError):
        ops.RotaryPositions(dict(d=64, pairs=(), dtype="bf16"))
    with pytest.raises(ValueError):
        ops.RotaryPositions(dict(d=64, pairs=(16, 16), base=(2.0,), dtype="bf16"))
    with pytest.raises(ValueError):
        ops.RotaryPositions(dict(d=64, pairs=(16, 16), dtype="bf16"), device="cpu")
    scan = ops.GatedScan(dict(D=32, gate="value", inp="plain", dtype="f32"))
    g = torch.zeros((2, 9, 32), device="cuda")
    st, n = torch.zeros((2, 32), device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    saved = scan.new_saved(2, 9)
    for bad in (dict(g=g[:, :8]), dict(g=g.bfloat16()), dict(x=g[..., :16]), dict(h0=st[:1]), dict(h0=st.double()),
                dict(lengths=n.long()), dict(lengths=n[:1]), dict(saved=saved[:-300] if saved.numel() > 300 else saved[:8]),
                dict(h_last=st.cpu()), dict(out=g.cpu())):
        with pytest.raises(ValueError):
            scan.forward(**dict(dict(g=g, x=g), **bad))
    with pytest.raises(TTTError):
        scan.forward(g, g, out=g)
    with pytest.raises(ValueError):
        scan.backward(g, g, g, saved[:8])
    norm = ops.GroupNorm(dict(C=32, groups=4, dtype="f32"))
    w = torch.ones(32, device="cuda")
    for bad in (dict(x=g.bfloat16()), dict(x=g[:, :0]), dict(x=g[..., :16]), dict(weight=w[:16]), dict(bias=w.double()),
                dict(stats=torch.zeros((2, 3, 2), device="cuda")), dict(x=torch.zeros((2, 3, 9, 8), device="cuda")),
                dict(out=torch.zeros((2, 4, 9, 8), device="cuda"))):
        with pytest.raises(ValueError):
            norm.forward(**dict(dict(x=g), **bad))
    scan.close()
    with pytest.raises(ValueError):
        scan.forward(g, g)
    with pytest.raises(TTTError):
        ops.GroupNorm(dict(C=32, groups=5, dtype="f32"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_column_ranges_of_a_fused_buffer_are_read_and_written(dtype):
    """Several heads or groups: positions from one third of a fused projection into another, the norm from
    one half of a buffer into the other, and their gradients the same way; what lies beside stays as it was."""
    ops, gen, dt = _ops(), _gen(31), DT[dtype]
    B, N, H, d = 2, 45, 3, 16
    fused = torch.full((B, N, 3, H, d), 7.0, dtype=dt, device="cuda")
    x = _randn(gen, B, H, N, d).to(dt)
    fused[:, :, 0] = x.transpose(1, 2).cuda()
    src, to = fused[:, :, 0].transpose(1, 2), fused[:, :, 2].transpose(1, 2)
    pos = torch.arange(N, dtype=torch.int32)[:, None].contiguous()
    rope = ops.RotaryPositions(dict(d=d, pairs=(6,), dtype=dtype))
    for call in (rope.forward, rope.backward):
        want = call(x.cuda(), pos.cuda())
        assert call(src, pos.cuda(), out=to) is to and torch.equal(to, want)
    assert torch.equal(src.cpu(), x) and (fused[:, :, 1] == 7.0).all()
    C, G = 48, 4
    norm = ops.GroupNorm(dict(C=C, groups=G, act="silu", dtype=dtype))
    for rows in (N, 4000):  # one block a group, and two kernels
        wide = torch.full((B, rows, 3 * C), 7.0, dtype=dt, device="cuda")
        x, dy = (_randn(gen, B, rows, C).to(dt).cuda() for _ in range(2))
        w, b = (_randn(gen, C).cuda() for _ in range(2))
        wide[..., :C] = x
        stats, again = norm.new_stats(B), norm.new_stats(B)
        want = norm.forward(x, w, b, stats=stats)
        assert torch.equal(norm.forward(wide[..., :C], w, b, stats=again, out=wide[..., 2 * C:]), want)
        grads = norm.backward(dy, x, w, b, stats)
        got = norm.backward(dy, wide[..., :C], w, b, again, dx=wide[..., 2 * C:])
        assert all(torch.equal(p, q) for p, q in zip(grads, got))
        assert torch.equal(wide[..., :C], x) and (wide[..., C:2 * C] == 7.0).all()
        with pytest.raises(Exception, match="ttt_norm_forward"):  # one channel of the input
            norm.forward(wide[..., :C], w, b, out=wide[..., C - 1:2 * C - 1])


# --------------------------------------------------------------- the block together
def test_positions_layer_norm_and_recurrence_as_one_block():
    """A token-mixing block as a model runs it: projections tokens first, rotary positions onto the layer's
    heads-first Q and K, the TTT layer, group norm (one group a head) with SiLU back to tokens first, the gated
    recurrence; against the fp64 oracle of the layer and the operators in 64 bits."""
    import oracle
    from synth_inputs import gen_inputs, make_config
    from weight_sequence_mixing_b200 import binding
    ops = _ops()
    B, H, N, d = 2, 3, 24 * 17, 64
    cfg = make_config(B=B, H=H, N=N, d=d, h=128, inner="mlp2_gelu", loss="mse", key_instnorm=True, dtype="bf16", data="vit",
                      seed=77)
    s = gen_inputs(cfg)
    gen = _gen(6)
    pos = torch.stack([torch.arange(N) // 17, torch.arange(N) % 17], 1).to(torch.int32)
    w, b, g = 1 + 0.2 * _randn(gen, H * d), 0.2 * _randn(gen, H * d), (_randn(gen, B, N, H * d) + 2).bfloat16()
    rope = ops.RotaryPositions(dict(d=d, pairs=(16, 16), base=100.0, dtype="bf16"))
    norm = ops.GroupNorm(dict(C=H * d, groups=H, act="silu", dtype="bf16"))
    scan = ops.GatedScan(dict(D=H * d, gate="sigmoid", inp="complement", dtype="bf16"))
    layer = binding.TTTLayer(cfg)
    tokens_first = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2)  # noqa: E731
    Q, K = rope.forward(tokens_first(s["Q"]), pos.cuda()), rope.forward(tokens_first(s["K"]), pos.cuda())
    O, W = layer.forward(Q, K, s["V"].cuda(), None, s["W0"].cuda())
    y = norm.forward(O, w.cuda(), b.cuda())
    h, last = scan.forward(g.cuda(), y)
    scan.check_status()
    layer.close()
    Q64, _ = ref.rope(s["Q"].double(), pos, (16, 16), 100.0, "halves")
    K64, _ = ref.rope(s["K"].double(), pos, (16, 16), 100.0, "halves")
    O64, _ = oracle.forward(cfg, Q64.bfloat16(), K64.bfloat16(), s["V"], None, s["W0"])
    O64 = torch.from_numpy(O64)
    y64 = ref.norm(O64.transpose(1, 2).reshape(B, N, H * d), H, w.double(), b.double(), "silu", 1e-5)[0]["y"]
    h64 = ref.scan(g.double(), y64, "sigmoid", "complement")[0]["h"]
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    # the layer's own bound (2e-2 relative), which the norm keeps relative to its unit variance (SiLU's slope is
    # at most 1.1); the recurrence averages errors and signal over the same tokens, which leaves their ratio
    # within a factor of two; bf16 roundings of Q, K, y and h add 2^-8 each
    assert rel(O, O64) <= 2e-2 + 2 * 2.0 ** -8
    assert rel(y, y64) <= 1.2 * 2e-2 + 3 * 2.0 ** -8 and rel(h, h64) <= 2 * (2e-2 + 4 * 2.0 ** -8)
