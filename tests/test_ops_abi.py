"""Configurations and calls of the operators in ttt_ops.h that are refused, on the host,
before anything is enqueued (no GPU: the pointers are made up)."""
import ctypes

import pytest

P = 1 << 20  # a made-up device address


def _lib():
    from weight_sequence_mixing_b200 import binding, token_ops
    return binding, token_ops


def _open(name, cfg):
    binding, _ = _lib()
    h = ctypes.c_void_p()
    st = getattr(binding.LIB, f"ttt_{name}_create")(ctypes.byref(cfg), ctypes.byref(h))
    return st, h


def _rope_cfg(d=64, pairs=(16, 16), base=(100.0, 100.0), pairing=0, dtype=1, axes=None):
    _, ops = _lib()
    c = ops.RopeConfig(d=d, axes=len(pairs) if axes is None else axes, pairing=pairing, dtype=dtype)
    for i, (n, b) in enumerate(zip(pairs, base)):
        c.pairs[i], c.base[i] = n, b
    return c


def _s(*v):
    return (ctypes.c_int64 * 3)(*v)


@pytest.mark.parametrize("kw", [dict(d=0), dict(d=63), dict(pairs=(16, 17)), dict(pairs=(0, 16)), dict(axes=0), dict(axes=5),
                                dict(base=(0.0, 1.0)), dict(base=(float("nan"), 1.0)), dict(base=(float("inf"), 1.0)),
                                dict(base=(-2.0, 1.0)), dict(pairing=2), dict(dtype=2), dict(pairs=(-1, 16))])
def test_rope_configurations_that_are_refused(kw):
    binding, _ = _lib()
    st, h = _open("rope", _rope_cfg(**kw))
    assert st == binding.TTT_ERR_INVALID_ARG and not h.value


def test_rope_with_more_pairs_than_a_handle_holds_is_unsupported():
    binding, _ = _lib()
    st, h = _open("rope", _rope_cfg(d=1024, pairs=(200, 57), base=(2.0, 2.0)))
    assert st == binding.TTT_ERR_UNSUPPORTED and not h.value


ROPE_OK = dict(B=2, H=3, N=5, x=P, xs=(3 * 5 * 64, 5 * 64, 64), pos=P + (1 << 16), pos_dtype=0, pos_batch=0,
               y=P + (1 << 18), ys=(3 * 5 * 64, 5 * 64, 64), inverse=0)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(H=0), dict(N=-1), dict(x=None), dict(y=None), dict(pos=None), dict(pos_dtype=2), dict(pos_batch=-1),
    dict(inverse=2), dict(x=P + 1), dict(y=P + (1 << 18) + 1), dict(pos=P + (1 << 16) + 2),
    dict(xs=(960, -320, 64)),                    # a negative stride
    dict(ys=(960, 320, 32)),                     # rows of the output overlap
    dict(ys=(0, 320, 64)),                       # batch entries of the output in one place
    dict(y=P + 64),                              # the output inside the input
    dict(y=P, ys=(960, 64, 192)),                # the input's place in another order
    dict(pos=P + (1 << 18)),                     # positions inside the output
], ids=str)
def test_rope_calls_that_are_refused(kw):
    binding, _ = _lib()
    st, h = _open("rope", _rope_cfg())
    assert st == 0
    a = dict(ROPE_OK, **kw)
    st = binding.LIB.ttt_rope_apply(h, a["B"], a["H"], a["N"], a["x"], _s(*a["xs"]), a["pos"], a["pos_dtype"],
                                    a["pos_batch"], a["y"], _s(*a["ys"]), a["inverse"], None)
    assert st == binding.TTT_ERR_INVALID_ARG
    assert binding.LIB.ttt_rope_apply(None, 2, 3, 5, P, _s(960, 320, 64), P, 0, 0, P, _s(960, 320, 64), 0,
                                      None) == binding.TTT_ERR_INVALID_ARG
    binding.LIB.ttt_rope_destroy(h)


def test_rope_of_no_tokens_does_nothing():
    binding, _ = _lib()
    st, h = _open("rope", _rope_cfg())
    assert binding.LIB.ttt_rope_apply(h, 2, 3, 0, None, _s(0, 0, 64), None, 0, 0, None, _s(0, 0, 64), 0, None) == 0
    binding.LIB.ttt_rope_destroy(h)


@pytest.mark.parametrize("kw", [dict(D=0), dict(gate=3), dict(gate=-1), dict(input=2), dict(dtype=2)])
def test_scan_configurations_that_are_refused(kw):
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(**dict(dict(D=64, gate=1, input=1, dtype=1), **kw)))
    assert st == binding.TTT_ERR_INVALID_ARG and not h.value


M = 1 << 20
FWD_OK = dict(B=2, L=700, g=64 * M, gs=(700 * 64, 0, 64), x=80 * M, xs=(700 * 64, 0, 64), h0=96 * M, lengths=97 * M,
              h=112 * M, hs=(700 * 64, 0, 64), h_last=98 * M, saved=128 * M, ws=160 * M, wsn=1 << 30, status=99 * M)


def _forward(h, a):
    binding, _ = _lib()
    return binding.LIB.ttt_scan_forward(h, a["B"], a["L"], a["g"], _s(*a["gs"]), a["x"], _s(*a["xs"]), a["h0"],
                                        a["lengths"], a["h"], _s(*a["hs"]), a["h_last"], a["saved"], a["ws"], a["wsn"],
                                        a["status"], None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(L=-1), dict(g=None), dict(x=None), dict(h=None), dict(g=64 * M + 1), dict(h=112 * M + 1),
    dict(h0=96 * M + 2), dict(lengths=97 * M + 1), dict(h_last=98 * M + 2), dict(saved=128 * M + 8), dict(ws=160 * M + 8),
    dict(status=99 * M + 2), dict(gs=(44800, 0, -64)), dict(hs=(44800, 0, 32)), dict(hs=(0, 0, 64)),
    dict(h=80 * M), dict(h=64 * M + 128), dict(h_last=112 * M), dict(h0=98 * M + 4), dict(saved=112 * M),
    dict(lengths=98 * M),
], ids=str)
def test_scan_forward_calls_that_are_refused(kw):
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(D=64, gate=1, input=1, dtype=1))
    assert st == 0
    assert _forward(h, dict(FWD_OK, **kw)) == binding.TTT_ERR_INVALID_ARG
    assert _forward(None, FWD_OK) == binding.TTT_ERR_INVALID_ARG
    assert _forward(h, dict(FWD_OK, L=(1 << 30) + 1)) == binding.TTT_ERR_UNSUPPORTED
    need = binding.LIB.ttt_scan_workspace_size(h, 2, 700)
    if need:
        assert _forward(h, dict(FWD_OK, wsn=need - 1)) == binding.TTT_ERR_WORKSPACE
        assert _forward(h, dict(FWD_OK, ws=None)) == binding.TTT_ERR_WORKSPACE
    binding.LIB.ttt_scan_destroy(h)


def test_scan_clear_calls_that_are_refused():
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(D=64, gate=1, input=1, dtype=1))
    call = lambda B=2, L=700, n=97 * M, y=112 * M, s=(44800, 0, 64): binding.LIB.ttt_scan_clear(  # noqa: E731
        h, B, L, n, y, _s(*s), None)
    for bad in (dict(B=0), dict(L=-1), dict(n=None), dict(n=97 * M + 2), dict(y=None), dict(y=112 * M + 1),
                dict(s=(44800, 0, 63)), dict(n=112 * M)):
        assert call(**bad) == binding.TTT_ERR_INVALID_ARG, bad
    assert call(L=(1 << 30) + 1) == binding.TTT_ERR_UNSUPPORTED
    binding.LIB.ttt_scan_destroy(h)


BWD_OK = dict(B=2, L=700, dh=64 * M, dh_last=98 * M, g=80 * M, x=96 * M + 4 * M, lengths=97 * M, saved=128 * M,
              dg=112 * M, dx=120 * M, dh0=99 * M, ws=160 * M, wsn=1 << 30, status=None,
              dhs=(44800, 0, 64), gs=(44800, 0, 64), xs=(44800, 0, 64), dgs=(44800, 0, 64), dxs=(44800, 0, 64))


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(L=-1), dict(dh=None), dict(g=None), dict(x=None), dict(saved=None), dict(dg=None), dict(dx=None),
    dict(dh=64 * M + 1), dict(dh_last=98 * M + 2), dict(dh0=99 * M + 2), dict(saved=128 * M + 4), dict(dgs=(44800, 0, 63)),
    dict(dxs=(64, 0, 64)), dict(dx=112 * M), dict(dx=64 * M), dict(dg=80 * M), dict(dh0=98 * M), dict(dx=128 * M),
], ids=str)
def test_scan_backward_calls_that_are_refused(kw):
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(D=64, gate=1, input=1, dtype=1))
    assert st == 0
    a = dict(BWD_OK, **kw)
    st = binding.LIB.ttt_scan_backward(h, a["B"], a["L"], a["dh"], _s(*a["dhs"]), a["dh_last"], a["g"], _s(*a["gs"]),
                                       a["x"], _s(*a["xs"]), a["lengths"], a["saved"], a["dg"], _s(*a["dgs"]), a["dx"],
                                       _s(*a["dxs"]), a["dh0"], a["ws"], a["wsn"], a["status"], None)
    assert st == binding.TTT_ERR_INVALID_ARG
    binding.LIB.ttt_scan_destroy(h)


@pytest.mark.parametrize("kw", [dict(C=0), dict(groups=0), dict(groups=5), dict(act=3), dict(act=-1), dict(eps=-1e-5),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(dtype=2)])
def test_norm_configurations_that_are_refused(kw):
    binding, ops = _lib()
    st, h = _open("norm", ops.NormConfig(**dict(dict(C=64, groups=8, act=1, eps=1e-5, dtype=1), **kw)))
    assert st == binding.TTT_ERR_INVALID_ARG and not h.value


NORM_OK = dict(B=2, N=50, x=64 * M, xs=(3200, 8, 64), weight=80 * M, bias=81 * M, y=96 * M, ys=(3200, 8, 64),
               stats=82 * M, ws=112 * M, wsn=1 << 30, status=None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(N=0), dict(x=None), dict(y=None), dict(x=64 * M + 1), dict(weight=80 * M + 2), dict(stats=82 * M + 2),
    dict(ws=112 * M + 8), dict(xs=(3200, -8, 64)), dict(ys=(3200, 7, 64)), dict(ys=(3200, 0, 64)), dict(y=64 * M + 64),
    dict(y=64 * M, ys=(3200, 400, 8)), dict(stats=80 * M), dict(stats=96 * M),
], ids=str)
def test_norm_forward_calls_that_are_refused(kw):
    binding, ops = _lib()
    st, h = _open("norm", ops.NormConfig(C=64, groups=8, act=1, eps=1e-5, dtype=1))
    assert st == 0
    a = dict(NORM_OK, **kw)
    st = binding.LIB.ttt_norm_forward(h, a["B"], a["N"], a["x"], _s(*a["xs"]), a["weight"], a["bias"], a["y"],
                                      _s(*a["ys"]), a["stats"], a["ws"], a["wsn"], a["status"], None)
    assert st == binding.TTT_ERR_INVALID_ARG
    binding.LIB.ttt_norm_destroy(h)


@pytest.mark.parametrize("kw", [
    dict(stats=None), dict(dy=None), dict(dx=None), dict(dx=64 * M + 16), dict(dx=48 * M), dict(dw=81 * M), dict(dw=83 * M + 2),
    dict(db=83 * M), dict(dxs=(3200, 8, 56)),
], ids=str)
def test_norm_backward_calls_that_are_refused(kw):
    binding, ops = _lib()
    st, h = _open("norm", ops.NormConfig(C=64, groups=8, act=1, eps=1e-5, dtype=1))
    assert st == 0
    a = dict(dict(dy=64 * M, x=48 * M, stats=82 * M, dx=96 * M, dw=83 * M, db=84 * M, dxs=(3200, 8, 64)), **kw)
    call = lambda ws, n: binding.LIB.ttt_norm_backward(  # noqa: E731
        h, 2, 50, a["dy"], _s(3200, 8, 64), a["x"], _s(3200, 8, 64), 80 * M, 81 * M, a["stats"], a["dx"], _s(*a["dxs"]),
        a["dw"], a["db"], ws, n, None, None)
    assert call(112 * M, 1 << 30) == binding.TTT_ERR_INVALID_ARG
    a.update(stats=82 * M, dy=64 * M, dx=96 * M, dw=83 * M, db=84 * M, dxs=(3200, 8, 64))
    need = binding.LIB.ttt_norm_workspace_size(h, 2, 50, 1)
    assert need > 0 and call(112 * M, need - 1) == binding.TTT_ERR_WORKSPACE
    assert call(None, 0) == binding.TTT_ERR_WORKSPACE
    binding.LIB.ttt_norm_destroy(h)


def test_columns_of_one_buffer_that_share_an_element_are_refused():
    """g, x and h as column ranges of one [B, L, 3D] buffer, with h one column too early or too late."""
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(D=64, gate=1, input=1, dtype=1))
    a = dict(FWD_OK, gs=(700 * 192, 0, 192), xs=(700 * 192, 0, 192), hs=(700 * 192, 0, 192), g=64 * M, x=64 * M + 128)
    assert _forward(h, dict(a, h=64 * M + 254)) == binding.TTT_ERR_INVALID_ARG  # x's last column
    assert _forward(h, dict(a, h=64 * M + 258)) == binding.TTT_ERR_INVALID_ARG  # g's first, one token on
    binding.LIB.ttt_scan_destroy(h)


def test_the_binding_refuses_what_is_not_on_its_device():
    """Host checks of the native module, before any call of the library."""
    import torch
    binding, ops = _lib()
    op = ops.RotaryPositions(dict(d=8, pairs=(4,), dtype="bf16"), device="cuda:0")
    x, pos = torch.zeros((1, 1, 1, 8), dtype=torch.bfloat16), torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="cuda:0"):
        op.forward(x, pos)
    with pytest.raises(ValueError, match="shape"):
        op.forward(x[..., :4], pos)
    with pytest.raises(ValueError, match="shape"):
        op.forward(x.float(), pos)
    with pytest.raises(TypeError):
        op.forward([0.0] * 8, pos)
    with pytest.raises(TypeError):
        op.forward(x, None)
    op.close()
    op.close()
    with pytest.raises(ValueError, match="closed"):
        op.forward(x, pos)
    with pytest.raises(binding.TTTError):
        ops.RotaryPositions(dict(d=7, pairs=(4,), dtype="bf16"))
    with pytest.raises(KeyError):
        ops.RotaryPositions(dict(d=8, pairs=(4,), dtype="f16"))
    with pytest.raises(ValueError):
        ops.RotaryPositions(dict(d=8, pairs=(4,), dtype="bf16"), device="cpu")


def test_scan_timeout_selftest_calls_that_are_refused():
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(D=64, gate=1, input=1, dtype=1))
    call = lambda h=h, L=700, status=99 * M, ms=20, ws=160 * M: binding.LIB.ttt_selftest_scan_timeout(  # noqa: E731
        h, 2, L, 64 * M, _s(L * 64, 0, 64), 80 * M, _s(L * 64, 0, 64), 112 * M, _s(L * 64, 0, 64), ws, 1 << 30, status, ms,
        None)
    for bad in (dict(h=None), dict(status=None), dict(ms=0), dict(ms=2001), dict(ms=-1), dict(ws=160 * M + 8)):
        assert call(**bad) == binding.TTT_ERR_INVALID_ARG, bad
    assert call(ws=None) == binding.TTT_ERR_WORKSPACE
    for L in (0, 1, 16, 17, 256):  # no tile waits for another
        assert call(L=L) == binding.TTT_ERR_UNSUPPORTED, L
    binding.LIB.ttt_scan_destroy(h)


@pytest.mark.parametrize("L,states", [(0, 0), (1, 1), (16, 1), (128, 1), (129, 2), (256, 2), (257, 3), (5001, 40)])
def test_scan_keeps_the_states_that_backward_reads(L, states):
    """One for each of the backward pass's tiles of 128 tokens, fp32."""
    binding, ops = _lib()
    st, h = _open("scan", ops.ScanConfig(D=33, gate=1, input=1, dtype=1))
    assert st == 0 and binding.LIB.ttt_scan_saved_size(h, 5, L) == 5 * states * 33 * 4
    binding.LIB.ttt_scan_destroy(h)


def test_sizes_past_the_stated_limits_are_unsupported():
    binding, ops = _lib()
    for d, want in ((4096, 0), (4097, binding.TTT_ERR_UNSUPPORTED)):
        st, h = _open("rope", _rope_cfg(d=d))
        assert st == want, d
        binding.LIB.ttt_rope_destroy(h)
    st, h = _open("rope", _rope_cfg())
    s = _s(1 << 47, 1 << 47, 64)
    assert binding.LIB.ttt_rope_apply(h, 1, 1, (1 << 40) + 1, 1 << 50, s, 1 << 52, 0, 0, 1 << 54, s, 0,
                                      None) == binding.TTT_ERR_UNSUPPORTED
    binding.LIB.ttt_rope_destroy(h)
    far = lambda k: k << 50  # noqa: E731
    for dtype, c in ((0, 32), (1, 64)):
        st, h = _open("scan", ops.ScanConfig(D=c + 1, gate=1, input=1, dtype=dtype))  # two columns of channels
        assert st == 0
        for backward, tile in ((False, 256), (True, 128)):
            B, L = (1 << 28) + 1, tile + 1  # two tiles
            s = _s(L * (c + 1), 0, c + 1)
            if backward:
                st = binding.LIB.ttt_scan_backward(h, B, L, far(1), s, None, far(2), s, far(3), s, None, far(4), far(5), s,
                                                   far(6), s, None, far(7), 1 << 62, None, None)
            else:
                st = binding.LIB.ttt_scan_forward(h, B, L, far(1), s, far(2), s, None, None, far(3), s, None, None, far(7),
                                                  1 << 62, None, None)
            assert st == binding.TTT_ERR_UNSUPPORTED, (dtype, backward)
        binding.LIB.ttt_scan_destroy(h)
