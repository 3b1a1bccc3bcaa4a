"""Refusals and host-side rules of the block boundary and of rotary positions (CPU only:
every call here returns before the library makes its first CUDA call)."""
import ctypes
import math

import pytest
import torch

import _between64 as ref
from row_wise_rmsnorm_fwd_gb300 import binding, build

OK, INVALID, UNSUPPORTED = (binding.RMSNORM_OK, binding.RMSNORM_ERR_INVALID_ARG,
                            binding.RMSNORM_ERR_UNSUPPORTED)

# fake, 256-byte aligned "device" addresses, 256 MB apart: never dereferenced
(X, RES, H, Y, DY, DH, DX, DRES, POST, PRE, GATE, DPOST, DPRE, DGATE, WS, FREQ,
 POS) = (0x10000000 * k for k in range(1, 18))
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def options(**kw):
    return ctypes.byref(binding.make_options(**kw))


def test_declared_and_exported(lib):
    names = set(binding.declared_functions())
    for family in ("rmsnorm_block_fwd", "rmsnorm_block_bwd", "rmsnorm_rope_fwd", "rmsnorm_rope_bwd"):
        for suffix in ("_f32", "_bf16", "_ex"):
            assert family + suffix in names and hasattr(lib, family + suffix)
    assert {"rmsnorm_block_bwd_workspace", "rmsnorm_rope_bwd_workspace", "rmsnorm_rope_freqs"} <= names
    assert ctypes.sizeof(binding.rmsnorm_block_t) == 56
    assert ctypes.sizeof(binding.rmsnorm_rope_heads_t) == 120
    assert ctypes.sizeof(binding.rmsnorm_rope_t) == 56
    assert ctypes.sizeof(binding.rmsnorm_rope_rule_t) == 56


def block(post_w=POST, pre_w=PRE, gate=GATE, gate_rows=4, residual_scale=1.0, branch_scale=1.0,
          post_eps=1e-6, pre_eps=1e-6, post_norm=1, pre_norm=1):
    return binding.rmsnorm_block_t(post_w, pre_w, gate, gate_rows, residual_scale, branch_scale,
                                   post_eps, pre_eps, post_norm, pre_norm)


NAN, INF = float("nan"), float("inf")
BAD_RULES = [dict(gate_rows=0), dict(gate_rows=-3), dict(residual_scale=NAN), dict(branch_scale=INF),
             dict(post_eps=-1e-9), dict(pre_eps=NAN), dict(post_eps=INF), dict(post_norm=2),
             dict(pre_norm=-1), dict(post_w=POST + 2), dict(pre_w=PRE + 1), dict(gate=GATE + 3)]
BAD_OPTIONS = [dict(path="ringreg"), dict(path="cluster"), dict(threads=64), dict(epilogue="relu"),
               dict(fault_inject=3), dict(grid=3), dict(cluster=2), dict(cluster=3, path="staged")]


def test_block_forward_refuses(lib):
    def f(x=X, residual=RES, h=H, y=Y, rows=4, hidden=8, dt=0, opt=None, rule=None, **kw):
        b = block(**kw) if rule is None else rule
        return lib.rmsnorm_block_fwd_ex(dt, x, residual, h, y, rows, hidden,
                                        ctypes.byref(b) if b else None, opt, None)

    for kw in BAD_RULES + [
            dict(x=0), dict(residual=0), dict(h=0), dict(y=0), dict(pre_norm=0), dict(rule=False),
            dict(rows=-1), dict(hidden=0), dict(hidden=-1), dict(hidden=2 ** 20 + 1),
            dict(rows=2 ** 60), dict(dt=2), dict(x=X + 2), dict(h=H + 1), dict(y=Y + 2),
            dict(h=X + 16), dict(y=H), dict(y=H + 32), dict(h=POST), dict(y=PRE + 16),
            dict(h=GATE - 96), dict(y=RES + 64), dict(h=RES - 4)]:
        assert f(**kw) == INVALID, kw
    for o in BAD_OPTIONS:
        assert f(opt=options(**o)) == INVALID, o
    for o in (dict(fault_inject=1), dict(fault_inject=2, path="staged", cluster=2)):
        assert f(opt=options(**o)) == UNSUPPORTED, o          # the test build's
    for h, y in ((H, Y), (X, RES), (RES, X), (X, Y)):
        assert f(rows=0, h=h, y=y) == OK
    assert f(rows=0, pre_norm=0, y=0) == OK
    assert f(rows=0, gate=0, gate_rows=0) == OK


def test_block_backward_refuses(lib):
    def f(dy=DY, dh=DH, x=X, h=H, dx=DX, dres=DRES, dpost=DPOST, dpre=DPRE, dgate=DGATE, rows=4,
          hidden=8, ws=WS, n=BIG, dt=0, opt=None, **kw):
        return lib.rmsnorm_block_bwd_ex(dt, dy, dh, x, h, dx, dres, dpost, dpre, dgate, rows, hidden,
                                        ctypes.byref(block(**kw)), ws, n, opt, None)

    n = 1 << 20
    for kw in BAD_RULES + [
            dict(dy=0), dict(x=0), dict(h=0), dict(dx=0), dict(dres=0), dict(pre_norm=0),
            dict(post_norm=0), dict(gate=0), dict(pre_norm=0, dy=0), dict(rows=-1), dict(hidden=0),
            dict(hidden=2 ** 20 + 1), dict(rows=2 ** 60), dict(dt=-1), dict(dy=DY + 2),
            dict(dpost=DPOST + 2), dict(dgate=DGATE + 1), dict(ws=WS + 8), dict(ws=0),
            dict(dx=DRES), dict(dx=DRES + 16), dict(dx=X + 16), dict(dres=H - 32), dict(dx=POST),
            dict(dres=GATE), dict(dpost=DX), dict(dpre=DPOST), dict(dgate=DPRE + 16),
            dict(dpre=DY), dict(dgate=GATE), dict(ws=DX - 64, n=n), dict(ws=DGATE, n=n),
            dict(ws=PRE, n=n)]:
        assert f(**{"n": n, **kw}) == INVALID, kw
    for o in BAD_OPTIONS:
        assert f(n=n, opt=options(**o)) == INVALID, o
    assert f(rows=0, dpost=0, dpre=0, dgate=0, ws=0, n=0) == OK
    assert f(rows=0, dpost=0, dpre=0, dgate=0, dx=X, dres=DY, ws=0, n=0) == OK
    size = ctypes.c_size_t(7)
    w = lambda dt=0, rows=4, hidden=8, **kw: lib.rmsnorm_block_bwd_workspace(  # noqa: E731
        dt, rows, hidden, ctypes.byref(block(**kw)), ctypes.byref(size))
    assert w(dt=3) == w(rows=-1) == w(hidden=0) == w(gate_rows=0) == INVALID
    assert lib.rmsnorm_block_bwd_workspace(0, 4, 8, ctypes.byref(block()), None) == INVALID
    assert w(rows=0) == OK and size.value == 0


def heads(x=X, dy=0, out=Y, w=POST, dw=0, n=4, d=8, strides=None, out_strides=None):
    three = lambda s: (ctypes.c_int64 * 3)(*s)  # noqa: E731
    s = strides or (3 * n * d, n * d, d)
    return binding.rmsnorm_rope_heads_t(x, dy, out, w, dw, n, three(s), three(s), three(out_strides or s))


def rope(freqs=FREQ, positions=POS, n_positions=6, start=0, position_bytes=8, rot_dim=8,
         interleaved=0, norm=1, eps=1e-6, mscale=1.0):
    return binding.rmsnorm_rope_t(freqs, positions, n_positions, start, position_bytes, rot_dim,
                                  interleaved, norm, eps, mscale)


BAD_ROPES = [dict(freqs=0), dict(freqs=FREQ + 4), dict(n_positions=0), dict(position_bytes=2),
             dict(positions=POS + 4), dict(positions=POS + 2, position_bytes=4), dict(rot_dim=0),
             dict(rot_dim=7), dict(rot_dim=10), dict(interleaved=2), dict(norm=-1), dict(eps=-1.0),
             dict(eps=NAN), dict(mscale=INF)]
# q and k in one array of 6 heads of 8 to a token, 2 batches of 3 tokens
PACKED = (3 * 48, 48, 8)
BAD_VIEWS = [
    (dict(strides=(96, -32, 8)), {}), (dict(out_strides=(96, 32, 7)), {}),
    (dict(out_strides=(96, 8, 8)), {}), (dict(out_strides=(0, 32, 8)), {}),
    (dict(out_strides=(48, 32, 8)), {}), (dict(strides=(2 ** 62, 2 ** 62, 2 ** 62)), {}),
    (dict(out=X + 32), {}), (dict(out=X, out_strides=(192, 32, 8)), {}), (dict(n=0), {}),
    (dict(x=0), {}), (dict(out=0), {}), (dict(x=X + 2), {}), (dict(out=Y + 1), {}),
    (dict(w=POST + 2), {}), (dict(out=POST), {}), (dict(out=FREQ), {}), (dict(out=POS - 64), {}),
    ({}, dict(out=Y)), ({}, dict(out=Y + 4)), ({}, dict(out=X)),
    # interleaved heads that meet: k one head further to the left than it may be
    (dict(x=X, out=X, strides=PACKED), dict(x=X + 4 * 24, out=X + 4 * 24, strides=PACKED, n=2)),
]


def test_rope_forward_refuses(lib):
    def f(q=None, k=None, batch=2, seq=3, dim=8, dt=0, opt=None, r=True, **kw):
        rule = ctypes.byref(rope(**kw)) if r else None
        return lib.rmsnorm_rope_fwd_ex(dt, q, k, batch, seq, dim, rule, opt, None)

    q, k = heads(), heads(x=DY, out=DX, n=2)
    b = ctypes.byref
    for kw in BAD_ROPES + [dict(r=False), dict(batch=-1), dict(seq=-1), dict(dim=1), dict(dim=1025),
                           dict(dt=2), dict(batch=2 ** 40), dict(batch=2 ** 62, seq=2 ** 62)]:
        assert f(b(q), b(k), **kw) == INVALID, kw
    assert f(None, b(k)) == INVALID
    for one, two in BAD_VIEWS:
        two = {"x": DY, "out": DX, "n": 2, **two}
        assert f(b(heads(**one)), b(heads(**two))) == INVALID, (one, two)
    assert f(b(heads(dw=DPOST)), b(k)) == INVALID
    for o in BAD_OPTIONS:
        assert f(b(q), b(k), opt=options(**o)) == INVALID, o
    assert f(b(q), b(k), batch=0) == OK
    assert f(b(q), None, seq=0) == OK


def test_rope_backward_refuses(lib):
    def f(q=None, k=None, batch=2, seq=3, dim=8, dt=0, ws=WS, n=1 << 20, opt=None, **kw):
        return lib.rmsnorm_rope_bwd_ex(dt, q, k, batch, seq, dim, ctypes.byref(rope(**kw)), ws, n,
                                       opt, None)

    b = ctypes.byref
    q = heads(dy=DY, dw=DPOST)
    k = heads(x=RES, dy=DH, out=DX, n=2, dw=DPRE)
    for kw in BAD_ROPES + [dict(ws=0), dict(ws=WS + 8), dict(norm=0), dict(ws=Y - 64), dict(ws=X),
                           dict(ws=DPRE), dict(ws=FREQ)]:
        assert f(b(q), b(k), **kw) == INVALID, kw
    for one in (dict(dy=0), dict(dw=DPOST + 1), dict(dw=Y), dict(dw=X), dict(dw=POST), dict(x=0),
                dict(dw=DPRE), dict(out=DY + 32), dict(out=DH), dict(out=RES)):
        assert f(b(heads(**{"dy": DY, "dw": DPOST, **one})), b(k)) == INVALID, one
    assert f(b(heads(dy=DY)), b(heads(x=RES, dy=DH, out=DX, n=2)), batch=0, ws=0, n=0) == OK
    size = ctypes.c_size_t(7)
    w = lambda *a: lib.rmsnorm_rope_bwd_workspace(*a, ctypes.byref(size))  # noqa: E731
    for a in ((2, 1, 1, 1, 8), (0, -1, 1, 1, 8), (0, 1, 1, 0, 8), (0, 1, 1, 1, 1), (0, 1, 1, 1, 1025),
              (0, 2 ** 40, 2, 1, 8), (0, 2 ** 62, 2 ** 62, 1, 8)):
        assert w(*a) == INVALID, a
    assert lib.rmsnorm_rope_bwd_workspace(0, 1, 1, 1, 8, None) == INVALID
    assert w(0, 0, 5, 1, 8) == OK and size.value == 0


RULES = [dict(), dict(base=5e5), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
         dict(scaling="ramp", factor=4.0, original_len=4096),
         dict(scaling="ramp", factor=16.0, original_len=64, low=0.5, high=2.0),
         dict(scaling="bands", factor=8.0, original_len=8192, base=5e5),
         dict(scaling="bands", factor=2.0, original_len=100, low=0.25, high=8.0)]


@pytest.mark.parametrize("rot", [4, 20, 64, 128])
@pytest.mark.parametrize("rule", RULES)
def test_frequencies(rot, rule):
    """Against 64-bit formulas, whose powers and quotients are off by 2^-50 of a frequency
    (exponents of up to 13 at 2^-53 each, times ln(base) < 14: 14 * 13 * 2^-53 < 2^-45)."""
    freqs, mscale = binding.rmsnorm_rope_freqs(rot, device="cpu", **rule)
    want, scale = ref.rope_frequencies(rot, **rule)
    assert freqs.dtype == torch.int64 and freqs.shape == (rot // 2,)
    assert abs(mscale - scale) <= 2.0 ** -24 * scale
    for got, f in zip(freqs.tolist(), want.tolist()):
        assert abs(got % 2 ** 64 / 2 ** 64 * 2 * math.pi - f) <= 2.0 ** -45 * f + 2.0 ** -62


def test_frequencies_with_divisors():
    div = [1.0 + i for i in range(16)]
    one, _ = binding.rmsnorm_rope_freqs(32, device="cpu")
    two, _ = binding.rmsnorm_rope_freqs(32, device="cpu", divisors=div)
    for a, b, d in zip(one.tolist(), two.tolist(), div):
        assert abs(b % 2 ** 64 * int(d) - a % 2 ** 64) <= d + a % 2 ** 64 * 2.0 ** -60
    # more than a turn a position: modulo a turn
    f, _ = binding.rmsnorm_rope_freqs(2, device="cpu", divisors=[1 / (2 * math.pi * 1.25)])
    assert abs(f.item() % 2 ** 64 / 2 ** 64 - 0.25) < 1e-14


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=2 ** 40), dict(scaling="other"),
    dict(divisors=[1.0]), dict(original_len=2 ** 70)])
def test_frequencies_refuse_in_python(kw):
    with pytest.raises(ValueError):
        binding.rmsnorm_rope_freqs(**{"rot_dim": 8, "device": "cpu", **kw})


@pytest.mark.parametrize("kw", [
    dict(base=1.0), dict(base=NAN), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=NAN),
    dict(scaling="ramp", factor=2.0), dict(scaling="ramp", factor=2.0, original_len=8, low=3.0, high=3.0),
    dict(scaling="bands", factor=2.0, original_len=8, low=-1.0), dict(rot_dim=2, scaling="base", factor=2.0),
    dict(divisors=[1.0, 0.0, 1.0, 1.0]), dict(divisors=[1.0, INF, 1.0, 1.0]), dict(rot_dim=1026)])
def test_frequencies_refuse(kw):
    with pytest.raises(binding.RmsnormError):
        binding.rmsnorm_rope_freqs(**{"rot_dim": 8, "device": "cpu", **kw})


def test_cpu_tensors_are_refused():
    x, w = torch.zeros(3, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        binding.rmsnorm_block_fwd_f32(x, x, w, w)
    with pytest.raises(ValueError):
        binding.rmsnorm_block_bwd_f32(x, x, x, x, w, w)
    q, f = torch.zeros(3, 2, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        binding.rmsnorm_rope_fwd_f32(q, q, f)
    with pytest.raises(ValueError):
        binding.rmsnorm_rope_bwd_f32(q, q, f)
    with pytest.raises(TypeError):
        binding.rmsnorm_block_fwd_bf16(x, x)
    with pytest.raises(TypeError):
        binding.rmsnorm_rope_fwd_bf16(q, q, f)
