"""Refusals and host-side rules of the training operators (CPU only: every
call here returns before the library makes its first CUDA call)."""
import ctypes

import pytest
import torch

import _train64 as ref
from row_wise_rmsnorm_fwd_gb300 import binding, build

OK, INVALID, UNSUPPORTED = (binding.RMSNORM_OK, binding.RMSNORM_ERR_INVALID_ARG,
                            binding.RMSNORM_ERR_UNSUPPORTED)

# fake, 256-byte aligned "device" addresses, 256 MB apart: never dereferenced
X, DY, W, B, Y, MEAN, RSTD, DW, DB, WS = (0x10000000 * k for k in range(1, 11))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def options(**kw):
    return ctypes.byref(binding.make_options(**kw))


def test_declared_and_exported(lib):
    names = set(binding.declared_functions())
    for family in ("layernorm_fwd", "layernorm_bwd", "rmsnorm_bwd", "rowsoftmax_relbias_fwd",
                   "rowsoftmax_relbias_bwd"):
        for suffix in ("_f32", "_bf16", "_ex"):
            assert family + suffix in names and hasattr(lib, family + suffix)
    assert {"layernorm_bwd_workspace", "rmsnorm_bwd_workspace", "rowsoftmax_relbias_bwd_workspace",
            "rowsoftmax_relbias_bucket"} <= names
    assert ctypes.sizeof(binding.rowsoftmax_relbias_t) == 48


def test_layernorm_forward_refuses(lib):
    def f(x=X, w=W, b=B, y=Y, mean=MEAN, rstd=RSTD, rows=4, hidden=8, eps=1e-5, dt=0, opt=None):
        return lib.layernorm_fwd_ex(dt, x, w, b, y, mean, rstd, rows, hidden, eps, opt, None)

    for kw in (dict(x=0), dict(y=0), dict(rows=-1), dict(hidden=0), dict(hidden=-1),
               dict(hidden=2 ** 31), dict(rows=2 ** 62, hidden=2 ** 20), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(eps=-1e-9), dict(dt=2), dict(x=X + 1), dict(w=W + 2),
               dict(mean=MEAN + 2), dict(y=X + 16), dict(w=Y + 8), dict(b=Y), dict(mean=Y + 4),
               dict(mean=X), dict(rstd=MEAN + 4), dict(rstd=MEAN), dict(rstd=W),
               dict(opt=options(cluster=2)), dict(opt=options(threads=32)),
               dict(opt=options(path="rowreg")), dict(opt=options(epilogue=1)),
               dict(opt=options(fault_inject=3))):
        assert f(**kw) == INVALID, kw
    assert f(opt=options(path="twopass", fault_inject=1)) == UNSUPPORTED
    assert f(rows=0) == OK and f(rows=0, y=X) == OK and f(rows=0, w=0, b=0, mean=0, rstd=0) == OK
    assert lib.layernorm_fwd_f32(0, W, B, Y, None, None, 4, 8, 1e-5, None) == INVALID
    assert lib.layernorm_fwd_bf16(X + 1, W, B, Y, None, None, 4, 8, 1e-5, None) == INVALID
    assert lib.layernorm_fwd_bf16(X, W, B, Y, None, None, 0, 8, 1e-5, None) == OK


def test_norm_backward_refuses(lib):
    def layer(dy=DY, x=X, w=W, mean=MEAN, rstd=RSTD, dx=Y, dw=DW, db=DB, rows=4, hidden=8, ws=WS,
              n=1 << 20, dt=0, opt=None):
        return lib.layernorm_bwd_ex(dt, dy, x, w, mean, rstd, dx, dw, db, rows, hidden, ws, n, opt,
                                    None)

    def rms(dy=DY, x=X, w=W, dx=Y, dw=DW, rows=4, hidden=8, eps=1e-6, ws=WS, n=1 << 20, dt=0,
            opt=None):
        return lib.rmsnorm_bwd_ex(dt, dy, x, w, dx, dw, rows, hidden, eps, ws, n, opt, None)

    both = (dict(dy=0), dict(x=0), dict(dx=0), dict(rows=-1), dict(hidden=0), dict(hidden=2 ** 31),
            dict(rows=2 ** 60, hidden=2 ** 10), dict(dt=-1), dict(dy=DY + 2), dict(dw=DW + 2),
            dict(ws=WS + 8), dict(ws=0), dict(dx=X + 16), dict(dx=DY + 4), dict(dx=W),
            dict(dw=X), dict(dw=Y), dict(dw=W), dict(ws=X), dict(ws=DW - 64), dict(ws=Y),
            dict(opt=options(grid=4)), dict(opt=options(path="cluster")),
            dict(opt=options(stages=2)))
    for kw in both:
        assert layer(**kw) == INVALID, kw
        assert rms(**kw) == INVALID, kw
    for kw in (dict(mean=0), dict(rstd=0), dict(mean=MEAN + 1), dict(db=DB + 1), dict(db=DW),
               dict(dx=MEAN), dict(ws=DB), dict(db=RSTD)):
        assert layer(**kw) == INVALID, kw
    for kw in (dict(eps=-1.0), dict(eps=float("nan"))):
        assert rms(**kw) == INVALID, kw
    assert layer(rows=0, dw=0, db=0) == OK and rms(rows=0, dw=0, ws=0) == OK
    assert layer(opt=options(fault_inject=1)) == UNSUPPORTED
    size = ctypes.c_size_t(7)
    for fn in (lib.layernorm_bwd_workspace, lib.rmsnorm_bwd_workspace):
        assert fn(0, 4, 8, None) == INVALID
        assert fn(3, 4, 8, ctypes.byref(size)) == INVALID
        assert fn(0, -1, 8, ctypes.byref(size)) == INVALID
        assert fn(0, 0, 8, ctypes.byref(size)) == OK and size.value == 0


def test_relbias_refuses(lib):
    def rule(**kw):
        a = dict(num_buckets=32, max_distance=128, bidirectional=1, causal=0, scale=1.0, reserved=0,
                 q_offset=0, q_start=None, kv_len=None)
        a.update(kw)
        return binding.rowsoftmax_relbias_t(*a.values())

    def f(x=X, table=W, y=Y, b=2, h=3, q=4, k=8, a=None, dt=0, opt=None, **kw):
        a = rule(**kw) if a is None else a
        return lib.rowsoftmax_relbias_fwd_ex(dt, x, table, y, b, h, q, k, ctypes.byref(a), opt, None)

    def g(dy=DY, y=Y, dx=X, dt=DW, b=2, h=3, q=4, k=8, ws=WS, n=1 << 20, type=0, opt=None, **kw):
        return lib.rowsoftmax_relbias_bwd_ex(type, dy, y, dx, dt, b, h, q, k,
                                             ctypes.byref(rule(**kw)), ws, n, opt, None)

    for kw in (dict(b=-1), dict(h=0), dict(q=-1), dict(k=0), dict(k=(1 << 30) + 1), dict(h=65536),
               dict(b=1 << 16, q=1 << 16), dict(b=1 << 32, q=0), dict(num_buckets=1),
               dict(num_buckets=257), dict(num_buckets=33), dict(num_buckets=2),
               dict(max_distance=8), dict(max_distance=4097), dict(max_distance=-1),
               dict(bidirectional=2), dict(causal=-1), dict(reserved=1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q_offset=(1 << 40) + 1),
               dict(q_offset=-(1 << 40) - 1), dict(q_start=B + 2), dict(kv_len=B + 1),
               dict(opt=options(vec_bytes=16)), dict(opt=options(path="staged")),
               dict(opt=options(fault_inject=1)),
               dict(b=1 << 15, q=1 << 15, h=65535, k=1 << 30)):
        assert f(**kw) == INVALID, kw
        assert g(**kw) == INVALID, kw
    for kw in (dict(x=0), dict(table=0), dict(y=0), dict(dt=2), dict(x=X + 2), dict(y=X + 4),
               dict(table=Y + 8), dict(q_start=Y), dict(kv_len=Y + 16)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(dy=0), dict(y=0), dict(dx=0), dict(type=5), dict(dt=DW + 1), dict(dx=Y + 4),
               dict(dt=X), dict(dt=DY), dict(ws=0), dict(ws=WS + 4), dict(ws=X), dict(ws=DW),
               dict(kv_len=X), dict(q_start=WS)):
        assert g(**kw) == INVALID, kw
    assert f(b=0) == OK and f(q=0) == OK and g(b=0, dt=0) == OK and g(q=0, dt=0, ws=0) == OK
    assert lib.rowsoftmax_relbias_fwd_ex(0, X, W, Y, 1, 1, 1, 1, None, None, None) == INVALID
    size = ctypes.c_size_t(7)
    a = rule()
    assert lib.rowsoftmax_relbias_bwd_workspace(0, 0, 3, 4, 8, ctypes.byref(a),
                                                ctypes.byref(size)) == OK and size.value == 0
    assert lib.rowsoftmax_relbias_bwd_workspace(0, 1, 3, 4, 8, ctypes.byref(a), None) == INVALID


@pytest.mark.parametrize("both", [True, False])
@pytest.mark.parametrize("num_buckets,distance", [
    (32, 128), (32, 64), (64, 128), (16, 500), (4, 2), (4, 3), (256, 4096), (256, 500), (128, 4096),
    (10, 17), (62, 4095), (34, 1024), (12, 81), (8, 16), (250, 63), (200, 4000)])
def test_bucket_rule_in_whole_numbers(lib, num_buckets, distance, both):
    """Every distance on both sides of every edge, against exact fractions."""
    half = num_buckets // 2 if both else num_buckets
    if distance <= half // 2:
        assert binding.rowsoftmax_relbias_bucket(0, num_buckets, distance, both) == -1
        return
    edges = ref.bucket_edges(half, distance)
    probes = {0, 1, distance, distance + 1, 2 ** 40} | {e + d for e in edges for d in (-1, 0, 1)}
    for n in sorted(p for p in probes if p >= 0):
        for r in (n, -n):
            away = n if both else max(-r, 0)
            want = sum(e <= away for e in edges) - 1 + (half if both and r > 0 else 0)
            got = binding.rowsoftmax_relbias_bucket(r, num_buckets, distance, both)
            assert got == want, (r, got, want)


def test_well_known_buckets(lib):
    """32 buckets up to distance 128: 0..7 one by one, then 8, 12, 16, 23, 32,
    46, 64, 91 (8 * 16^(k/8), rounded up) open the next ones."""
    edges = [0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91]
    assert ref.bucket_edges(16, 128) == edges
    for k, e in enumerate(edges):
        assert binding.rowsoftmax_relbias_bucket(-e, 32) == k
        if e:
            assert binding.rowsoftmax_relbias_bucket(e, 32) == 16 + k
    assert binding.rowsoftmax_relbias_bucket(-(2 ** 63), 32) == 15
    assert binding.rowsoftmax_relbias_bucket(5, 32, 128, False) == 0


def test_tensors_are_refused_on_the_host(lib):
    x = torch.zeros((4, 8))
    w = torch.ones(8)
    with pytest.raises(ValueError, match="CUDA"):
        binding.layernorm_fwd_f32(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        binding.rmsnorm_bwd_f32(x, x, w)
    with pytest.raises(TypeError):
        binding.layernorm_fwd_bf16(x, w)
    with pytest.raises(TypeError):
        binding.layernorm_fwd_ex(x.half(), w.half())
    with pytest.raises(ValueError, match="non-empty"):
        binding.layernorm_fwd_f32(torch.zeros((3, 0)))
    with pytest.raises(ValueError, match="scores"):
        binding.rowsoftmax_relbias_fwd_f32(torch.zeros((2, 3, 4, 5)), torch.zeros((32, 3)))
    with pytest.raises(ValueError, match="scores"):
        binding.rowsoftmax_relbias_bwd_f32(x, x, 32)


def test_references_against_autograd():
    """The 64-bit backward references against torch's differentiation of the
    64-bit forward ones."""
    for rows, hidden in ((5, 7), (3, 64)):
        x = ref.make((rows, hidden), "f32", 1).double().requires_grad_()
        w = ref.make((hidden,), "f32", 2).double().requires_grad_()
        b = ref.make((hidden,), "f32", 3).double().requires_grad_()
        dy = ref.make((rows, hidden), "f32", 4).double()
        (y, mean, rstd), _ = ref.layernorm(x, w, b, 1e-5)
        want = torch.autograd.grad(y, (x, w, b), dy)
        got, _ = ref.layernorm_bwd(dy, x.detach(), w.detach(), mean.detach(), rstd.detach())
        for g, r in zip(got, want):
            assert (g - r).abs().max() < 1e-9
        y = x * ((x * x).mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        want = torch.autograd.grad(y, (x, w), dy)
        got, _ = ref.rmsnorm_bwd(dy, x.detach(), w.detach(), 1e-6)
        for g, r in zip(got, want):
            assert (g - r).abs().max() < 1e-9
    rule = ref.Rule(causal=True, scale=0.3, q_start=[3, 0], kv_len=[6, 9])
    x = ref.make((2, 3, 4, 9), "f32", 5).double().requires_grad_()
    table = ref.make((32, 3), "f32", 6).double().requires_grad_()
    dy = ref.make((2, 3, 4, 9), "f32", 7).double()
    y, _ = ref.relbias(x, table, rule)
    want = torch.autograd.grad(y, (x, table), dy)
    got, _ = ref.relbias_bwd(dy, y.detach(), rule)
    for g, r in zip(got, want):
        assert (g - r).abs().max() < 1e-9
