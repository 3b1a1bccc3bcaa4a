"""Layer norm forward and backward, and RMSNorm backward, against 64-bit
references (GPU)."""
import ctypes

import pytest
import torch

import _train64 as ref
from _train64 import TYPES, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


# rows, hidden: one element, less than a vector, odd, ragged, each vector width,
# several rows per warp, one per CTA, rows too wide for one CTA's registers
SHAPES = [(1, 1), (5, 3), (3, 8), (7, 33), (33, 64), (300, 100), (9, 257), (200, 512),
          (31, 1000), (128, 2048), (17, 2050), (40, 3584), (19, 4097), (3, 8191), (160, 8192),
          (5, 8200), (3, 16384), (2, 16390), (2, 40000), (1, 70001),
          # rows that touch a boundary differently one after the other: every odd residue, few
          # rows per alignment, the last row's end on and off a boundary
          (1, 16), (2, 17), (9, 19), (16, 21), (23, 23), (8, 1025), (9, 1026), (41, 1028),
          (7, 12001), (10, 12002), (3, 16383)]
PATHS = [None, {"path": "twopass"}]


def inputs(t, rows, hidden, seed=1):
    x = make((rows, hidden), t, seed, mean=0.5, std=2.0)
    return (x, make((hidden,), t, seed + 1, mean=1.0, std=0.1), make((hidden,), t, seed + 2),
            make((rows, hidden), t, seed + 3))


def fwd(x, w, b, eps=1e-5, **kw):
    gpu = [None if v is None else v.cuda() for v in (x, w, b)]
    return binding.layernorm_fwd_ex(*gpu, eps=eps, stats=True, **kw)


def check_fwd(got, x, w, b, eps=1e-5):
    want, tol = ref.layernorm(x, w, b, eps)
    for g, r, t, n in zip(got, want, tol, ("y", "mean", "rstd")):
        close(g, r, t, n)


def check_layer_bwd(dy, x, w, options=None, eps=1e-5):
    _, mean, rstd = ref.layernorm(x, w, None, eps)[0]
    mean, rstd = mean.float(), rstd.float()
    gpu = [None if v is None else v.cuda() for v in (dy, x, w, mean, rstd)]
    got = binding.layernorm_bwd_ex(*gpu, options=options)
    want, tol = ref.layernorm_bwd(dy, x, w, mean, rstd)
    for g, r, t, n in zip(got, want, tol, ("dx", "dw", "db")):
        close(g, r, t, n)


def check_rms_bwd(dy, x, w, options=None, eps=1e-6):
    gpu = [None if v is None else v.cuda() for v in (dy, x, w)]
    got = binding.rmsnorm_bwd_ex(*gpu, eps=eps, options=options)
    want, tol = ref.rmsnorm_bwd(dy, x, w, eps)
    for g, r, t, n in zip(got, want, tol, ("dx", "dw")):
        close(g, r, t, n)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_forward(rows, hidden, t, options):
    x, w, b, _ = inputs(t, rows, hidden)
    check_fwd(fwd(x, w, b, options=options), x, w, b)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_layernorm_backward(rows, hidden, t, options):
    x, w, _, dy = inputs(t, rows, hidden)
    check_layer_bwd(dy, x, w, options)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_rmsnorm_backward(rows, hidden, t, options):
    x, w, _, dy = inputs(t, rows, hidden)
    check_rms_bwd(dy, x, w, options)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(2000, 64), (700, 1024), (1300, 2048), (611, 130), (900, 5120),
                                         (3001, 33), (2500, 255), (1999, 1001), (1500, 2050)])
def test_many_rows_per_cta(rows, hidden, t):
    x, w, b, dy = inputs(t, rows, hidden, 9)
    check_fwd(fwd(x, w, b), x, w, b)
    check_layer_bwd(dy, x, w)
    check_rms_bwd(dy, x, w)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(59999, 1024), (14777, 4096), (58500, 768), (7301, 5568)])
def test_rows_enough_for_two_between_barriers(rows, hidden, t):
    """Layer norm's backward pass with a dozen blocks of two rows for every CTA;
    the 64-bit reference runs on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(TYPES[t])  # noqa: E731
    x, dy, w = rand(rows, hidden) * 2 + 1, rand(rows, hidden), rand(hidden)
    _, mean, rstd = binding.layernorm_fwd_ex(x, w, stats=True)
    got = binding.layernorm_bwd_ex(dy, x, w, mean, rstd)
    want, tol = ref.layernorm_bwd(dy, x, w, mean, rstd)
    for a, b, e, n in zip(got, want, tol, ("dx", "dw", "db")):
        assert ((a.double() - b).abs() <= e).all(), n


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("with_w,with_b", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("hidden", [64, 257, 4096, 40000])
def test_without_weight_or_bias(hidden, t, with_w, with_b):
    x, w, b, dy = inputs(t, 6, hidden, 20)
    w, b = w if with_w else None, b if with_b else None
    check_fwd(fwd(x, w, b), x, w, b)
    check_layer_bwd(dy, x, w)
    check_rms_bwd(dy, x, w)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("hidden", [48, 333, 2048, 4099, 8192, 40000])
def test_rows_far_from_zero(hidden, options):
    """A mean a thousand times the spread: a variance formed as E[x^2] - E[x]^2
    in fp32 would be off by 10%."""
    x = make((7, hidden), "f32", 30, mean=1000.0)
    w, b = make((hidden,), "f32", 31, mean=1.0, std=0.1), make((hidden,), "f32", 32)
    got = fwd(x, w, b, options=options)
    check_fwd(got, x, w, b)
    var = x.double().var(-1, correction=0)
    assert ((got[2].double().cpu() ** -2 - 1e-5) / var - 1).abs().max() < 1e-4


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [64, 100, 259, 4096, 4098, 40000])
def test_constant_rows_and_bad_rows(hidden, t):
    """A constant row gives b exactly (rstd = eps^-1/2); a NaN or an infinity
    makes its own row NaN and no other."""
    x = make((6, hidden), t, 40)
    x[1] = 3.0
    x[3, hidden // 2] = float("nan")
    x[4, 0] = float("inf")
    w, b = make((hidden,), t, 41, mean=1.0), make((hidden,), t, 42)
    y, mean, rstd = fwd(x, w, b)
    torch.cuda.synchronize()
    assert (y[1].cpu() == b).all() and mean[1].item() == 3.0
    assert abs(rstd[1].item() * 1e-5 ** 0.5 - 1) < 1e-6
    assert y[3].isnan().all() and y[4].isnan().all()
    good = [0, 1, 2, 5]
    check_fwd([v[good] for v in (y, mean, rstd)], x[good], w, b)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [64, 77, 1024, 2050, 4096, 8192, 40000])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_pointers_off_a_vector_boundary(hidden, t, shift):
    """Views that start `shift` elements into a buffer; guards on both sides
    of every output stay as they were."""
    rows = 5
    x, w, b, dy = inputs(t, rows, hidden, 50)
    n = rows * hidden

    def shifted(v):
        buf = torch.full((v.numel() + 2 * shift,), 7.0, dtype=v.dtype, device="cuda")
        out = buf[shift:shift + v.numel()].view(v.shape)
        out.copy_(v)
        return buf, out

    (_, xs), (_, ws), (_, bs), (_, ds) = (shifted(v) for v in (x, w, b, dy))
    ybuf, y = shifted(torch.zeros_like(x))
    got = binding.layernorm_fwd_ex(xs, ws, bs, y=y, stats=True)
    check_fwd(got, x, w, b)
    (dxbuf, dx), (rmsbuf, dx2) = shifted(torch.zeros_like(x)), shifted(torch.zeros_like(x))
    zero = torch.zeros(hidden)
    (dwbuf, dw), (dbbuf, db) = shifted(zero), shifted(zero)
    _, mean, rstd = got
    want, tol = ref.layernorm_bwd(dy, x, w, mean.cpu(), rstd.cpu())
    out = binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd, dx=dx, dw=dw, db=db)
    for g, r, e in zip(out, want, tol):
        close(g, r, e)
    want, tol = ref.rmsnorm_bwd(dy, x, w, 1e-6)
    out = binding.rmsnorm_bwd_ex(ds, xs, ws, dx=dx2)
    for g, r, e in zip(out, want, tol):
        close(g, r, e)
    for buf, size in ((ybuf, n), (dxbuf, n), (rmsbuf, n), (dwbuf, hidden), (dbbuf, hidden)):
        assert (buf[:shift] == 7).all() and (buf[shift + size:] == 7).all()


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [64, 130, 1025, 2048, 8192, 16384, 40000])
def test_in_place(hidden, t, options):
    x, w, b, dy = inputs(t, 37, hidden, 60)
    xs, ws, bs, ds = (v.cuda() for v in (x, w, b, dy))
    y, mean, rstd = binding.layernorm_fwd_ex(xs, ws, bs, stats=True, options=options)
    over = xs.clone()
    assert binding.layernorm_fwd_ex(over, ws, bs, y=over, options=options) is over
    assert torch.equal(over, y)
    plain = binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd, options=options)
    for which in (0, 1):
        a, c = ds.clone(), xs.clone()
        got = binding.layernorm_bwd_ex(a, c, ws, mean, rstd, dx=(a, c)[which], options=options)
        for g, p in zip(got, plain):
            assert torch.equal(g, p)
    plain = binding.rmsnorm_bwd_ex(ds, xs, ws, options=options)
    for which in (0, 1):
        a, c = ds.clone(), xs.clone()
        got = binding.rmsnorm_bwd_ex(a, c, ws, dx=(a, c)[which], options=options)
        for g, p in zip(got, plain):
            assert torch.equal(g, p)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_optional_outputs_and_exact_workspace(t):
    """Gradients that are not asked for are not written; a workspace of exactly
    the stated size suffices and nothing behind it is touched."""
    x, w, _, dy = inputs(t, 100, 2048, 70)
    xs, ws, ds = x.cuda(), w.cuda(), dy.cuda()
    _, mean, rstd = binding.layernorm_fwd_ex(xs, ws, stats=True)
    full = binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd)
    size = binding.layernorm_bwd_workspace(xs)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd, workspace=room[:size])
    for g, f in zip(got, full):
        assert torch.equal(g, f)
    assert (room[size:] == 0xA5).all()
    dx, dw, db = binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd, weight_grads=False)
    assert torch.equal(dx, full[0]) and dw is None and db is None
    for name, i in (("dw", 1), ("db", 2)):
        out = torch.full((2048,), -1.0, device="cuda")
        got = binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd, weight_grads=False, **{name: out})
        assert torch.equal(got[i], full[i]) and got[3 - i] is None
    size = binding.rmsnorm_bwd_workspace(xs)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    full = binding.rmsnorm_bwd_ex(ds, xs, ws)
    got = binding.rmsnorm_bwd_ex(ds, xs, ws, workspace=room[:size])
    assert torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])
    assert (room[size:] == 0xA5).all()
    dx, dw = binding.rmsnorm_bwd_ex(ds, xs, ws, weight_grads=False)
    assert torch.equal(dx, full[0]) and dw is None
    with pytest.raises(binding.RmsnormError):
        binding.rmsnorm_bwd_ex(ds, xs, ws, workspace=room[:size - 16])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(1, 333), (9, 333), (40, 2049), (700, 1026), (5000, 97),
                                         (9, 16383), (9, 16384), (9, 16385), (9, 16391)])
def test_workspace_of_rows_of_any_length(rows, hidden, t):
    """The stated workspace suffices whatever the rows' alignment does."""
    x, w, _, dy = inputs(t, rows, hidden, 75)
    xs, ws, ds = x.cuda(), w.cuda(), dy.cuda()
    size = binding.rmsnorm_bwd_workspace(xs)
    room = torch.full((size + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    got = binding.rmsnorm_bwd_ex(ds, xs, ws, workspace=room[:size])
    want, tol = ref.rmsnorm_bwd(dy, x, w, 1e-6)
    for g, r, e in zip(got, want, tol):
        close(g, r, e)
    assert (room[size:] == 0xA5).all()


@pytest.mark.parametrize("hidden", [16385, 70001, 5000000])
def test_workspace_of_wide_rows_is_a_few_rows(hidden):
    """Few rows too wide for one CTA: a pair per row, and per column sum a row of
    fp32 for every four rows."""
    x = torch.empty((8, hidden), dtype=torch.bfloat16, device="cuda")
    parts = 2 * (hidden * 4 + 256)
    assert binding.rmsnorm_bwd_workspace(x) <= 8 * 8 + 256 + parts
    assert binding.layernorm_bwd_workspace(x) <= 8 * 8 + 256 + 2 * parts


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_no_rows(t):
    x = torch.empty((0, 3, 64), dtype=TYPES[t], device="cuda")
    w = torch.ones(64, dtype=TYPES[t], device="cuda")
    y, mean, rstd = binding.layernorm_fwd_ex(x, w, w, stats=True)
    assert y.shape == x.shape and mean.shape == (0, 3)
    dx, dw, db = binding.layernorm_bwd_ex(x, x, w, mean, rstd)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
    dx, dw = binding.rmsnorm_bwd_ex(x, x, w)
    assert dx.shape == x.shape and (dw == 0).all()


@pytest.mark.parametrize("op", ["layer", "rms"])
@pytest.mark.parametrize("hidden", [50, 2048])
def test_gradients_against_differences(op, hidden):
    """<grad, v> against (L(p + hv) - L(p - hv)) / 2h of L = sum(dy * y) in 64
    bits, for x, w and b: the difference's own error is of order h^2 = 1e-10."""
    x, w, b, dy = inputs("f32", 9, hidden, 80)
    if op == "layer":
        _, mean, rstd = fwd(x, w, b)
        got = binding.layernorm_bwd_f32(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    else:
        got = binding.rmsnorm_bwd_f32(dy.cuda(), x.cuda(), w.cuda(), eps=1e-5)

    def loss(x, w, b):
        c = x - x.mean(-1, keepdim=True) if op == "layer" else x
        y = c * ((c * c).mean(-1, keepdim=True) + 1e-5).rsqrt() * w
        return ((y + b if op == "layer" else y) * dy.double()).sum()

    point = [v.double() for v in (x, w, b)]
    for i, g in enumerate(got):
        v = make(point[i].shape, "f32", 90 + i).double()
        h = 1e-5
        there, back = list(point), list(point)
        there[i], back[i] = point[i] + h * v, point[i] - h * v
        slope = (loss(*there) - loss(*back)) / (2 * h)
        g64 = g.double().cpu()
        assert abs((g64 * v).sum() - slope) < 1e-5 * (g64 * v).abs().sum() + 1e-6


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_repeatable_on_other_streams_and_in_graphs(t):
    """Bitwise the same on a side stream, from two streams at once and replayed
    from a graph, with new inputs picked up."""
    x, w, b, dy = inputs(t, 500, 1024, 100)
    xs, ws, bs, ds = (v.cuda() for v in (x, w, b, dy))

    def step():
        y, mean, rstd = binding.layernorm_fwd_ex(xs, ws, bs, stats=True)
        return (y, *binding.layernorm_bwd_ex(ds, xs, ws, mean, rstd),
                *binding.rmsnorm_bwd_ex(ds, xs, ws))

    first = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
    torch.cuda.synchronize()
    for o in outs:
        for g, f in zip(o, first):
            assert torch.equal(g, f)
    # the stream as an argument: the kernels and the allocations are on it
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    got = binding.rmsnorm_bwd_ex(ds, xs, ws, stream=s)
    s.synchronize()
    assert torch.equal(got[0], first[4]) and torch.equal(got[1], first[5])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    for g, f in zip(held, first):
        assert torch.equal(g, f)
    xs.copy_(make(x.shape, t, 111, mean=-1.0))
    graph.replay()
    fresh = step()
    torch.cuda.synchronize()
    for g, f in zip(held, fresh):
        assert torch.equal(g, f)


def test_more_than_two_to_the_31_elements():
    """Row offsets past 32 bits: the last rows of 2^31 + 8 * 65536 elements."""
    hidden, rows = 8192, (1 << 18) + 64
    x = torch.randn((64, hidden), device="cuda").to(torch.bfloat16).repeat(rows // 64, 1)
    x[-3:] = make((3, hidden), "bf16", 120, mean=2.0).cuda()
    w = make((hidden,), "bf16", 121, mean=1.0)
    y, mean, rstd = binding.layernorm_fwd_bf16(x, w.cuda(), stats=True)
    last = x[-3:].cpu()
    check_fwd([v[-3:] for v in (y, mean, rstd)], last, w, None)
    dx, _, _ = binding.layernorm_bwd_bf16(y, x, w.cuda(), mean, rstd)
    want, tol = ref.layernorm_bwd(y[-3:].cpu(), last, w, mean[-3:].cpu(), rstd[-3:].cpu())
    close(dx[-3:], want[0], tol[0])
    dx, _ = binding.rmsnorm_bwd_bf16(y, x, w.cuda())
    want, tol = ref.rmsnorm_bwd(y[-3:].cpu(), last, w, 1e-6)
    close(dx[-3:], want[0], tol[0])


@pytest.fixture(scope="module")
def flib():
    lib = binding.open_library(build.FAULT_LIB_PATH)
    assert lib.rmsnorm_fault_injection_enabled() == 1
    return lib


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [500, 501, 2048, 8192])
@pytest.mark.parametrize("op", ["layernorm_fwd", "layernorm_bwd", "rmsnorm_bwd"])
def test_withheld_copy_ends_in_a_status(flib, op, hidden, t):
    """A staged kernel whose first copy never lands leaves after its wait's
    limit with RMSNORM_ERR_TIMEOUT in the status word; the next call is right."""
    rows = 1000
    x, w, b, dy = inputs(t, rows, hidden, 130)
    dt = binding.RMSNORM_DTYPE_F32 if t == "f32" else binding.RMSNORM_DTYPE_BF16
    xs, ws, bs, ds = (v.cuda() for v in (x, w, b, dy))
    out = torch.empty_like(xs)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = torch.empty(hidden, device="cuda"), torch.empty(hidden, device="cuda")
    room = torch.empty(binding.layernorm_bwd_workspace(xs), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call(**kw):
        o = ctypes.byref(binding.make_options(path="staged", **kw))
        p = [v.data_ptr() for v in (xs, ws, bs, ds, out, mean, rstd, dw, db, room)]
        x_, w_, b_, d_, o_, m_, r_, dw_, db_, room_ = p
        if op == "layernorm_fwd":
            return flib.layernorm_fwd_ex(dt, x_, w_, b_, o_, m_, r_, rows, hidden, 1e-5, o, stream)
        if op == "layernorm_bwd":
            return flib.layernorm_bwd_ex(dt, d_, x_, w_, m_, r_, o_, dw_, db_, rows, hidden, room_,
                                         room.numel(), o, stream)
        return flib.rmsnorm_bwd_ex(dt, d_, x_, w_, o_, dw_, rows, hidden, 1e-5, room_, room.numel(),
                                   o, stream)

    assert call(fault_inject=1, wait_timeout_ns=20_000_000) == binding.RMSNORM_OK
    assert flib.rmsnorm_last_device_status(stream) == binding.RMSNORM_ERR_TIMEOUT
    assert call() == binding.RMSNORM_OK
    assert flib.rmsnorm_last_device_status(stream) == binding.RMSNORM_OK
    if op == "layernorm_fwd":
        check_fwd((out, mean, rstd), x, w, b)
    elif op == "layernorm_bwd":
        want, tol = ref.layernorm_bwd(dy, x, w, mean.cpu(), rstd.cpu())
        for g, r, e in zip((out, dw, db), want, tol):
            close(g, r, e)
    else:
        want, tol = ref.rmsnorm_bwd(dy, x, w, 1e-5)
        for g, r, e in zip((out, dw), want, tol):
            close(g, r, e)


def test_forced_staged_path_refuses_what_it_cannot_serve():
    x, w, _, dy = inputs("f32", 3, 40000, 140)
    xs, ws, ds = x.cuda(), w.cuda(), dy.cuda()
    staged = {"path": "staged"}
    for call in (lambda: binding.layernorm_fwd_ex(xs, ws, options=staged),
                 lambda: binding.rmsnorm_bwd_ex(ds, xs, ws, options=staged)):
        with pytest.raises(binding.RmsnormError) as e:
            call()
        assert e.value.status == binding.RMSNORM_ERR_UNSUPPORTED
    off = torch.zeros(65, device="cuda")[1:].view(1, 64)
    with pytest.raises(binding.RmsnormError) as e:
        binding.layernorm_fwd_ex(off, options=staged)
    assert e.value.status == binding.RMSNORM_ERR_UNSUPPORTED
