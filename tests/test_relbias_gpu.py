"""Row softmax with a learned relative position bias, forward and backward,
against 64-bit references (GPU)."""
import pytest
import torch

import _train64 as ref
from _train64 import TYPES, Rule, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


PATHS = [None, {"path": "twopass"}]

# batch, heads, queries, keys and the rule
CASES = {
    "one": ((1, 1, 1, 1), Rule()),
    "few_keys": ((2, 3, 5, 7), Rule()),
    "square": ((2, 4, 64, 64), Rule(scale=0.125)),
    "odd": ((3, 5, 77, 333), Rule()),
    "causal": ((2, 3, 130, 130), Rule(both=False, causal=True)),
    "causal_both": ((2, 2, 40, 96), Rule(both=True, causal=True, q_offset=56)),
    "one_direction": ((1, 3, 50, 260), Rule(both=False, q_offset=100)),
    "more_queries_than_keys": ((1, 2, 90, 24), Rule(both=False, causal=True, q_offset=24 - 90)),
    "padded": ((4, 3, 33, 200), Rule(kv_len=[0, 1, 77, 200])),
    "padded_beyond": ((3, 2, 9, 50), Rule(kv_len=[-4, 60, 49])),
    "decode": ((6, 4, 1, 520), Rule(both=False, causal=True, q_start=[0, 7, 100, 519, 300, 600],
                                    kv_len=[1, 8, 101, 520, 301, 520])),
    "chunk": ((3, 2, 16, 304), Rule(both=False, causal=True, q_start=[-8, 20, 288],
                                    kv_len=[8, 36, 304])),
    "narrow_rule": ((2, 2, 30, 80), Rule(num_buckets=4, max_distance=2)),
    "two_buckets": ((1, 2, 30, 40), Rule(num_buckets=2, max_distance=2, both=False)),
    "many_buckets": ((1, 2, 300, 1000), Rule(num_buckets=256, max_distance=500)),
    "long_distance": ((1, 2, 20, 9000), Rule(num_buckets=64, max_distance=4096, q_offset=4500)),
    "long": ((2, 2, 9, 4096), Rule(q_offset=2000)),
    "longer": ((1, 2, 5, 20000), Rule(q_offset=19995)),
    "longest_odd": ((1, 1, 3, 33333), Rule(both=False, q_offset=33330, causal=True)),
    "far_queries": ((1, 2, 3, 100), Rule(q_offset=1 << 40)),
    "far_keys": ((1, 2, 3, 100), Rule(q_offset=-(1 << 40))),
    "many_rows": ((7, 2, 200, 48), Rule()),
    # windows too large for the register kernels beside several short rows
    "long_distance_few_keys": ((2, 2, 20, 64), Rule(num_buckets=64, max_distance=4096,
                                                    q_offset=3000)),
    "long_distance_decode": ((3, 2, 1, 70), Rule(num_buckets=128, max_distance=4096, both=False,
                                                 causal=True, q_start=[69, 5000, 12])),
    "many_heads": ((1, 3000, 2, 8), Rule()),
    # six vectors per thread: half a warp and a warp per row, either type
    "half_warp": ((2, 3, 20, 264), Rule(q_offset=100, kv_len=[131, 264])),
    "warp_odd": ((3, 2, 40, 601), Rule(both=False, causal=True, q_start=[561, 0, -20],
                                       kv_len=[601, 40, 597])),
    "warp_bf16": ((2, 2, 70, 1400), Rule(both=False, causal=True, q_offset=700)),
    # two warps of six vectors, many, and the widest rows that they hold
    "two_warps": ((2, 2, 21, 1400), Rule(kv_len=[1400, 900], q_offset=3)),
    "two_warps_odd": ((1, 3, 40, 2571), Rule(both=False, causal=True, q_offset=2531)),
    "many_warps": ((1, 2, 9, 6005), Rule(both=False, causal=True, q_offset=5996)),
    "widest": ((1, 2, 5, 12280), Rule(q_offset=6000)),
    "widest_bf16": ((2, 1, 3, 24560), Rule(both=False, causal=True, q_start=[24557, 9000])),
    "widest_bf16_odd": ((1, 2, 3, 20011), Rule(q_offset=19000, kv_len=[20010])),
    "warp_bf16_odd": ((2, 2, 33, 1283), Rule(q_offset=600, kv_len=[1283, 1025])),
}


def tensors(name, t, seed=1):
    shape, rule = CASES[name]
    x = make(shape, t, seed, std=2.0)
    table = make((rule.num_buckets, shape[1]), t, seed + 1)
    return x, table, make(shape, t, seed + 2), rule


def probabilities(x, table, rule):
    return ref.relbias(x, table, rule)[0].to(x.dtype)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_forward(name, t, options):
    x, table, _, rule = tensors(name, t)
    y = binding.rowsoftmax_relbias_fwd_ex(x.cuda(), table.cuda(), options=options, **rule.kwargs())
    want, tol = ref.relbias(x, table, rule)
    close(y, want, tol, name)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_backward(name, t, options):
    x, table, dy, rule = tensors(name, t)
    y = probabilities(x, table, rule)
    dx, dt = binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), rule.num_buckets,
                                               options=options, **rule.kwargs())
    want, tol = ref.relbias_bwd(dy, y, rule)
    close(dx, want[0], tol[0], f"{name} dx")
    close(dt, want[1], tol[1], f"{name} dtable")


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["padded", "causal", "decode", "chunk", "longest_odd"])
def test_nothing_is_read_at_masked_keys(name, t, options):
    """NaN and infinities there change no bit of any output."""
    x, table, dy, rule = tensors(name, t, 11)
    shape, _ = CASES[name]
    valid = rule.places(shape[0], shape[2], shape[3])[1][:, None].expand(shape)
    y = probabilities(x, table, rule)
    kw = rule.kwargs()
    clean = [binding.rowsoftmax_relbias_fwd_ex(x.cuda(), table.cuda(), options=options, **kw),
             *binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), rule.num_buckets,
                                                options=options, **kw)]
    for poison in (float("nan"), float("inf"), float("-inf")):
        xp, dp, yp = (torch.where(valid, v, torch.tensor(poison, dtype=v.dtype))
                      for v in (x, dy, y))
        got = [binding.rowsoftmax_relbias_fwd_ex(xp.cuda(), table.cuda(), options=options, **kw),
               *binding.rowsoftmax_relbias_bwd_ex(dp.cuda(), yp.cuda(), rule.num_buckets,
                                                  options=options, **kw)]
        for g, c in zip(got, clean):
            assert torch.equal(g, c)
    assert (clean[0].cpu()[~valid] == 0).all() and (clean[1].cpu()[~valid] == 0).all()


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("k", [9, 64, 700, 20000])
def test_special_scores(k, t, options):
    """Scores of the type's lowest value, -inf among others, rows of -inf,
    +inf, NaN, and rows far from zero."""
    dt = TYPES[t]
    low = torch.finfo(dt).min
    x = make((1, 2, 8, k), t, 21)
    x[:, :, 0] = low                       # uniform
    x[:, :, 1, : k // 2] = low             # the rest of the row alone
    x[:, :, 2, 1:] = float("-inf")         # one key
    x[:, :, 3] = float("-inf")             # NaN
    x[:, :, 4, k // 3] = float("nan")
    x[:, :, 5, k // 2] = float("inf")
    x[:, :, 6] += 3.0e7
    x[:, :, 7] = -low
    table = torch.zeros((32, 2), dtype=dt)
    y = binding.rowsoftmax_relbias_fwd_ex(x.cuda(), table.cuda(), options=options).cpu()
    want, tol = ref.relbias(x, table, Rule())
    assert y[:, :, [3, 4, 5]].isnan().all()
    rows = [0, 1, 2, 6, 7]
    # row 6: the scores are what they are after their own rounding, no bias is added
    close(y[:, :, rows], want[:, :, rows], tol[:, :, rows])
    assert ((y[:, :, 0].double() * k - 1).abs() < 2.0 ** -7).all()


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
def test_a_nan_stays_in_its_row(options):
    x, table, dy, rule = tensors("square", "f32", 31)
    y = probabilities(x, table, rule)
    kw = rule.kwargs()
    clean, _ = binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), 32, options=options, **kw)
    dy[1, 2, 10, 5] = float("nan")
    dx, dt = binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), 32, options=options, **kw)
    assert dx[1, 2, 10].isnan().all() and dt[:, 2].isnan().any()
    dx[1, 2, 10] = clean[1, 2, 10]
    assert torch.equal(dx, clean)
    assert not dt[:, [0, 1, 3]].isnan().any()


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["padded", "causal", "decode"])
def test_masked_keys_are_zero_in_a_nan_row(name, t, options):
    """A NaN at a row's first valid key leaves the masked keys' outputs zero,
    and the buckets that only masked keys would have reached clean."""
    x, table, dy, rule = tensors(name, t, 35)
    shape, _ = CASES[name]
    which, valid = rule.places(shape[0], shape[2], shape[3])
    y = probabilities(x, table, rule)
    x[..., 0] = dy[..., 0] = float("nan")
    kw = rule.kwargs()
    out = binding.rowsoftmax_relbias_fwd_ex(x.cuda(), table.cuda(), options=options, **kw).cpu()
    dx, dt = binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), 32, options=options, **kw)
    masked = ~valid[:, None].expand(shape)
    assert (out[masked] == 0).all() and (dx.cpu()[masked] == 0).all()
    assert out[~masked].isnan().all()
    reached = {int(b) for b in which[valid]}
    for k in range(32):
        assert dt[k].isnan().any().item() == (k in reached)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["odd", "square", "longer", "padded"])
@pytest.mark.parametrize("shift", [1, 4])
def test_pointers_off_a_vector_boundary(name, t, shift):
    x, table, dy, rule = tensors(name, t, 41)
    y = probabilities(x, table, rule)

    def shifted(v):
        buf = torch.full((v.numel() + 2 * shift,), 7.0, dtype=v.dtype, device="cuda")
        out = buf[shift:shift + v.numel()].view(v.shape)
        out.copy_(v)
        return buf, out

    kw = rule.kwargs()
    buf, out = shifted(torch.zeros_like(x))
    binding.rowsoftmax_relbias_fwd_ex(shifted(x)[1], shifted(table)[1], y=out, **kw)
    want, tol = ref.relbias(x, table, rule)
    close(out, want, tol)
    buf2, dx = shifted(torch.zeros_like(x))
    buf3, dt = shifted(torch.zeros((rule.num_buckets, x.shape[1])))
    binding.rowsoftmax_relbias_bwd_ex(shifted(dy)[1], shifted(y)[1], rule.num_buckets, dx=dx,
                                      dtable=dt, **kw)
    want, tol = ref.relbias_bwd(dy, y, rule)
    close(dx, want[0], tol[0])
    close(dt, want[1], tol[1])
    for b, v in ((buf, x), (buf2, x), (buf3, dt)):
        assert (b[:shift] == 7).all() and (b[shift + v.numel():] == 7).all()


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["square", "odd", "chunk", "longer"])
def test_in_place_and_optional_gradient(name, t, options):
    x, table, dy, rule = tensors(name, t, 51)
    kw = rule.kwargs()
    xs, ts, ds = x.cuda(), table.cuda(), dy.cuda()
    y = binding.rowsoftmax_relbias_fwd_ex(xs, ts, options=options, **kw)
    over = xs.clone()
    assert binding.rowsoftmax_relbias_fwd_ex(over, ts, y=over, options=options, **kw) is over
    assert torch.equal(over, y)
    dx, dt = binding.rowsoftmax_relbias_bwd_ex(ds, y, rule.num_buckets, options=options, **kw)
    for which in (0, 1):
        a, c = ds.clone(), y.clone()
        got = binding.rowsoftmax_relbias_bwd_ex(a, c, rule.num_buckets, dx=(a, c)[which],
                                                options=options, **kw)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dt)
    got = binding.rowsoftmax_relbias_bwd_ex(ds, y, rule.num_buckets, table_grad=False,
                                            options=options, **kw)
    assert torch.equal(got[0], dx) and got[1] is None


def test_exact_workspace():
    x, table, dy, rule = tensors("causal", "f32", 61)
    y = probabilities(x, table, rule).cuda()
    kw = rule.kwargs()
    full = binding.rowsoftmax_relbias_bwd_f32(dy.cuda(), y, 32, **kw)
    size = binding.rowsoftmax_relbias_bwd_workspace(y, 32, bidirectional=False)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = binding.rowsoftmax_relbias_bwd_f32(dy.cuda(), y, 32, workspace=room[:size], **kw)
    assert torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])
    assert (room[size:] == 0xA5).all()
    with pytest.raises(binding.RmsnormError):
        binding.rowsoftmax_relbias_bwd_f32(dy.cuda(), y, 32, workspace=room[:size - 16], **kw)


def test_no_rows():
    x = torch.empty((0, 2, 5, 8), device="cuda")
    table = torch.ones((32, 2), device="cuda")
    assert binding.rowsoftmax_relbias_fwd_f32(x, table).shape == x.shape
    dx, dt = binding.rowsoftmax_relbias_bwd_f32(x, x, 32)
    assert dx.shape == x.shape and dt.shape == (32, 2) and (dt == 0).all()


def test_gradients_against_differences():
    """<grad, v> against (L(p + hv) - L(p - hv)) / 2h of L = sum(dy * y) in 64
    bits, for the scores and the table."""
    x, table, dy, rule = tensors("causal_both", "f32", 71)
    rule.scale = 0.3
    kw = rule.kwargs()
    y = binding.rowsoftmax_relbias_fwd_f32(x.cuda(), table.cuda(), **kw)
    got = binding.rowsoftmax_relbias_bwd_f32(dy.cuda(), y, 32, **kw)

    def loss(x, table):
        return (ref.relbias(x, table, rule)[0] * dy.double()).sum()

    point = [x.double(), table.double()]
    for i, g in enumerate(got):
        v = make(point[i].shape, "f32", 80 + i).double()
        h = 1e-5
        there, back = list(point), list(point)
        there[i], back[i] = point[i] + h * v, point[i] - h * v
        slope = (loss(*there) - loss(*back)) / (2 * h)
        g64 = g.double().cpu()
        assert abs((g64 * v).sum() - slope) < 1e-5 * (g64 * v).abs().sum() + 1e-6


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_repeatable_on_other_streams_and_in_graphs(t):
    x, table, dy, rule = tensors("many_rows", t, 91)
    kw = rule.kwargs()
    xs, ts, ds = x.cuda(), table.cuda(), dy.cuda()

    def step():
        y = binding.rowsoftmax_relbias_fwd_ex(xs, ts, **kw)
        return (y, *binding.rowsoftmax_relbias_bwd_ex(ds, y, 32, **kw))

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
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    for g, f in zip(held, first):
        assert torch.equal(g, f)
    xs.copy_(make(x.shape, t, 92))
    graph.replay()
    fresh = step()
    torch.cuda.synchronize()
    for g, f in zip(held, fresh):
        assert torch.equal(g, f)


def test_offsets_past_32_bits():
    """2^31 + 2^27 scores: the last rows are right."""
    shape = (17, 32, 64, 65536)
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 20 GB")
    x = torch.randn((1, 1, 64, 65536), device="cuda").to(torch.bfloat16).expand(shape).contiguous()
    table = make((32, 32), "bf16", 101)
    rule = Rule(q_offset=65000)
    y = binding.rowsoftmax_relbias_fwd_bf16(x, table.cuda(), **rule.kwargs())
    cut = lambda v: v[-1:, -1:, -2:].cpu().contiguous()  # noqa: E731
    tail = Rule(q_offset=65062)
    want, tol = ref.relbias(cut(x), table[:, -1:], tail)
    close(cut(y), want, tol)
    dx, _ = binding.rowsoftmax_relbias_bwd_bf16(x, y, 32, **rule.kwargs())
    want, tol = ref.relbias_bwd(cut(x), cut(y), tail)
    close(cut(dx), want[0], tol[0])
