"""Edges of the training operators (GPU): eps = 0 and rows that leave a block
part empty, values whose squares are near the smallest float, constant rows,
the widths at which a path ends."""
import pytest
import torch

import _train64 as ref
from _train64 import TYPES, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

PATHS = [None, {"path": "twopass"}]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def rms_bwd(dy, x, w, eps, options=None):
    got = binding.rmsnorm_bwd_ex(*(None if v is None else v.cuda() for v in (dy, x, w)), eps=eps,
                                 options=options)
    want, tol = ref.rmsnorm_bwd(dy, x, w, eps)
    for g, r, e, n in zip(got, want, tol, ("dx", "dw")):
        close(g, r, e, f"{n} of {tuple(x.shape)}")


def layer_bwd(dy, x, w, options=None):
    _, mean, rstd = ref.layernorm(x, w, None, 1e-5)[0]
    mean, rstd = mean.float(), rstd.float()
    got = binding.layernorm_bwd_ex(*(None if v is None else v.cuda() for v in (dy, x, w, mean, rstd)),
                                   options=options)
    want, tol = ref.layernorm_bwd(dy, x, w, mean, rstd)
    for g, r, e, n in zip(got, want, tol, ("dx", "dw", "db")):
        close(g, r, e, f"{n} of {tuple(x.shape)}")


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hidden", [16, 64, 333, 512, 768, 1001, 2048, 2050, 4096, 5120, 8192, 8200])
def test_rmsnorm_backward_with_eps_zero(hidden, t, options):
    """The rows that a block lacks add nothing to dw, although their sum of
    squares is 0."""
    for rows in (1, 2, 3, 4, 5, 7, 8, 9, 13, 16, 17):
        x, dy = make((rows, hidden), t, rows, std=2.0), make((rows, hidden), t, rows + 50)
        rms_bwd(dy, x, make((hidden,), t, 3, mean=1.0, std=0.1), 0.0, options)
        if rows == 3:
            rms_bwd(dy, x, None, 0.0, options)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hidden", [64, 333, 2048, 4096, 8200])
def test_rows_whose_squares_are_tiny(hidden, t, options):
    """x of order 2^-62 and eps = 0: rstd is 2^62 and its square times the row's
    m(g * xh), here about 40, is past fp32; dx, at most 2^62 * 200, is not."""
    rows, w = 37, make((hidden,), t, 1, mean=1.0, std=0.1)
    x = make((rows, hidden), "f32", 2)
    dy = (40 * x + make((rows, hidden), "f32", 3)).to(TYPES[t])
    x = (x * 2.0 ** -62).to(TYPES[t])
    rms_bwd(dy, x, w, 0.0, options)
    _, mean, rstd = ref.layernorm(x, w, None, 0.0)[0]
    mean, rstd = mean.float(), rstd.float()
    got = binding.layernorm_bwd_ex(*(v.cuda() for v in (dy, x, w, mean, rstd)), options=options)
    want, tol = ref.layernorm_bwd(dy, x, w, mean, rstd)
    for g, r, e, n in zip(got, want, tol, ("dx", "dw", "db")):
        close(g, r, e, n)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hidden", [8196, 8200, 8201, 9000, 11001, 12288, 14400, 16383, 16384])
def test_wide_rows_in_one_pass(hidden, t):
    """Rows of more than 8192 elements: threads that lack their last vector and
    that fill theirs, rows off the 16-byte boundaries, with and without weights."""
    x, w, dy = make((7, hidden), t, 1, mean=0.5), make((hidden,), t, 2), make((7, hidden), t, 3)
    for weights in (w, None):
        rms_bwd(dy, x, weights, 1e-6)
        layer_bwd(dy, x, weights)


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hidden", [109, 448, 896, 1792, 3584, 7168])
def test_constant_rows_at_widths_without_a_reciprocal(hidden, t, options):
    """The mean of a constant row is the constant where its sum is exact, also at
    widths whose fp32 reciprocal times the sum is not: the row gives b."""
    w, b = make((hidden,), t, 1, mean=1.0), make((hidden,), t, 2)
    x = torch.tensor([3.0, -1000.0, 0.0, 60416.0, 1.5])[:, None].repeat(1, hidden).to(TYPES[t])
    y, mean, rstd = binding.layernorm_fwd_ex(x.cuda(), w.cuda(), b.cuda(), stats=True,
                                             options=options)
    assert (mean.cpu() == x[:, 0].float()).all()
    assert (y.cpu() == b).all()
    assert (rstd * 1e-5 ** 0.5 - 1).abs().max() < 1e-6


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("hidden", [48, 448, 3584])
def test_mean_of_a_row_with_an_infinity(hidden, options):
    x = make((4, hidden), "f32", 5)
    x[1, 7], x[2, 9] = float("inf"), float("-inf")
    _, mean, rstd = binding.layernorm_fwd_ex(x.cuda(), stats=True, options=options)
    assert rstd[1:3].isnan().all() and rstd[0].isfinite() and rstd[3].isfinite()
    if options is None:
        assert mean[1].item() == float("inf") and mean[2].item() == float("-inf")


@pytest.mark.parametrize("options", PATHS, ids=["auto", "twopass"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hidden", [8, 109, 448, 4096, 7168, 40000])
def test_constant_rows_whose_square_is_past_fp32(hidden, t, options):
    """Threads without an element of the row, whose mean of nothing is 0, change
    nothing."""
    w, b = make((hidden,), t, 1, mean=1.0), make((hidden,), t, 2)
    x = torch.tensor([2.0 ** 100, -2.0 ** 90, 1.0])[:, None].repeat(1, hidden).to(TYPES[t])
    y, mean, rstd = binding.layernorm_fwd_ex(x.cuda(), w.cuda(), b.cuda(), stats=True,
                                             options=options)
    assert (mean.cpu() == x[:, 0].float()).all()
    assert (y.cpu() == b).all()
    assert (rstd * 1e-5 ** 0.5 - 1).abs().max() < 1e-6


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("buckets,distance", [(32, 128), (64, 500), (128, 4096)])
@pytest.mark.parametrize("keys", [1, 8, 16, 31, 32, 64, 100])
def test_relbias_backward_of_many_short_rows(keys, buckets, distance, t):
    """Several rows to a warp, which add to its windows of sums in turn; the
    register kernel also where the automatic choice reads such rows twice."""
    shape = (3, 2, 150, keys)
    rule = ref.Rule(buckets, distance, scale=0.5, q_start=[0, -20, 4000],
                    kv_len=[keys, max(0, keys - 3), keys])
    x, table = make(shape, t, 1), make((buckets, 2), t, 2)
    y, dy = ref.relbias(x, table, rule)[0].to(TYPES[t]), make(shape, t, 3)
    want, tol = ref.relbias_bwd(dy, y, rule)
    for options in (None, {"path": "rowreg"}, {"path": "twopass"}):
        got, again = (binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), buckets,
                                                        options=options, **rule.kwargs())
                      for _ in range(2))
        for g, a, r, e, n in zip(got, again, want, tol, ("dx", "dtable")):
            close(g, r, e, n)
            assert torch.equal(g, a), n


@pytest.mark.parametrize("t", TYPES)
def test_relbias_backward_folds_windows_of_many_short_rows(t):
    """A CTA with more short rows than it sums before it folds its windows."""
    shape, rule = (1, 304, 5000, 8), ref.Rule(64, 500, q_start=[-2500])
    x, table = make(shape, t, 1), make((64, 304), t, 2)
    y, dy = ref.relbias(x, table, rule)[0].to(TYPES[t]), make(shape, t, 3)
    want, tol = ref.relbias_bwd(dy, y, rule)
    got = binding.rowsoftmax_relbias_bwd_ex(dy.cuda(), y.cuda(), 64, **rule.kwargs())
    for g, r, e, n in zip(got, want, tol, ("dx", "dtable")):
        close(g, r, e, n)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("keys", [1, 8, 32, 64])
def test_relbias_backward_of_short_rows_in_registers(keys, t):
    """The register kernel takes them whatever the size of the windows."""
    y = torch.rand((2, 2, 9, keys), device="cuda").to(TYPES[t])
    for buckets, distance in ((32, 128), (64, 500), (256, 500), (256, 4096)):
        binding.rowsoftmax_relbias_bwd_ex(y, y, buckets, max_distance=distance,
                                          options={"path": "rowreg"})


def staged_norm_bwd(name, t, hidden):
    """Whether the one-pass kernel of a backward pass takes rows of this length."""
    x = torch.ones((2, hidden), dtype=TYPES[t], device="cuda")
    stats = [torch.zeros(2, device="cuda"), torch.ones(2, device="cuda")]
    args = [x, x, None] + (stats if name == "layernorm_bwd_ex" else [])
    try:
        getattr(binding, name)(*args, options={"path": "staged"})
    except binding.RmsnormError as e:
        assert e.status == binding.RMSNORM_ERR_UNSUPPORTED
        return False
    return True


@pytest.mark.parametrize("name", ["layernorm_bwd_ex", "rmsnorm_bwd_ex"])
def test_widest_rows_of_the_one_pass_backward_kernel(name):
    """Two blocks of x and dy, of a row each, and off the 16-byte boundaries the
    weights beside them, must fit a CTA's shared memory: in fp32 rows of 14400
    elements, and of 11517 (2880 vectors that they touch); in both types none above
    16384."""
    for t, hidden, fits in (("f32", 14400, True), ("f32", 14404, False), ("f32", 16384, False),
                            ("f32", 11517, True), ("f32", 11518, False),
                            ("bf16", 16384, True), ("bf16", 16383, True), ("bf16", 16392, False)):
        assert staged_norm_bwd(name, t, hidden) == fits, (t, hidden)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("with_w", [True, False])
@pytest.mark.parametrize("hidden,groups", [(1024, 4), (4096, 1), (768, 4), (5568, 1)])
def test_a_dozen_blocks_of_two_rows_for_every_cta(hidden, groups, with_w, t):
    """Layer norm's backward pass with enough rows, on any number of SMs, for two
    rows between barriers (CTAs of `groups` rows, at most four to an SM and fewer
    for wide rows); the 64-bit reference runs on the GPU."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 12 * 2 * groups * sms * min(4, 16384 // hidden) + 11
    g = torch.Generator(device="cuda").manual_seed(hidden)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(TYPES[t])  # noqa: E731
    x, dy, w = rand(rows, hidden) * 2 + 1, rand(rows, hidden), rand(hidden) if with_w else None
    _, mean, rstd = binding.layernorm_fwd_ex(x, w, stats=True)
    got = binding.layernorm_bwd_ex(dy, x, w, mean, rstd)
    if w is None:
        w = torch.ones(hidden, device="cuda")
    want, tol = ref.layernorm_bwd(dy, x, w, mean, rstd)
    for a, b, e, n in zip(got, want, tol, ("dx", "dw", "db")):
        assert ((a.double() - b).abs() <= e).all(), n
