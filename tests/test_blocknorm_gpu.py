"""The block boundary (norms, gate, residual scales), forward and backward, against
64-bit references (GPU)."""
import itertools

import pytest
import torch

import _between64 as ref
from _between64 import Block
from _train64 import TYPES, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

PATHS = ["auto", "twopass"]
# leading dims and width: from one element to wide rows, off every boundary among them
SHAPES = [((1,), 1), ((3,), 7), ((2, 3), 64), ((33,), 130), ((5, 4), 256), ((3, 37), 514),
          ((300,), 96), ((2, 65), 1024), ((17,), 2050), ((3, 8), 3584), ((64,), 4096), ((9,), 8192),
          ((5,), 9001), ((4,), 16384), ((3,), 16391), ((2,), 70001), ((2,), 131072)]
RULES = {"both": Block(), "scaled": Block(rs=0.75, bs=-1.5), "post": Block(pre=False, bs=0.5),
         "pre": Block(post=False, rs=2.0), "none": Block(post=False, pre=False, rs=0.25, bs=3.0)}
GATES = ["none", "channel", "sequence", "element"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def inputs(lead, n, t, rule, gate="none", weights=True, seed=1):
    """x, residual, h, dy, dh, post_w, pre_w, gate on the CPU; what a rule lacks is None."""
    shape = (*lead, n)
    v = {"x": make(shape, t, seed, mean=0.1, std=0.7), "residual": make(shape, t, seed + 1, std=1.5),
         "h": make(shape, t, seed + 2, mean=-0.2, std=1.2), "dy": None,
         "dh": make(shape, t, seed + 4), "post_w": None, "pre_w": None, "gate": None}
    if rule.pre:
        v["dy"] = make(shape, t, seed + 3)
    if weights:
        if rule.post:
            v["post_w"] = make((n,), t, seed + 5, mean=1.0, std=0.2)
        if rule.pre:
            v["pre_w"] = make((n,), t, seed + 6, mean=1.0, std=0.2)
    if gate != "none":
        lead_g = {"channel": (), "sequence": lead[:1], "element": lead}[gate]
        v["gate"] = make((*lead_g, n), t, seed + 7, mean=0.4, std=0.5)
    return v


def on(v):
    return {k: None if t is None else t.cuda() for k, t in v.items()}


def forward(g, rule, **kw):
    return binding.rmsnorm_block_fwd_ex(g["x"], g["residual"], g["post_w"], g["pre_w"], g["gate"],
                                        **rule.kwargs(), **kw)


def backward(g, rule, **kw):
    return binding.rmsnorm_block_bwd_ex(g["dy"], g["dh"], g["x"], g["h"], g["post_w"], g["pre_w"],
                                        g["gate"], **rule.kwargs(), **kw)


def check(names, got, want, tol):
    for n, a, b, c in zip(names, got, want, tol):
        assert (a is None) == (b is None), n
        if b is not None:
            close(a, b, c, n)


def check_forward(v, rule, got):
    check(("h", "y"), got, *ref.block_fwd(v["x"], v["residual"], v["post_w"], v["pre_w"], v["gate"],
                                          rule))


BWD = ("dx", "dresidual", "dpost_w", "dpre_w", "dgate")


def check_backward(v, rule, got):
    check(BWD, got, *ref.block_bwd(v["dy"], v["dh"], v["x"], v["h"], v["post_w"], v["pre_w"],
                                   v["gate"], rule))


def same(a, b):
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert torch.equal(x.isnan(), y.isnan())
            assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead,n", SHAPES)
def test_forward_shapes(lead, n, t, path):
    for rule, gate in (("both", "none"), ("scaled", "channel"), ("pre", "sequence")):
        v = inputs(lead, n, t, RULES[rule], gate)
        check_forward(v, RULES[rule], forward(on(v), RULES[rule], options={"path": path}))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead,n", SHAPES)
def test_backward_shapes(lead, n, t, path):
    for rule, gate in (("both", "none"), ("scaled", "channel"), ("scaled", "sequence")):
        v = inputs(lead, n, t, RULES[rule], gate)
        check_backward(v, RULES[rule], backward(on(v), RULES[rule], options={"path": path}))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("rule", RULES)
def test_every_rule(rule, gate, t, path):
    for lead, n, weights in (((5, 13), 192, True), ((3, 11), 1030, False), ((2, 9), 2048, True)):
        v = inputs(lead, n, t, RULES[rule], gate, weights)
        g = on(v)
        check_forward(v, RULES[rule], forward(g, RULES[rule], options={"path": path}))
        check_backward(v, RULES[rule], backward(g, RULES[rule], options={"path": path}))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead", [(700,), (7, 300), (1000, 3), (1, 1), (4, 1), (3000, 1)])
def test_gates_of_many_lengths(lead, t, path):
    """Gate rows of one to many rows: more gate rows than CTAs, more CTAs than gate rows."""
    rule = RULES["scaled"]
    for n, gate in ((128, "sequence"), (520, "sequence"), (128, "element"), (264, "channel")):
        v = inputs(lead, n, t, rule, gate)
        check_backward(v, rule, backward(on(v), rule, options={"path": path}))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("cluster", [2, 4, 8, 16])
@pytest.mark.parametrize("n", [136, 1024, 4104, 16384, 65536, 131072])
def test_rows_over_a_cluster(n, cluster, t):
    """Forced splits, uneven ones among them, agree with the references, several blocks of
    rows to a cluster; what cannot be split so is refused."""
    options = {"path": "staged", "cluster": cluster}
    v = inputs((3, 5), n, t, RULES["scaled"], "sequence")
    g = on(v)
    per = -(-n * v["x"].element_size() // 16 // cluster)
    threads = -(-per // 2)
    vectors = n * v["x"].element_size() // 16
    for run, check_it, most in ((forward, check_forward, 1024), (backward, check_backward, 512)):
        if threads > most or (cluster - 1) * per >= vectors:
            with pytest.raises(binding.RmsnormError) as e:
                run(g, RULES["scaled"], options=options)
            assert e.value.status == binding.RMSNORM_ERR_UNSUPPORTED
            continue
        check_it(v, RULES["scaled"], run(g, RULES["scaled"], options=options))
    if n == 1024:
        for rule in RULES.values():
            v = inputs((301, 3), n, t, rule, "sequence")
            check_forward(v, rule, forward(on(v), rule, options=options))
            check_backward(v, rule, backward(on(v), rule, options=options))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("cluster,n", [(0, 64), (0, 512), (0, 2048), (2, 136), (2, 1024), (4, 1024),
                                       (0, 66), (0, 1030)])
def test_nothing_behind_the_workspace(cluster, n, t):
    """More units of work than there are parts for: the workspace is left as it was behind its
    size, and the sums are right."""
    rule = RULES["scaled"]
    options = {"path": "staged", "cluster": cluster} if cluster else None
    for gate in ("channel", "sequence"):
        v = inputs((60, 50), n, t, rule, gate)
        g = on(v)
        size = binding.rmsnorm_block_bwd_workspace(g["x"], g["gate"])
        room = torch.full((size + (1 << 22),), 77, dtype=torch.uint8, device="cuda")
        got = backward(g, rule, workspace=room[:size], options=options)
        assert (room[size:] == 77).all()
        check_backward(v, rule, got)


def test_refused_in_python():
    """Arguments that the binding refuses before the library is called."""
    x, r, w = (make(s, "f32", 1).cuda() for s in ((4, 6, 64), (4, 6, 64), (64,)))
    fwd, bwd = binding.rmsnorm_block_fwd_f32, binding.rmsnorm_block_bwd_f32
    for a, kw in (((x.transpose(0, 1), r), {}), ((x, r[:3]), {}), ((x, r.double()), {}), ((x, r.cpu()), {}),
                  ((x, r, w[:32]), {}), ((x, r, w, w.cpu()), {}), ((x, r, w), dict(post_norm=False)),
                  ((x, r, None, w), dict(pre_norm=False)), ((x, r), dict(y=x, pre_norm=False)),
                  ((x, r), dict(h=x[:2])), ((x, r, w, w, w[:32]), {}), ((x, r, w, w, x[:, :3]), {}),
                  ((x, r, w, w, x[:3, :1].contiguous()), {}), ((x, r, w, w, x[:1].contiguous()), {}),
                  ((x, r, w, w, x[:, 0].expand(1, 4, 64).contiguous()), {}),
                  ((x.bfloat16(), r), {})):
        with pytest.raises((ValueError, TypeError)):
            fwd(*a, **kw)
    for a, kw in (((None, r, x, x), {}), ((x, r, x, None), {}), ((x, r, x, x), dict(pre_norm=False)),
                  ((x, r[:2], x, x), {}), ((x, r, x, x), dict(dgate=w)), ((x, r, x, x), dict(dpost_w=w.double())),
                  ((None, r, x, None), dict(pre_norm=False, dpre_w=w)),
                  ((x, r, x, x), dict(post_norm=False, dpost_w=w)), ((x, r, x, x), dict(dx=x[0])),
                  ((x, r, x, x, w), dict(workspace=torch.empty(8, dtype=torch.uint8)))):
        with pytest.raises((ValueError, TypeError)):
            bwd(*a, **kw)
    for kw in (dict(residual_scale=float("nan")), dict(post_eps=-1.0), dict(h=x, y=x),
               dict(branch_scale=1e300)):
        with pytest.raises((ValueError, binding.RmsnormError)):
            fwd(x, r, w, w, **kw)


@pytest.mark.parametrize("t", TYPES)
def test_gate_shapes(t):
    """[hidden], [1, hidden], [batch, hidden], [batch, 1, hidden], [batch, seq, hidden]."""
    rule = RULES["scaled"]
    v = inputs((4, 6), 96, t, rule)
    for shape in ((96,), (1, 96), (1, 1, 96), (4, 96), (4, 1, 96), (4, 6, 96)):
        v["gate"] = make(shape, t, 9, mean=0.4)
        wide = v["gate"] if len(shape) != 2 or shape[0] != 4 else v["gate"][:, None]
        r = dict(v, gate=wide)
        check_forward(r, rule, forward(on(v), rule))
        got = backward(on(v), rule)
        assert got[4].shape == shape
        want, tol = ref.block_bwd(*(r[k] for k in ("dy", "dh", "x", "h", "post_w", "pre_w", "gate")),
                                  rule)
        close(got[4], want[4].reshape(shape), tol[4].reshape(shape), "dgate")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
def test_unaligned_pointers(t, path):
    """Every array off the 16-byte boundaries by its own number of elements."""
    rule = RULES["scaled"]
    v = inputs((3, 21), 1024, t, rule, "sequence")
    g = {}
    for i, (k, a) in enumerate(v.items()):
        if a is None:
            g[k] = None
            continue
        room = torch.empty(a.numel() + 16, dtype=a.dtype, device="cuda")
        g[k] = room[1 + i % 8:1 + i % 8 + a.numel()].view(a.shape)
        g[k].copy_(a)
    out = [torch.empty(v["x"].numel() + 16, dtype=v["x"].dtype, device="cuda")[3:3 + v["x"].numel()]
           .view(v["x"].shape) for _ in range(2)]
    check_forward(v, rule, forward(g, rule, h=out[0], y=out[1], options={"path": path}))
    check_backward(v, rule, backward(g, rule, dx=out[0], dresidual=out[1], options={"path": path}))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead,n", [((3, 21), 1024), ((400,), 72), ((5, 7), 2051), ((2,), 3), ((1,), 5),
                                    ((2000,), 33), ((3, 100), 1030), ((7,), 4095), ((4, 3), 6004)])
def test_weights_and_outputs_off_the_boundaries(lead, n, t):
    """Inputs on their boundaries, the weights, the gate and the outputs not; ragged rows,
    the arrays' last bytes among them."""
    rule = RULES["scaled"]
    for by in (1, 2, 4):
        for gate in ("sequence", "channel"):
            v = inputs(lead, n, t, rule, gate, seed=by)
            g = on(v)
            off = lambda a: torch.empty(a.numel() + 16, dtype=a.dtype, device="cuda")[by:by + a.numel()].view(a.shape)  # noqa: E731
            for k in ("post_w", "pre_w", "gate"):
                g[k] = off(v[k]).copy_(v[k])
            one, two = off(v["x"]), off(v["x"])
            check_forward(v, rule, forward(g, rule, h=one, y=two))
            check_backward(v, rule, backward(g, rule, dx=one, dresidual=two))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead,n", [((7,), 1), ((40, 50), 3), ((9, 5), 259), ((1000,), 514),
                                    ((500,), 2050), ((300,), 4095), ((200,), 8191), ((3, 70), 12002),
                                    ((5,), 16391)])
def test_rows_in_registers(lead, n, t):
    """Rows of short vectors held in registers, several to a CTA one after the other."""
    for rule, gate in (("scaled", "sequence"), ("post", "channel"), ("pre", "none"), ("none", "element")):
        v = inputs(lead, n, t, RULES[rule], gate)
        g = on(v)
        options = {"path": "rowreg"}
        if n == 16391:                      # more vectors than a CTA holds
            with pytest.raises(binding.RmsnormError) as e:
                forward(g, RULES[rule], options=options)
            assert e.value.status == binding.RMSNORM_ERR_UNSUPPORTED
            continue
        check_forward(v, RULES[rule], forward(g, RULES[rule], options=options))
        where = dict(h=g["residual"], y=g["x"]) if RULES[rule].pre else dict(h=g["residual"])
        check_forward(v, RULES[rule], forward(g, RULES[rule], options=options, **where))
    with pytest.raises(binding.RmsnormError):
        g = on(inputs((3,), 64, t, RULES["both"]))
        forward(g, RULES["both"], options={"path": "rowreg"})


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [5, 33, 1027, 2050, 4097, 6004])
def test_nothing_behind_the_arrays(n, t):
    """Arrays that end where their memory does hold NaN from there on: nothing of it is
    used, and nothing there is written."""
    rule = RULES["scaled"]
    v = inputs((3, 3), n, t, rule, "channel")
    rooms = {}
    g = {}
    for k, a in v.items():
        rooms[k] = torch.full((a.numel() + 64,), float("nan"), dtype=a.dtype, device="cuda")
        g[k] = rooms[k][:a.numel()].view(a.shape)
        g[k].copy_(a)
    outs = [torch.full((v["x"].numel() + 64,), 7.0, dtype=v["x"].dtype, device="cuda") for _ in range(2)]
    one, two = (o[:v["x"].numel()].view(v["x"].shape) for o in outs)
    check_forward(v, rule, forward(g, rule, h=one, y=two))
    check_backward(v, rule, backward(g, rule, dx=one, dresidual=two))
    for o in outs:
        assert (o[v["x"].numel():] == 7.0).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [64, 1030, 4096, 9001, 16384])
def test_in_place(n, t, path):
    """Every input that an output may be written over gives the same bits."""
    rule = RULES["scaled"]
    v = inputs((3, 5), n, t, rule, "sequence")
    want = forward(on(v), rule, options={"path": path})
    for h, y in itertools.permutations(("x", "residual", None), 2):
        g = on(v)
        same(want, forward(g, rule, h=g.get(h), y=g.get(y), options={"path": path}))
    want = backward(on(v), rule, options={"path": path})
    for dx, dr in itertools.permutations(("dy", "dh", "x", "h", None), 2):
        g = on(v)
        same(want, backward(g, rule, dx=g.get(dx), dresidual=g.get(dr), options={"path": path}))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
def test_without_dh_and_without_gradients(t, path):
    rule = RULES["both"]
    v = inputs((6, 10), 768, t, rule, "sequence")
    g = on(v)
    full = backward(g, rule, options={"path": path})
    for kw in (dict(weight_grads=False), dict(weight_grads=False, dgate=torch.empty(6, 768, device="cuda")),
               dict(weight_grads=False, dpre_w=torch.empty(768, device="cuda")),
               dict(weight_grads=False, dpost_w=torch.empty(768, device="cuda"))):
        got = backward(g, rule, options={"path": path}, **kw)
        for n, a, b in zip(BWD, got, full):
            assert (a is None) == (n not in kw and n not in ("dx", "dresidual"))
            if a is not None:
                assert torch.equal(a, b), n
    v["dh"] = None
    check_backward(v, rule, backward(on(v), rule, options={"path": path}))
    none = Block(post=False, pre=False, bs=2.0)
    v["dy"] = None
    got = backward({**on(v), "post_w": None, "pre_w": None, "dh": None}, none,
                   options={"path": path})
    assert not got[0].any() and not got[1].any() and not got[4].any()


@pytest.mark.parametrize("t", TYPES)
def test_no_rows(t):
    for rule in RULES.values():
        g = on(inputs((0, 5), 40, t, rule, "channel"))
        h, y = forward(g, rule)
        assert h.shape == (0, 5, 40) and (y is None) == (not rule.pre)
        got = backward(g, rule)
        assert got[0].shape == (0, 5, 40)
        for d in got[2:]:
            assert d is None or (d.shape == (40,) and not d.any())
    g = on(inputs((0, 5), 40, t, RULES["both"], "sequence"))
    assert backward(g, RULES["both"])[4].shape == (0, 40)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [64, 2048, 2050])
def test_special_rows(n, t, path):
    """A row with NaN or infinity changes no other row; rows of zeros with eps = 0 are NaN
    as the definition has it (h is not: the branch of zeros is NaN only where it is
    normed), with eps > 0 they are zeros."""
    rule = RULES["scaled"]
    v = inputs((9,), n, t, rule, "channel")
    clean = on(v)
    want_f, want_b = forward(clean, rule, options={"path": path}), backward(clean, rule, options={"path": path})
    for name, value in itertools.product(("x", "residual", "h", "dy", "dh"),
                                         (float("nan"), float("inf"), float("-inf"))):
        w = dict(v)
        w[name] = v[name].clone()
        w[name][4, n // 2] = value
        g = on(w)
        keep = [0, 1, 2, 3, 5, 6, 7, 8]
        if name in ("x", "residual"):
            got = forward(g, rule, options={"path": path})
            for a, b in zip(got, want_f):
                assert torch.equal(a[keep], b[keep]), name
            assert not got[1][4].isfinite().any() or value != value or (got[1][4] == 0).sum() >= n - 1
            assert not got[1][4, n // 2].isfinite()
        if name != "residual":
            got = backward(g, rule, options={"path": path})
            for a, b in zip(got[:2], want_b[:2]):
                assert torch.equal(a[keep], b[keep]), name
            assert not got[1][4, n // 2].isfinite() or name == "x"
            if name == "x":
                assert torch.equal(got[1], want_b[1])       # dresidual does not read x
    zero = Block(post_eps=0.0, pre_eps=0.0)
    g = on(v)
    g["x"][2], g["residual"][3] = 0, 0
    h, y = forward(g, zero, options={"path": path})
    assert h[2].isnan().all() and y[2].isnan().all()
    assert h[[0, 1, 3, 4, 5]].isfinite().all() and y[[0, 1, 3, 4, 5]].isfinite().all()
    g["residual"][2] = 0
    h, y = forward(g, rule, options={"path": path})
    assert not h[2].any() and not y[2].any()
    got = backward(dict(g, gate=None), zero, options={"path": path})
    assert got[0][2].isnan().all() and got[1].isfinite().all()
    assert got[3].isfinite().all() and got[2].isnan().all()


@pytest.mark.parametrize("path", PATHS)
def test_infinite_branch_without_its_norm(path):
    """Without the norm x is only a factor of dgate: an infinity in it leaves dx finite."""
    rule = RULES["pre"]
    v = inputs((9,), 640, "f32", rule, "channel")
    v["x"][3, 100] = float("inf")
    got = backward(on(v), rule, options={"path": path})
    assert got[0].isfinite().all() and got[1].isfinite().all()
    assert not got[4][100].isfinite() and got[4][:100].isfinite().all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale", [1e-18, 1e-16, 1e15])
def test_tiny_and_large_rows(scale, path):
    """Rows whose squares are near fp32's smallest and largest numbers, eps = 0: the
    formulas scale with them.  Squares of 1e-18 are whole in fp32 to 2^-24 of their sum only
    above 2^-126 = 1e-38: scale^2 = 1e-36 keeps them normal."""
    rule = Block(post_eps=0.0, pre_eps=0.0)
    v = inputs((7,), 1152, "f32", rule, "channel")
    v["x"] = (v["x"] * scale).float()
    v["h"] = (v["h"] * scale).float()
    # gradients that the small rows' large factors leave in range
    v["dy"], v["dh"] = v["dy"] * min(1.0, scale), v["dh"]
    check_backward(v, rule, backward(on(v), rule, options={"path": path}))
    v["residual"] = (v["residual"] * scale).float()
    low = Block(post_eps=0.0, pre_eps=0.0, bs=1.0)
    check_forward(v, low, forward(on(v), low, options={"path": path}))


@pytest.mark.parametrize("path", PATHS)
def test_branch_that_takes_the_residual_back(path):
    """residual = -branch but for little: the sum of squares is of what is left, not a
    difference of large sums."""
    rule = Block(post=False, pre_eps=0.0)
    v = inputs((7,), 2048, "f32", rule)
    v["residual"] = -v["x"] * (1 + 2.0 ** -12 * make((7, 2048), "f32", 77).sign())
    check_forward(v, rule, forward(on(v), rule, options={"path": path}))


@pytest.mark.parametrize("t", TYPES)
def test_against_differences(t):
    """The directional derivative of sum(dy y + dh h), by differences in 64 bits."""
    rule = RULES["scaled"]
    v = inputs((3, 5), 48, "f32", rule, "sequence")
    out = ref.block_fwd(v["x"], v["residual"], v["post_w"], v["pre_w"], v["gate"], rule)[0]
    v["h"] = out[0].float()
    got = backward(on(v), rule)
    wide = {k: a.double() for k, a in v.items()}

    def loss(**kw):
        w = {**wide, **kw}
        h, y = ref.block_fwd(w["x"], w["residual"], w["post_w"], w["pre_w"], w["gate"], rule)[0]
        return ((wide["dy"] * y).sum() + (wide["dh"] * h).sum()).item()

    step = 1e-5
    for name, d in zip(("x", "residual", "post_w", "pre_w", "gate"), got):
        way = make(v[name].shape, "f32", 31).double()
        slope = (loss(**{name: wide[name] + step * way})
                 - loss(**{name: wide[name] - step * way})) / (2 * step)
        dot = (d.cpu().double() * way).sum().item()
        size = (d.cpu().double() * way).norm().item()
        # h was rounded to fp32 (u of values of order one, through second derivatives of the
        # order of one), the kernel's own 1e-5 of its terms, differences 1e-10 * third ones
        assert abs(dot - slope) <= 1e-4 * size + 1e-5, name


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead,n,gate", [((4, 700), 1024, "sequence"), ((2000,), 130, "channel"),
                                         ((60,), 16384, "none"), ((3, 50), 2050, "element")])
def test_repeatable_and_any_workspace(lead, n, gate, t):
    rule = RULES["scaled"]
    g = on(inputs(lead, n, t, rule, gate))
    size = binding.rmsnorm_block_bwd_workspace(g["x"], g["gate"])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    first, again = backward(g, rule), backward(g, rule, workspace=ws)
    same(first, again)
    same(forward(g, rule), forward(g, rule))
    with pytest.raises(binding.RmsnormError):
        backward(g, rule, workspace=ws[:size - 16])


def test_offsets_beyond_32_bits():
    """The last rows of arrays of more than 2^31 elements."""
    n, rule = 8192, RULES["both"]
    rows = 2 ** 31 // n + 5
    last = 3
    v = inputs((last,), n, "bf16", rule)
    big = {}
    for k in ("x", "residual", "h", "dy", "dh"):
        big[k] = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
        big[k][-last:] = v[k].cuda()
        if k != "dy":
            big[k][:-last] = 1
    big.update({k: v[k].cuda() for k in ("post_w", "pre_w")}, gate=None)
    h, y = forward(big, rule)
    check_forward(v, rule, (h[-last:], y[-last:]))
    del h, y
    got = backward(big, rule)
    want, tol = ref.block_bwd(v["dy"], v["dh"], v["x"], v["h"], v["post_w"], v["pre_w"], None, rule)
    for i in (0, 1):
        close(got[i][-last:], want[i], tol[i], BWD[i])
    close(got[3], want[3], tol[3], "dpre_w")         # dy is zero elsewhere
