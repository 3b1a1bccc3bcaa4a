"""Rotary positions with head norms, forward and backward, against 64-bit references
(GPU)."""
import pytest
import torch

import _between64 as ref
from _between64 import Rope
from _train64 import TYPES, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

PATHS = ["auto", "twopass"]
# leading dims, heads of q and k, head_dim, rot_dim
SHAPES = [((1, 1), 1, 1, 2, 2), ((2, 3), 3, 1, 7, 4), ((3, 5), 4, 2, 64, 64), ((2, 9), 5, 3, 80, 20),
          ((1, 33), 8, 8, 96, 48), ((4, 1), 32, 8, 128, 128), ((40,), 7, 1, 128, 64),
          ((2, 17), 4, 4, 100, 50), ((1, 6), 2, 2, 192, 64), ((3, 4), 3, 3, 256, 256),
          ((1, 5), 2, 1, 320, 32), ((2, 2), 2, 1, 576, 512), ((1, 3), 1, 1, 1024, 1024),
          ((1, 3), 1, 2, 1023, 2), ((700,), 2, 1, 64, 32), ((2, 90), 40, 8, 128, 128)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def freqs_of(rot, **kw):
    f, m = binding.rmsnorm_rope_freqs(rot, device="cpu", **kw)
    return f, m


def inputs(lead, hq, hk, dim, t, norm=True, seed=1):
    v = {"q": make((*lead, hq, dim), t, seed, std=1.3), "k": make((*lead, hk, dim), t, seed + 1),
         "dq": make((*lead, hq, dim), t, seed + 2), "dk": make((*lead, hk, dim), t, seed + 3),
         "q_w": None, "k_w": None}
    if norm:
        v["q_w"] = make((dim,), t, seed + 4, mean=1.0, std=0.2)
        v["k_w"] = make((dim,), t, seed + 5, mean=1.0, std=0.2)
    return v


def on(v):
    return {k: None if t is None else t.cuda() for k, t in v.items()}


def forward(g, freqs, rule, positions=None, **kw):
    return binding.rmsnorm_rope_fwd_ex(g["q"], g["k"], freqs, positions, g["q_w"], g["k_w"],
                                       **rule.kwargs(), **kw)


def backward(g, freqs, rule, positions=None, **kw):
    x = (g["q"], g["k"]) if rule.norm else (None, None)
    return binding.rmsnorm_rope_bwd_ex(g["dq"], g["dk"], freqs, positions, *x, g["q_w"], g["k_w"],
                                       **rule.kwargs(), **kw)


def check_forward(v, rule, positions, got):
    for n, out in zip("qk", got):
        close(out, *ref.rope_fwd(v[n], v[n + "_w"], rule, positions), n)


def check_backward(v, rule, positions, got):
    for n, dx, dw in zip("qk", got[:2], got[2:]):
        want, tol = ref.rope_bwd(v["d" + n], v[n], v[n + "_w"], rule, positions)
        close(dx, want[0], tol[0], "d" + n)
        if v[n + "_w"] is None:
            assert dw is None
        else:
            close(dw, want[1], tol[1], f"d{n}_w")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("lead,hq,hk,dim,rot", SHAPES)
def test_shapes(lead, hq, hk, dim, rot, inter, norm, t, path):
    freqs, _ = freqs_of(rot)
    rule = Rope(freqs, inter, norm)
    v = inputs(lead, hq, hk, dim, t, norm)
    g, f = on(v), freqs.cuda()
    check_forward(v, rule, None, forward(g, f, rule, options={"path": path}))
    check_backward(v, rule, None, backward(g, f, rule, options={"path": path}))


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=4.0),
                                     dict(scaling="base", factor=8.0, base=5e5),
                                     dict(scaling="ramp", factor=4.0, original_len=2048),
                                     dict(scaling="bands", factor=8.0, original_len=8192, base=5e5),
                                     dict(divisors=[1.0 + i / 8 for i in range(48)])])
@pytest.mark.parametrize("t", TYPES)
def test_scalings_and_positions(t, scaling):
    """Positions per token and per sequence place, 32 and 64 bits, near and far, negative
    ones among them, and a start."""
    freqs, mscale = freqs_of(96, **scaling)
    g = torch.Generator().manual_seed(3)
    v = inputs((3, 21), 4, 2, 96, t)
    for start, positions in ((0, None), (77, None), (0, torch.randint(0, 1 << 20, (3, 21), generator=g)),
                             (-5, torch.randint(0, 1 << 31, (21,), generator=g)),
                             (1 << 40, torch.randint(-(1 << 62), 1 << 62, (3, 21), generator=g)),
                             (3, torch.randint(-100, 100, (21,), generator=g).int()),
                             (1, torch.randint(0, 1 << 30, (3, 21), generator=g).int())):
        rule = Rope(freqs, mscale=mscale, start=start)
        at = None if positions is None else positions.cuda()
        check_forward(v, rule, positions, forward(on(v), freqs.cuda(), rule, at))
        check_backward(v, rule, positions, backward(on(v), freqs.cuda(), rule, at))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_views(inter, t, path):
    """q and k inside one projection's output (also turned in place there), heads before
    tokens, heads interleaved, and outputs with strides of their own."""
    freqs, _ = freqs_of(64)
    f = freqs.cuda()
    rule = Rope(freqs, inter)
    b, s, hq, hk, d = 2, 19, 6, 2, 64
    v = inputs((b, s), hq, hk, d, t)
    want_f, want_b = forward(on(v), f, rule), backward(on(v), f, rule)

    def packed(q, k):
        a = torch.full((b, s, hq + 2 * hk + 1, d), 7.0, dtype=q.dtype, device="cuda")
        views = a[:, :, :hq], a[:, :, hq:hq + hk]
        views[0].copy_(q)
        views[1].copy_(k)
        return a, *views

    def heads_first(q, k):
        one, two = (torch.empty(b, h, s, d, dtype=q.dtype, device="cuda").transpose(1, 2)
                    for h in (hq, hk))
        one.copy_(q)
        two.copy_(k)
        return None, one, two

    def sequence_first(q, k):
        a = torch.full((s, b, hq + hk, d + 8), 7.0, dtype=q.dtype, device="cuda")
        views = a[:, :, :hq, 8:].transpose(0, 1), a[:, :, hq:, 8:].transpose(0, 1)
        views[0].copy_(q)
        views[1].copy_(k)
        return a, *views

    for lay in (packed, heads_first, sequence_first):
        whole, q, k = lay(v["q"].cuda(), v["k"].cuda())
        g = dict(on(v), q=q, k=k)
        got = forward(g, f, rule, options={"path": path})
        assert got[0].is_contiguous() and got[1].is_contiguous()
        check_forward(v, rule, None, got)
        _, dq, dk = lay(v["dq"].cuda(), v["dk"].cuda())
        check_backward(v, rule, None, backward(dict(g, dq=dq, dk=dk), f, rule, options={"path": path}))
        # outputs laid out the same way
        _, oq, ok = lay(torch.zeros_like(v["q"]).cuda(), torch.zeros_like(v["k"]).cuda())
        forward(g, f, rule, q_out=oq, k_out=ok, options={"path": path})
        assert torch.equal(oq, got[0]) and torch.equal(ok, got[1])
        # in place; what lies around the heads stays
        before = None if whole is None else whole.clone()
        forward(g, f, rule, q_out=q, k_out=k, options={"path": path})
        assert torch.equal(q, got[0]) and torch.equal(k, got[1])
        if whole is not None:
            q.fill_(7.0)
            k.fill_(7.0)
            rest = lay(torch.full_like(v["q"], 7.0).cuda(), torch.full_like(v["k"], 7.0).cuda())[0]
            before_rest = before.clone()
            assert torch.equal(whole, rest) and before_rest.shape == rest.shape
    for t1, t2 in zip(want_f, forward(on(v), f, rule)):
        assert torch.equal(t1, t2)
    # the gradient over dy, and over x
    for which in ("d", ""):
        g = on(v)
        got = backward(g, f, rule, dq_in=g[which + "q"], dk_in=g[which + "k"], options={"path": "auto"})
        for a, c in zip(got, want_b):
            assert torch.equal(a, c)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("by", [1, 2, 3, 4])
@pytest.mark.parametrize("dim,rot", [(16, 8), (32, 32), (64, 64), (128, 32)])
def test_pointers_off_the_boundaries(dim, rot, by, t):
    """q, k, the gradients, the outputs and the weights off the 16-byte boundaries, heads and
    tokens some elements apart; what lies between them stays."""
    freqs, _ = freqs_of(rot)
    f = freqs.cuda()
    for inter in (False, True):
        for norm in (True, False):
            rule = Rope(freqs, inter, norm, start=9)
            v = inputs((2, 11), 3, 2, dim, t, norm)

            def off(a):
                if a is None:
                    return None
                if a.dim() == 1:
                    return torch.empty(dim + 8, dtype=a.dtype, device="cuda")[by:by + dim].copy_(a)
                room = torch.full((*a.shape[:-1], dim + by), 7.0, dtype=a.dtype, device="cuda")
                return room[..., by:].copy_(a)

            g = {n: off(a) for n, a in v.items()}
            outs = [off(torch.zeros_like(v[n])) for n in "qk"]
            got = forward(g, f, rule, q_out=outs[0], k_out=outs[1])
            check_forward(v, rule, None, got)
            check_backward(v, rule, None, backward(g, f, rule, dq_in=outs[0], dk_in=outs[1]))
            for o in outs:
                whole = o.as_strided((*o.shape[:-1], dim + by), o.stride(), o.storage_offset() - by)
                assert (whole[..., :by] == 7.0).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lead,hq,hk,dim", [((1,), 300, 3, 64), ((3,), 1, 70, 128), ((5000,), 1, 1, 64),
                                            ((2, 3), 129, 129, 32), ((800,), 3, 1, 256)])
def test_many_heads_and_few(lead, hq, hk, dim, t):
    freqs, _ = freqs_of(dim)
    rule = Rope(freqs)
    v = inputs(lead, hq, hk, dim, t)
    g = on(v)
    check_forward(v, rule, None, forward(g, freqs.cuda(), rule))
    check_backward(v, rule, None, backward(g, freqs.cuda(), rule))


def test_refused_in_python():
    """Arguments that the binding refuses before the library is called."""
    freqs, _ = freqs_of(32)
    f = freqs.cuda()
    q, k, w = (make(s, "f32", 1).cuda() for s in ((2, 6, 4, 64), (2, 6, 2, 64), (64,)))
    fwd = lambda *a, **kw: binding.rmsnorm_rope_fwd_f32(*a, **kw)  # noqa: E731
    for a, kw in (((q[..., ::2], None, f), {}), ((q, k[:, :5], f), {}), ((q, k.double(), f), {}),
                  ((q, k.cpu(), f), {}), ((q, k, f.int()), {}), ((q, k, f.cpu()), {}), ((q, k, f[:0]), {}),
                  ((q[0, 0], None, f), {}), ((q[..., :16], None, f), {}), ((q, k, f[::2]), {}),
                  ((q, k, f, torch.arange(5, device="cuda")), {}), ((q, k, f, torch.arange(6)), {}),
                  ((q, k, f, torch.arange(6.0, device="cuda")), {}),
                  ((q, k, f, torch.arange(12, device="cuda")[::2]), {}), ((q, k, f, None, w[:32]), {}),
                  ((q, None, f, None, None, w), {}), ((q, k, f, None, w), dict(norm=False)),
                  ((q, None, f), dict(k_out=k)), ((q, k, f), dict(q_out=k)), ((q, k, f), dict(start=2 ** 63))):
        with pytest.raises((ValueError, TypeError)):
            fwd(*a, **kw)
    for kw in (dict(mscale=1e300), dict(eps=-1.0)):      # not a finite fp32 number, for one
        with pytest.raises((ValueError, binding.RmsnormError)):
            fwd(q, k, f, **kw)
    with pytest.raises(binding.RmsnormError):            # an output over half of its input
        a = torch.zeros(2, 6, 6, 64, device="cuda")
        fwd(a[:, :, :4], None, f, q_out=a[:, :, 2:])
    with pytest.raises(binding.RmsnormError):            # an output that lies over itself
        fwd(q, k, f, q_out=torch.zeros(2, 6, 1, 64, device="cuda").expand(2, 6, 4, 64))
    bwd = lambda *a, **kw: binding.rmsnorm_rope_bwd_f32(*a, **kw)  # noqa: E731
    for a, kw in (((q, k, f, None, q), {}), ((q, k, f, None, q, k[:1]), {}), ((q, None, f, None, q, k), {}),
                  ((q, k, f), dict(q_w=w)), ((q, k, f), dict(dq_w=w)), ((q, None, f), dict(dk_in=k)),
                  ((q, k, f, None, q, k), dict(dq_w=w[:32])), ((q, k, f, None, q, k, w, w), dict(dk_in=q))):
        with pytest.raises((ValueError, TypeError)):
            bwd(*a, **kw)


@pytest.mark.parametrize("t", TYPES)
def test_expanded_inputs_and_q_alone(t):
    """Inputs whose strides are zero (one gradient for every head), and no k."""
    freqs, _ = freqs_of(32)
    rule = Rope(freqs)
    v = inputs((2, 6), 4, 4, 32, t)
    one = v["dq"][:, :, :1].expand(2, 6, 4, 32)
    v["dq"] = one
    g = on(v)
    g["dq"] = v["dq"][:, :, :1].cuda().expand(2, 6, 4, 32)
    assert g["dq"].stride(2) == 0
    check_backward(v, rule, None, backward(g, freqs.cuda(), rule))
    both = forward(g, freqs.cuda(), rule)
    q, k = binding.rmsnorm_rope_fwd_ex(g["q"], None, freqs.cuda(), None, g["q_w"], **rule.kwargs())
    assert k is None and torch.equal(q, both[0])
    got = binding.rmsnorm_rope_bwd_ex(g["dq"], None, freqs.cuda(), None, g["q"], None, g["q_w"],
                                      **rule.kwargs())
    assert got[1] is None and got[3] is None
    # tokens without a batch: the same numbers
    flat = {n: None if a is None else a.flatten(0, 1) if a.dim() == 4 else a for n, a in v.items()}
    at = torch.arange(6).repeat(2)
    check_forward(flat, rule, at, forward(on(flat), freqs.cuda(), rule, at.cuda()))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,rot", [(64, 32), (128, 128), (50, 20)])
def test_special_heads(dim, rot, t, path):
    """A head with NaN or infinity changes no other; without the norm only its own pair.
    A head of zeros is zero, with eps = 0 NaN."""
    freqs, _ = freqs_of(rot)
    f = freqs.cuda()
    keep = torch.ones(2, 5, 3, dtype=torch.bool)
    keep[1, 2, 1] = False
    for norm in (True, False):
        rule = Rope(freqs, False, norm)
        v = inputs((2, 5), 3, 3, dim, t, norm)
        want_f = forward(on(v), f, rule, options={"path": path})
        want_b = backward(on(v), f, rule, options={"path": path})
        for value in (float("nan"), float("inf")):
            for at in (0, rot - 1, dim - 1):
                w = {n: None if a is None else a.clone() for n, a in v.items()}
                w["q"][1, 2, 1, at] = value
                w["dq"][1, 2, 1, at] = value
                got = forward(on(w), f, rule, options={"path": path})
                assert torch.equal(got[0][keep], want_f[0][keep]) and torch.equal(got[1], want_f[1])
                assert not got[0][1, 2, 1, at].isfinite()
                back = backward(on(w), f, rule, options={"path": path})
                assert torch.equal(back[0][keep], want_b[0][keep]) and torch.equal(back[1], want_b[1])
                if not norm:
                    mates = {at} if at >= rot else {at, (at + rot // 2) % rot}
                    for a in (got[0], back[0]):
                        bad = set((~a[1, 2, 1].isfinite()).nonzero().flatten().tolist())
                        assert bad <= mates and at in bad
    rule = Rope(freqs, eps=0.0)
    v = inputs((2, 5), 3, 3, dim, t)
    v["q"][1, 2, 1] = 0
    got = forward(on(v), f, rule, options={"path": path})
    assert got[0][1, 2, 1].isnan().all() and got[0][keep].isfinite().all()
    assert not forward(on(v), f, Rope(freqs), options={"path": path})[0][1, 2, 1].any()


@pytest.mark.parametrize("t", TYPES)
def test_no_tokens(t):
    freqs, _ = freqs_of(64)
    rule = Rope(freqs)
    for lead in ((0, 7), (3, 0), (0,)):
        g = on(inputs(lead, 4, 2, 64, t))
        got = forward(g, freqs.cuda(), rule)
        assert got[0].shape == (*lead, 4, 64)
        back = backward(g, freqs.cuda(), rule)
        assert back[0].shape == (*lead, 4, 64) and not back[2].any() and not back[3].any()


def test_against_differences():
    """The directional derivative of sum(dq q' + dk k'), by differences in 64 bits."""
    freqs, mscale = freqs_of(24, scaling="ramp", factor=4.0, original_len=512)
    rule = Rope(freqs, True, mscale=mscale, start=100)
    v = inputs((2, 7), 3, 2, 40, "f32")
    got = backward(on(v), freqs.cuda(), rule)
    wide = {k: a.double() for k, a in v.items()}

    def loss(**kw):
        w = {**wide, **kw}
        return sum((wide["d" + n] * ref.rope_fwd(w[n], w[n + "_w"], rule, None)[0]).sum()
                   for n in "qk").item()

    for name, d in zip(("q", "k", "q_w", "k_w"), got):
        way = make(v[name].shape, "f32", 31).double()
        slope = (loss(**{name: wide[name] + 1e-5 * way})
                 - loss(**{name: wide[name] - 1e-5 * way})) / 2e-5
        dot, size = ((d.cpu().double() * way).sum().item(), (d.cpu().double() * way).norm().item())
        # the kernel's own 1e-5 of its terms, differences 1e-10 * third derivatives
        assert abs(dot - slope) <= 1e-4 * size + 1e-6, name


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_turned_back(inter, t):
    """Without the norm the backward pass undoes the forward pass."""
    freqs, _ = freqs_of(128)
    rule = Rope(freqs, inter, norm=False, start=123456)
    v = inputs((2, 50), 4, 2, 128, t, norm=False)
    g = on(v)
    q, k = forward(g, freqs.cuda(), rule)
    back = backward(dict(g, dq=q, dk=k), freqs.cuda(), rule)
    for n, out in zip("qk", back[:2]):
        x = v[n].double()
        pairs = rule.pairs(x)
        size = rule.joined(*[pairs[0].abs() + pairs[1].abs()] * 2, x)
        # turned twice, rounded twice
        tol = 2 * size * (ref.TURN * 2 + 2 * ref.half_step(v[n].dtype))
        close(out, x, tol, n)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("tokens", [3, 4000])
def test_repeatable_and_any_workspace(tokens, t):
    freqs, _ = freqs_of(64)
    f = freqs.cuda()
    rule = Rope(freqs)
    g = on(inputs((tokens,), 5, 2, 64, t))
    size = binding.rmsnorm_rope_bwd_workspace(g["q"], g["k"])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for a, b in zip(backward(g, f, rule), backward(g, f, rule, workspace=ws)):
        assert torch.equal(a, b)
    with pytest.raises(binding.RmsnormError):
        backward(g, f, rule, workspace=ws[:size - 16])
    part = backward(g, f, rule, weight_grads=False)
    assert part[2] is None and part[3] is None
    dw = torch.empty(64, device="cuda")
    part = backward(g, f, rule, weight_grads=False, dk_w=dw)
    assert part[2] is None and torch.equal(part[3], backward(g, f, rule)[3])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim", [64, 1023])
def test_gradients_without_weights_and_the_workspace(dim, t):
    """dq_w of ones, if it is given, and nothing written behind the workspace."""
    freqs, _ = freqs_of(32)
    f = freqs.cuda()
    rule = Rope(freqs)
    v = inputs((3, 700), 5, 2, dim, t)
    v["q_w"] = None
    g = on(v)
    size = binding.rmsnorm_rope_bwd_workspace(g["q"], g["k"])
    room = torch.full((size + (1 << 20),), 77, dtype=torch.uint8, device="cuda")
    dw = torch.empty(dim, device="cuda")
    got = backward(g, f, rule, workspace=room[:size], dq_w=dw)
    assert (room[size:] == 77).all() and got[2] is dw
    want, tol = ref.rope_bwd(v["dq"], v["q"], None, rule, None)
    close(dw, want[1], tol[1], "dq_w")
    close(got[0], want[0], tol[0], "dq")
    assert backward(g, f, rule)[2] is None


def test_offsets_beyond_32_bits():
    """The last tokens of arrays of more than 2^31 elements."""
    freqs, _ = freqs_of(128)
    heads, last = 32, 2
    tokens = 2 ** 31 // (heads * 128) + 7
    rule = Rope(freqs, start=5)
    v = inputs((last,), heads, 1, 128, "bf16")
    big = {}
    for n in ("q", "dq"):
        big[n] = torch.ones((tokens, heads, 128), dtype=torch.bfloat16, device="cuda")
        big[n][-last:] = v[n].cuda()
    at = torch.arange(tokens, device="cuda")
    out, _ = binding.rmsnorm_rope_fwd_bf16(big["q"], None, freqs.cuda(), at, v["q_w"].cuda(),
                                           **rule.kwargs())
    close(out[-last:], *ref.rope_fwd(v["q"], v["q_w"], rule, at[-last:].cpu()), "q")
    got = binding.rmsnorm_rope_bwd_bf16(big["dq"], None, freqs.cuda(), at, big["q"], None,
                                        v["q_w"].cuda(), dq_in=out, **rule.kwargs())
    want, tol = ref.rope_bwd(v["dq"], v["q"], v["q_w"], rule, at[-last:].cpu())
    close(got[0][-last:], want[0], tol[0], "dq")
