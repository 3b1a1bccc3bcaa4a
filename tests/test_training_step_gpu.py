"""The training operators used together (GPU): an attention block in its pre-norm
form, forward and backward, with layer norm, the softmax with a relative position
bias and RMSNorm from the library and plain matrix products in between."""
import threading

import pytest
import torch

import _train64 as ref
from _train64 import TYPES, Rule, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

BATCH, HEADS, SEQ, DIM = 3, 4, 71, 16
HIDDEN = HEADS * DIM
EPS = 1e-5
RULES = {
    # an encoder: padded keys, one sequence empty
    "padded": Rule(kv_len=[71, 30, 0], scale=DIM ** -0.5),
    # a decoder: causal, sequences of two lengths
    "causal": Rule(both=False, causal=True, kv_len=[71, 50, 71], scale=DIM ** -0.5),
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def values(t, seed=1):
    """Inputs, parameters (both differentiated) and fixed matrices, on the CPU."""
    p = {"x": make((BATCH, SEQ, HIDDEN), t, seed, mean=0.2),
         "w1": make((HIDDEN,), t, seed + 1, mean=1.0, std=0.1),
         "b1": make((HIDDEN,), t, seed + 2, std=0.1),
         "table": make((32, HEADS), t, seed + 3, std=0.5),
         "w2": make((HIDDEN,), t, seed + 4, mean=1.0, std=0.1)}
    fixed = {"qkv": make((HIDDEN, 3 * HIDDEN), t, seed + 5, std=HIDDEN ** -0.5),
             "out": make((HIDDEN, HIDDEN), t, seed + 6, std=HIDDEN ** -0.5),
             "dy": make((BATCH, SEQ, HIDDEN), t, seed + 7)}
    return p, fixed


def split(v):
    return v.unflatten(-1, (HEADS, DIM)).transpose(1, 2)


def joined(v):
    return v.transpose(1, 2).flatten(2)


def product(how, a, b):
    """A product in 64 bits, rounded to the operands' type."""
    return torch.einsum(how, a.double(), b.double()).to(a.dtype).contiguous()


def step(p, fixed, kw):
    """Forward and backward on the GPU: y and the gradients of p."""
    x = p["x"]
    n, mean, rstd = binding.layernorm_fwd_ex(x, p["w1"], p["b1"], eps=EPS, stats=True)
    q, k, v = (split(c) for c in product("bsi,io->bso", n, fixed["qkv"]).chunk(3, -1))
    s = product("bhid,bhjd->bhij", q, k)
    a = binding.rowsoftmax_relbias_fwd_ex(s, p["table"], **kw)
    o = joined(product("bhij,bhjd->bhid", a, v))
    r = x + product("bsi,io->bso", o, fixed["out"])
    norm = binding.rmsnorm_fwd_f32 if x.dtype == torch.float32 else binding.rmsnorm_fwd_bf16
    y = norm(r, p["w2"], eps=EPS)

    dr, dw2 = binding.rmsnorm_bwd_ex(fixed["dy"], r, p["w2"], eps=EPS)
    do = split(product("bso,io->bsi", dr, fixed["out"]))
    da, dv = product("bhid,bhjd->bhij", do, v), product("bhij,bhid->bhjd", a, do)
    ds, dtable = binding.rowsoftmax_relbias_bwd_ex(da, a, 32, **kw)
    dq, dk = product("bhij,bhjd->bhid", ds, k), product("bhij,bhid->bhjd", ds, q)
    dn = product("bso,io->bsi", torch.cat([joined(g) for g in (dq, dk, dv)], -1), fixed["qkv"])
    dx, dw1, db1 = binding.layernorm_bwd_ex(dn, x, p["w1"], mean, rstd)
    return {"y": y, "x": dr + dx, "w1": dw1, "b1": db1, "table": dtable, "w2": dw2}


def loss(p, fixed, rule):
    """sum(dy * y) in 64 bits."""
    n = ref.layernorm(p["x"], p["w1"], p["b1"], EPS)[0][0]
    q, k, v = (split(c) for c in torch.einsum("bsi,io->bso", n, fixed["qkv"]).chunk(3, -1))
    a = ref.relbias(torch.einsum("bhid,bhjd->bhij", q, k), p["table"], rule)[0]
    o = joined(torch.einsum("bhij,bhjd->bhid", a, v))
    r = p["x"] + torch.einsum("bsi,io->bso", o, fixed["out"])
    y = r * (r * r).mean(-1, keepdim=True).add(EPS).rsqrt() * p["w2"]
    return (fixed["dy"] * y).sum(), y


def on_gpu(v):
    return {n: t.cuda() for n, t in v.items()}


@pytest.mark.parametrize("name", RULES)
def test_gradients_of_the_block_against_differences(name):
    """<grad, v> against (L(p + hv) - L(p - hv)) / 2h in 64 bits, one parameter at
    a time.  Allowed: the steps between a parameter's gradient and the loss are at
    most twelve (six forward, six backward), each rounds to fp32 and is off by at
    most K * 2^-24 = 1e-5 of its terms, and the fixed matrices have norm about 1 (a
    factor of at most 4 each, once forward and once backward): 12 * 16 * 1e-5 of
    the terms' norm; the differences themselves are off by about h^2."""
    rule = RULES[name]
    p, fixed = values("f32")
    got = {n: g.double().cpu() for n, g in step(on_gpu(p), on_gpu(fixed), rule.kwargs()).items()}
    p64, f64 = ({n: t.double() for n, t in d.items()} for d in (p, fixed))
    y = loss(p64, f64, rule)[1]
    assert (got["y"] - y).abs().max() <= 6 * 16 * 1e-5 * y.abs().max()
    h = 1e-5
    for i, n in enumerate(p):
        v = make(p[n].shape, "f32", 50 + i).double()
        slope = (loss({**p64, n: p64[n] + h * v}, f64, rule)[0]
                 - loss({**p64, n: p64[n] - h * v}, f64, rule)[0]) / (2 * h)
        terms = (got[n] * v).norm()
        assert abs((got[n] * v).sum() - slope) <= 12 * 16 * 1e-5 * terms + 1e-5, n


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("name", RULES)
def test_block_in_a_graph(name, t):
    """A captured step, replayed on other values and beside eager steps on another
    stream, gives what the eager step gives, bit for bit."""
    kw = RULES[name].kwargs()
    p, fixed = (on_gpu(v) for v in values(t))
    step(p, fixed, kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(p, fixed, kw)
    side = torch.cuda.Stream()
    for seed in (1, 21):
        fresh = on_gpu(values(t, seed)[0])
        for n in p:
            p[n].copy_(fresh[n])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            beside = step(fresh, fixed, kw)
        want = step(fresh, fixed, kw)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(held[n], want[n]), n
            assert torch.equal(beside[n], want[n]), n


def test_two_threads_at_once():
    """Steps from two host threads, a stream each, give what one thread gives."""
    kw = RULES["padded"].kwargs()
    p, fixed = (on_gpu(v) for v in values("bf16"))
    want = step(p, fixed, kw)
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [step(p, fixed, kw) for _ in range(20)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for outs in got.values():
        for o in outs:
            for n in want:
                assert torch.equal(o[n], want[n]), n


@pytest.mark.parametrize("t", TYPES)
def test_streams_given_as_handles(t):
    """stream= as a torch stream, as its handle, and 0 for the default one."""
    x, w = make((40, 96), t, 1).cuda(), make((96,), t, 2).cuda()
    s, table = make((2, 3, 20, 40), t, 3).cuda(), make((32, 3), t, 4).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def all_of(stream):
        y, mean, rstd = binding.layernorm_fwd_ex(x, w, stats=True, stream=stream)
        a = binding.rowsoftmax_relbias_fwd_ex(s, table, stream=stream)
        return (y, *binding.layernorm_bwd_ex(y, x, w, mean, rstd, stream=stream),
                *binding.rmsnorm_bwd_ex(y, x, w, stream=stream), a,
                *binding.rowsoftmax_relbias_bwd_ex(s, a, 32, stream=stream))

    want = all_of(None)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        got = all_of(stream)
        torch.cuda.synchronize()
        for g, f in zip(got, want):
            assert torch.equal(g, f)
