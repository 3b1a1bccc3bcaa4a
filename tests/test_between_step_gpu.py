"""The block boundary and the rotary positions used together (GPU): an attention block with
head norms and rotary positions on the queries and keys inside the projection's output,
and the boundary behind it (norm, a gate for each sequence, residual scales, the next
block's norm), forward and backward, with plain matrix products in between."""
import threading

import pytest
import torch

import _between64 as ref
from _between64 import Block, Rope
from _train64 import TYPES, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

BATCH, SEQ, HEADS, KV, DIM = 2, 37, 4, 2, 16
HIDDEN = HEADS * DIM
EPS = 1e-5
RULE = Block(rs=0.875, bs=0.5, post_eps=EPS, pre_eps=EPS)
NAMES = ("x", "w0", "q_w", "k_w", "post_w", "pre_w", "gate")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def rope_rule():
    freqs, mscale = binding.rmsnorm_rope_freqs(DIM, scaling="ramp", factor=4.0, original_len=512,
                                               device="cpu")
    return freqs, Rope(freqs, mscale=mscale, eps=EPS, start=3)


def values(t, seed=1):
    """Inputs and parameters (differentiated), and fixed matrices and gradients, on the CPU."""
    near_one = dict(mean=1.0, std=0.1)
    p = {"x": make((BATCH, SEQ, HIDDEN), t, seed, mean=0.2), "w0": make((HIDDEN,), t, seed + 1, **near_one),
         "q_w": make((DIM,), t, seed + 2, **near_one), "k_w": make((DIM,), t, seed + 3, **near_one),
         "post_w": make((HIDDEN,), t, seed + 4, **near_one),
         "pre_w": make((HIDDEN,), t, seed + 5, **near_one),
         "gate": make((BATCH, HIDDEN), t, seed + 6, mean=0.5, std=0.2)}
    fixed = {"qkv": make((HIDDEN, (HEADS + 2 * KV) * DIM), t, seed + 7, std=HIDDEN ** -0.5),
             "out": make((HIDDEN, HIDDEN), t, seed + 8, std=HIDDEN ** -0.5),
             "dy": make((BATCH, SEQ, HIDDEN), t, seed + 9), "dh": make((BATCH, SEQ, HIDDEN), t, seed + 10)}
    return p, fixed


def product(how, a, b):
    """A product in 64 bits, rounded to the operands' type."""
    return torch.einsum(how, a.double(), b.double()).to(a.dtype).contiguous()


def many(v):
    """Each key head beside the query heads that share it."""
    return v.repeat_interleave(HEADS // KV, 2)


def step(p, fixed, freqs, rule, stream=None):
    """Forward and backward on the GPU: h, y and the gradients of p."""
    x = p["x"]
    how = dict(stream=stream)
    norm = binding.rmsnorm_fwd_f32 if x.dtype == torch.float32 else binding.rmsnorm_fwd_bf16
    n = norm(x, p["w0"], eps=EPS, **how)
    qkv = product("bsi,io->bso", n, fixed["qkv"]).unflatten(-1, (HEADS + 2 * KV, DIM))
    q, k, v = qkv.split((HEADS, KV, KV), 2)
    at = torch.arange(SEQ, device=x.device)
    tq, tk = binding.rmsnorm_rope_fwd_ex(q, k, freqs, at, p["q_w"], p["k_w"], **rule.kwargs(), **how)
    s = product("bihd,bjhd->bhij", tq, many(tk)) * DIM ** -0.5
    a = binding.rowsoftmax_fwd_ex(s.contiguous(), **how)
    o = product("bhij,bjhd->bihd", a, many(v)).flatten(2)
    branch = product("bsi,io->bso", o, fixed["out"])
    h, y = binding.rmsnorm_block_fwd_ex(branch, x, p["post_w"], p["pre_w"], p["gate"], **RULE.kwargs(),
                                        **how)

    db, dres, dpost, dpre, dgate = binding.rmsnorm_block_bwd_ex(
        fixed["dy"], fixed["dh"], branch, h, p["post_w"], p["pre_w"], p["gate"], **RULE.kwargs(), **how)
    do = product("bso,io->bsi", db, fixed["out"]).unflatten(-1, (HEADS, DIM))
    da, dv = product("bihd,bjhd->bhij", do, many(v)), product("bhij,bihd->bjhd", a, do)
    ds = (a.double() * (da.double() - (a.double() * da.double()).sum(-1, keepdim=True))
          * DIM ** -0.5).to(x.dtype)
    dtq, dtk = product("bhij,bjhd->bihd", ds, many(tk)), product("bhij,bihd->bjhd", ds, tq)
    fold = lambda g: g.unflatten(2, (KV, HEADS // KV)).double().sum(3).to(x.dtype)  # noqa: E731
    # written into the gradient of the projection's output, where q and k lie
    dqkv = torch.empty_like(qkv)
    dq, dk, dvs = dqkv.split((HEADS, KV, KV), 2)
    dvs.copy_(fold(dv))
    _, _, dq_w, dk_w = binding.rmsnorm_rope_bwd_ex(dtq, fold(dtk), freqs, at, q, k, p["q_w"], p["k_w"],
                                                   dq_in=dq, dk_in=dk, **rule.kwargs(), **how)
    dn = product("bso,io->bsi", dqkv.flatten(2), fixed["qkv"])
    dx, dw0 = binding.rmsnorm_bwd_ex(dn, x, p["w0"], eps=EPS, **how)
    return {"h": h, "y": y, "x": dres + dx, "w0": dw0, "q_w": dq_w, "k_w": dk_w, "post_w": dpost,
            "pre_w": dpre, "gate": dgate}


def loss(p, fixed, rule):
    """sum(dy y + dh h) in 64 bits, and y."""
    x = p["x"]
    n = x * ref.norm_factor(x, EPS) * p["w0"]
    q, k, v = torch.einsum("bsi,io->bso", n, fixed["qkv"]).unflatten(-1, (HEADS + 2 * KV, DIM)) \
        .split((HEADS, KV, KV), 2)
    q, k = (ref.rope_fwd(t, p[w], rule, None)[0] for t, w in ((q, "q_w"), (k, "k_w")))
    a = (torch.einsum("bihd,bjhd->bhij", q, many(k)) * DIM ** -0.5).softmax(-1)
    o = torch.einsum("bhij,bjhd->bihd", a, many(v)).flatten(2)
    (h, y), _ = ref.block_fwd(torch.einsum("bsi,io->bso", o, fixed["out"]), x, p["post_w"], p["pre_w"],
                              p["gate"], RULE)
    return (fixed["dy"] * y).sum() + (fixed["dh"] * h).sum(), y


def on_gpu(v):
    return {n: t.cuda() for n, t in v.items()}


def test_gradients_of_the_block_against_differences():
    """<grad, v> against (L(p + hv) - L(p - hv)) / 2h in 64 bits, one parameter at a time.
    Allowed: the steps between a parameter's gradient and the loss are at most sixteen (eight
    forward, eight backward), each rounds to fp32 and is off by at most 1e-5 of its terms
    (chains of 160 additions at 2^-24), and the fixed matrices have norm about 1 (a factor
    of at most 4 each, once forward and once backward): 16 * 16 * 1e-5 of the terms'
    norm; the differences themselves are off by about h^2."""
    freqs, rule = rope_rule()
    p, fixed = values("f32")
    got = {n: g.double().cpu() for n, g in step(on_gpu(p), on_gpu(fixed), freqs.cuda(), rule).items()}
    p64, f64 = ({n: t.double() for n, t in d.items()} for d in (p, fixed))
    y = loss(p64, f64, rule)[1]
    assert (got["y"] - y).abs().max() <= 8 * 16 * 1e-5 * y.abs().max()
    h = 1e-5
    for i, n in enumerate(NAMES):
        v = make(p[n].shape, "f32", 50 + i).double()
        slope = (loss({**p64, n: p64[n] + h * v}, f64, rule)[0]
                 - loss({**p64, n: p64[n] - h * v}, f64, rule)[0]) / (2 * h)
        terms = (got[n] * v).norm()
        assert abs((got[n] * v).sum() - slope) <= 16 * 16 * 1e-5 * terms + 1e-5, n


@pytest.mark.parametrize("t", TYPES)
def test_block_in_a_graph(t):
    """A captured step, replayed on other values and beside eager steps on another stream,
    gives what the eager step gives, bit for bit."""
    freqs, rule = rope_rule()
    f = freqs.cuda()
    p, fixed = (on_gpu(v) for v in values(t))
    step(p, fixed, f, rule)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(p, fixed, f, rule)
    with torch.cuda.graph(second):
        other = step(p, fixed, f, rule)
    side = torch.cuda.Stream()
    for seed in (1, 21):
        fresh = on_gpu(values(t, seed)[0])
        for n in p:
            p[n].copy_(fresh[n])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            second.replay()                    # two captured steps at once, workspaces of their own
            beside = step(fresh, fixed, f, rule)
        want = step(fresh, fixed, f, rule)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(held[n], want[n]), n
            assert torch.equal(other[n], want[n]), n
            assert torch.equal(beside[n], want[n]), n


def test_two_threads_at_once():
    """Steps from two host threads, a stream each, give what one thread gives."""
    freqs, rule = rope_rule()
    f = freqs.cuda()
    p, fixed = (on_gpu(v) for v in values("bf16"))
    want = step(p, fixed, f, rule)
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [step(p, fixed, f, rule) for _ in range(10)]
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
    freqs, rule = rope_rule()
    f = freqs.cuda()
    x, r, w = (make(s, t, i).cuda() for i, s in enumerate(((40, 96), (40, 96), (96,))))
    q, k = make((40, 4, DIM), t, 7).cuda(), make((40, 2, DIM), t, 8).cuda()
    qw = make((DIM,), t, 9).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def all_of(stream):
        h, y = binding.rmsnorm_block_fwd_ex(x, r, w, w, stream=stream)
        a = binding.rmsnorm_block_bwd_ex(y, r, x, h, w, w, stream=stream)
        tq, tk = binding.rmsnorm_rope_fwd_ex(q, k, f, None, qw, qw, stream=stream)
        b = binding.rmsnorm_rope_bwd_ex(tq, tk, f, None, q, k, qw, qw, stream=stream)
        return [h, y, *(g for g in a if g is not None), tq, tk, *b]

    want = all_of(None)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        got = all_of(stream)
        torch.cuda.synchronize()
        for g, e in zip(got, want):
            assert torch.equal(g, e)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [192, 1030, 4096, 16384])
def test_back_to_back(n, t):
    """A chain of dependent calls, each of which may start before the one before it has
    ended, gives what synchronised calls give."""
    freqs, _ = binding.rmsnorm_rope_freqs(64, device="cuda")
    rows = 60
    r, w = make((rows, n), t, 2).cuda(), make((n,), t, 3, mean=1.0, std=0.1).cuda()
    q0 = make((rows, 6, 64), t, 4).cuda()
    qw = make((64,), t, 5, mean=1.0, std=0.1).cuda()

    def chain(sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        x, q, out = make((rows, n), t, 1).cuda(), q0.clone(), []
        for _ in range(6):
            h, y = binding.rmsnorm_block_fwd_ex(x, r, w, w, w)
            wait()
            dx, dr, *sums = binding.rmsnorm_block_bwd_ex(y, h, x, h, w, w, w)
            wait()
            q, k = binding.rmsnorm_rope_fwd_ex(q, q, freqs, None, qw, qw)
            wait()
            dq, dk, *more = binding.rmsnorm_rope_bwd_ex(k, q, freqs, None, q, k, qw, qw)
            wait()
            # a write right behind a read
            binding.rmsnorm_block_fwd_ex(dx, h, w, w, w, h=x, y=h)
            wait()
            q = dq
            out += [h, y, dx, dr, *sums, q, dk, *more, x.clone()]
        torch.cuda.synchronize()
        return out

    for a, b in zip(chain(False), chain(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [192, 1030, 4096])
def test_weights_written_by_the_call_before(n, t):
    """Weights and gates that a call writes right behind one that read them, and right before
    one that reads them again."""
    x, r = make((400, n), t, 1).cuda(), make((400, n), t, 2).cuda()
    rows = [make((1, n), t, 10 + i).cuda() for i in range(6)]
    freqs, _ = binding.rmsnorm_rope_freqs(64, device="cuda")
    q = make((500, 6, 64), t, 4).cuda()
    heads = [make((1, 1, 64), t, 20 + i).cuda() for i in range(6)]

    def chain(sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        w, qw, out = torch.ones_like(rows[0][0]), torch.ones_like(heads[0][0, 0]), []
        for i in range(6):
            h, y = binding.rmsnorm_block_fwd_ex(x, r, w, w, w)
            wait()
            d = binding.rmsnorm_block_bwd_ex(y, h, x, h, w, w, w)
            wait()
            tq, _ = binding.rmsnorm_rope_fwd_ex(q, None, freqs, None, qw)
            wait()
            binding.rmsnorm_rope_fwd_ex(heads[i], None, freqs, None, q_out=qw[None, None])
            wait()
            e = binding.rmsnorm_rope_bwd_ex(tq, None, freqs, None, q, None, qw)
            wait()
            binding.rmsnorm_block_fwd_ex(rows[i], rows[i], h=w[None], pre_norm=False)
            wait()
            out += [h, y, *d, tq, e[0], e[2]]
        torch.cuda.synchronize()
        return out

    for a, b in zip(chain(False), chain(True)):
        assert torch.equal(a, b)


# ------------------------------------------------------------- failure detection --

@pytest.fixture(scope="module")
def flib():
    build.build()
    lib = binding.open_library(build.FAULT_LIB_PATH)
    assert lib.rmsnorm_fault_injection_enabled() == 1
    torch.cuda.init()
    yield lib
    torch.cuda.synchronize()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [1024, 1030, 16384])
@pytest.mark.parametrize("fault,cluster", [(1, 0), (1, 2), (2, 2), (2, 4)])
def test_a_wait_that_runs_out(flib, monkeypatch, fault, cluster, n, t):
    """Withheld copies and sums: the waits end after their limit, the status word says so, and
    the next call is right."""
    monkeypatch.setattr(binding, "_lib", flib)
    if cluster and n % 8:
        pytest.skip("rows off the boundaries are not split")
    g = {k: v.cuda() for k, v in {
        "x": make((300, n), t, 1), "r": make((300, n), t, 2), "h": make((300, n), t, 3),
        "w": make((n,), t, 4)}.items()}
    path = {"path": "staged", "cluster": cluster}
    small = n == 1030 or not (t == "f32" and n == 16384 and cluster in (0, 2))

    def run(**kw):
        options = {**path, **kw}
        fwd = binding.rmsnorm_block_fwd_ex(g["x"], g["r"], g["w"], g["w"], options=options)
        state = flib.rmsnorm_last_device_status(torch.cuda.current_stream().cuda_stream)
        bwd, after = None, state
        if small:
            bwd = binding.rmsnorm_block_bwd_ex(g["r"], g["x"], g["x"], g["h"], g["w"], g["w"],
                                               options={**options, "cluster": cluster})
            after = flib.rmsnorm_last_device_status(torch.cuda.current_stream().cuda_stream)
        return fwd, bwd, state, after

    try:
        fwd, bwd, state, after = run()
    except binding.RmsnormError as e:
        # a forced split that this width does not allow: nothing to inject into
        assert e.status == binding.RMSNORM_ERR_UNSUPPORTED
        pytest.skip("unsupported split")
    assert state == after == binding.RMSNORM_OK
    _, _, state, after = run(fault_inject=fault, wait_timeout_ns=20_000_000)
    assert state == after == binding.RMSNORM_ERR_TIMEOUT
    again = run()
    assert again[2] == again[3] == binding.RMSNORM_OK
    for a, b in zip(fwd, again[0]):
        assert torch.equal(a, b)
    if bwd:
        for a, b in zip(bwd, again[1]):
            assert (a is None and b is None) or torch.equal(a, b)
