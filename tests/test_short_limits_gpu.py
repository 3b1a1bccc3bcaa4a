"""Limits of device-side waits that are shorter than a copy takes (GPU).  A kernel whose wait has
run out may only leave once what is under way to its shared memory has landed, so a limit below a
millisecond counts as one: a wait that never ends takes at least that long, and a call with
nothing wrong ends as with the default limit."""
import pytest
import torch

from _train64 import TYPES, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

LEAST_MS = 1.0


@pytest.fixture
def flib(monkeypatch):
    build.build()
    lib = binding.open_library(build.FAULT_LIB_PATH)
    assert lib.rmsnorm_fault_injection_enabled() == 1
    torch.cuda.init()
    monkeypatch.setattr(binding, "_lib", lib)
    yield lib
    torch.cuda.synchronize()


def calls(n, t):
    """name -> call(options) of the operators whose kernels wait for copies of their own."""
    x, r, h = (make((600, n), t, i).cuda() for i in range(3))
    w = make((n,), t, 5, mean=1.0, std=0.1).cuda()

    def block_bwd(o):
        return binding.rmsnorm_block_bwd_ex(r, h, x, h, w, w, options=o)

    return {"rmsnorm": lambda o: [binding.rmsnorm_fwd_ex(x, w, eps=1e-6, options=o)],
            "softmax": lambda o: [binding.rowsoftmax_fwd_ex(x, options=o)],
            "layer norm": lambda o: [binding.layernorm_fwd_ex(x, w, w, options=o)],
            "rmsnorm backward": lambda o: binding.rmsnorm_bwd_ex(r, x, w, options=o),
            "block": lambda o: binding.rmsnorm_block_fwd_ex(x, r, w, w, options=o),
            "block backward": block_bwd}


def flat(out):
    return [v for v in (out if isinstance(out, (list, tuple)) else [out])
            if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("limit", [1, 1000, 999_999])
@pytest.mark.parametrize("name", ["rmsnorm", "softmax", "layer norm", "rmsnorm backward", "block",
                                  "block backward"])
def test_limits_below_a_millisecond(flib, name, limit, t):
    call = calls(4096, t)[name]

    def state():
        return flib.rmsnorm_last_device_status(torch.cuda.current_stream().cuda_stream)

    want = flat(call({"path": "staged"}))
    assert state() == binding.RMSNORM_OK
    got = flat(call({"path": "staged", "wait_timeout_ns": limit}))
    assert state() == binding.RMSNORM_OK
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    call({"path": "staged", "wait_timeout_ns": limit, "fault_inject": 1})
    b.record()
    assert state() == binding.RMSNORM_ERR_TIMEOUT
    assert a.elapsed_time(b) >= LEAST_MS
    for a, b in zip(want, flat(call({"path": "staged"}))):
        assert torch.equal(a, b)
    assert state() == binding.RMSNORM_OK


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("cluster", [2, 4])
def test_limits_over_a_cluster(flib, cluster, t):
    """The block boundary's sums of split rows."""
    both = calls(8192, t)

    def state():
        return flib.rmsnorm_last_device_status(torch.cuda.current_stream().cuda_stream)

    for name in ("block", "block backward"):
        o = {"path": "staged", "cluster": cluster}
        try:
            want = flat(both[name](o))
        except binding.RmsnormError as e:
            assert e.status == binding.RMSNORM_ERR_UNSUPPORTED
            continue
        got = flat(both[name]({**o, "wait_timeout_ns": 1}))
        assert state() == binding.RMSNORM_OK
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        both[name]({**o, "wait_timeout_ns": 1, "fault_inject": 2})
        b.record()
        assert state() == binding.RMSNORM_ERR_TIMEOUT
        assert a.elapsed_time(b) >= LEAST_MS
