"""A wait of the block boundary's cluster kernels that runs out for one thread of a CTA alone, as
it can where the sums arrive close to the limit: each thread has a clock of its own (GPU).

The test build makes the last thread of rank 0 take its first wait as run out.  In the last row of
a cluster nothing but the kernel's own agreement tells the other threads; in any earlier row the
next row's barrier does."""
import pytest
import torch

from _train64 import TYPES, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

LATE = 3
LIMIT_NS = 20_000_000


@pytest.fixture
def flib(monkeypatch):
    build.build()
    lib = binding.open_library(build.FAULT_LIB_PATH)
    assert lib.rmsnorm_fault_injection_enabled() == 1
    torch.cuda.init()
    monkeypatch.setattr(binding, "_lib", lib)
    yield lib
    torch.cuda.synchronize()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("norms", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("n,cluster", [(1024, 2), (16384, 4)])
@pytest.mark.parametrize("rows", [1, 2, 900])
def test_one_thread_late(flib, rows, n, cluster, norms, t):
    post, pre = norms
    g = {k: make((rows, n), t, i).cuda() for i, k in enumerate(("x", "r", "h", "dy", "dh"))}
    w = make((n,), t, 9, mean=1.0, std=0.1).cuda()
    weights = (w if post else None, w if pre else None)
    rule = dict(post_norm=post, pre_norm=pre)

    def state():
        return flib.rmsnorm_last_device_status(torch.cuda.current_stream().cuda_stream)

    def fwd(**kw):
        out = binding.rmsnorm_block_fwd_ex(g["x"], g["r"], *weights, **rule,
                                           options=dict(path="staged", cluster=cluster, **kw))
        return out, state()

    def bwd(**kw):
        out = binding.rmsnorm_block_bwd_ex(g["dy"] if pre else None, g["dh"], g["x"], g["h"],
                                           *weights, **rule,
                                           options=dict(path="staged", cluster=cluster, **kw))
        return out, state()

    for run in (fwd, bwd):
        want, ok = run()
        assert ok == binding.RMSNORM_OK
        assert run(fault_inject=LATE, wait_timeout_ns=LIMIT_NS)[1] == binding.RMSNORM_ERR_TIMEOUT
        got, ok = run()
        assert ok == binding.RMSNORM_OK
        for a, b in zip(want, got):
            assert (a is None and b is None) or torch.equal(a, b)


def test_late_thread_is_test_build_only(flib):
    x = torch.ones(2, 1024, device="cuda")
    for options, status in ((dict(fault_inject=LATE), binding.RMSNORM_ERR_UNSUPPORTED),
                            (dict(fault_inject=LATE, path="staged"), binding.RMSNORM_ERR_UNSUPPORTED),
                            (dict(fault_inject=LATE + 1, path="staged", cluster=2),
                             binding.RMSNORM_ERR_INVALID_ARG)):
        with pytest.raises(binding.RmsnormError) as e:
            binding.rmsnorm_block_fwd_ex(x, x, options=options)
        assert e.value.status == status
