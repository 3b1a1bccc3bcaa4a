"""The block boundary's forward kernel for ragged rows staged in shared memory, forced: the
automatic choice takes it for rows below 512 bytes only, so that its rows of several warps, of
many blocks to a CTA and at the end of the arrays are compared with the 64-bit references here
(GPU; bounds as in _between64)."""
import pytest
import torch

import _between64 as ref
from _between64 import Block
from _train64 import TYPES, close, make
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu

STAGED = {"path": "staged"}
RULES = {"both": Block(rs=0.75, bs=-1.5), "post": Block(pre=False), "pre": Block(post=False, rs=2.0),
         "none": Block(post=False, pre=False, bs=0.5)}
# elements of 24 KB, the widest row
WIDEST = {"f32": 6144, "bf16": 12288}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def off(t):
    """The tensor on the GPU one element behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
    assert flat.data_ptr() % 16 == 0
    return flat[1:1 + t.numel()].view(t.shape).copy_(t)


def run(rows, n, t, rule, gate, aside, **kw):
    x, r = make((rows, n), t, 1, mean=0.1, std=0.7), make((rows, n), t, 2, std=1.5)
    post = make((n,), t, 3, mean=1.0, std=0.2) if rule.post else None
    pre = make((n,), t, 4, mean=1.0, std=0.2) if rule.pre else None
    g = {"none": None, "channel": make((n,), t, 5, mean=0.4, std=0.5),
         "row": make((rows, n), t, 5, mean=0.4, std=0.5)}[gate]
    put = off if aside else (lambda v: v.cuda())
    small = [None if v is None else put(v) for v in (post, pre, g)]
    got = binding.rmsnorm_block_fwd_ex(x.cuda(), r.cuda(), *small, **rule.kwargs(), options=STAGED,
                                       **kw)
    want, bound = ref.block_fwd(x, r, post, pre, g, rule)
    for name, a, b, c in zip(("h", "y"), got, want, bound):
        assert (a is None) == (b is None), name
        if b is not None:
            close(a, b, c, name)


# rows that end 2 to 14 bytes behind a boundary, in several warps, many to a CTA and one to
# a CTA, more rows than CTAs and fewer
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [7, 66, 130, 259, 518, 1027, 2050, 4097, 6002])
@pytest.mark.parametrize("rows", [1, 5, 700])
def test_ragged_widths(rows, n, t):
    if n * TYPES[t].itemsize < 16:
        pytest.skip("rows of less than 16 bytes are not staged")
    run(rows, n, t, RULES["both"], "channel", False)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
def test_ragged_rules(gate, rule, t):
    for rows, n in ((37, 259), (333, 1030)):
        run(rows, n, t, RULES[rule], gate, False)


@pytest.mark.parametrize("t", TYPES)
def test_widest_rows(t):
    """Rows of 24 KB, in one-element pieces because their weights lie off the boundaries."""
    n = WIDEST[t]
    for rows, width in ((3, n), (200, n), (5, n - 288), (9, n - 1)):
        run(rows, width, t, RULES["both"], "channel", True)
    for width in (n + 1, n + 8):
        with pytest.raises(binding.RmsnormError) as e:
            run(3, width, t, RULES["both"], "channel", True)
        assert e.value.status == binding.RMSNORM_ERR_UNSUPPORTED


@pytest.mark.parametrize("t", TYPES)
def test_ragged_in_place(t):
    n, rule = 1027, RULES["both"]
    x, r = make((700, n), t, 1).cuda(), make((700, n), t, 2).cuda()
    w = make((n,), t, 3, mean=1.0, std=0.2).cuda()
    want = binding.rmsnorm_block_fwd_ex(x, r, w, w, w, **rule.kwargs(), options=STAGED)
    for h, y in ((0, 1), (1, 0)):
        a = [x.clone(), r.clone()]
        got = binding.rmsnorm_block_fwd_ex(a[0], a[1], w, w, w, h=a[h], y=a[y], **rule.kwargs(),
                                           options=STAGED)
        for g, e in zip(got, want):
            assert torch.equal(g, e)
