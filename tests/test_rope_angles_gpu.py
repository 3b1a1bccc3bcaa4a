"""Cosines and sines of the rotary kernels over the whole circle, against 64 bits (GPU).

A head (1, 0) per pair, without a norm, comes out as the pair's (cos, sin) with nothing rounded
after them.  Bounds in u = 2^-24, of a kernel that takes the nearest quarter turn away from the upper
32 bits of the turns and sums Taylor series of the x that is left, |x| <= pi / 4:

  x        turns below 2^-32: 2 pi 2^-32 = 0.03 u; conversion to fp32, the constant 2 pi / 2^32 and
           their product: u |x| each, 2.36 u; together 2.4 u, which sine and cosine pass on at most
  sine     x + (x q) s with q = x^2: terms behind x^9 / 9! 0.03 u; the last fma u |sin x| <= 0.71 u;
           |x q s| <= 0.081, whose factors are off by 2 u and 3 u of themselves: 0.4 u; 1.2 u
  cosine   1 + q c: the last fma u; |q c| <= 0.293, factors off by u and 1.5 u: 0.74 u; 1.8 u
  mscale   u of the product

so (2.4 + 1.8) u, and u more with an mscale other than one, times |mscale|.  _between64 counts 6 u for
this (its comment names other steps) and its TURN of 10 u adds the rotation's two products, their sum
and the pair's own rounding."""
import math

import pytest
import torch

from _train64 import U
from row_wise_rmsnorm_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    yield
    torch.cuda.synchronize()


def around_quarters():
    """Numbers of 2^-32 turns: next to every eighth of a turn, the smallest, and all over."""
    near = [(k << 29) + d & 0xFFFFFFFF for k in range(8) for d in range(-40, 41)]
    g = torch.Generator().manual_seed(1)
    many = torch.randint(0, 1 << 32, (1 << 18,), generator=g)
    even = torch.arange(0, 1 << 32, (1 << 32) // 100003)
    return torch.cat([torch.tensor(near), many, even])


@pytest.mark.parametrize("path", ["auto", "twopass"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("mscale", [1.0, 1.3862943649291992])
def test_cosine_and_sine(mscale, interleaved, path):
    turns = around_quarters()
    tokens, half = turns.numel(), 8
    # frequency i: (2 i + 1) * 2^32 + 2^31 * i of 2^-64 turns a position, so that a position is a
    # number of turns with bits on both sides of the 32nd
    freqs = torch.tensor([((2 * i + 1) << 32) + (i << 31) for i in range(half)])
    q = torch.zeros(tokens, 1, 2 * half)
    (q[..., 0::2] if interleaved else q[..., :half]).fill_(1.0)
    out, _ = binding.rmsnorm_rope_fwd_ex(q.cuda(), None, freqs.cuda(), turns.cuda(), norm=False,
                                         interleaved=interleaved, mscale=mscale,
                                         options={"path": path})
    out = out.double().cpu()[:, 0]
    c, s = (out[:, 0::2], out[:, 1::2]) if interleaved else (out[:, :half], out[:, half:])
    bound = (4.2 + (mscale != 1.0)) * U * mscale
    for i, f in enumerate(freqs.tolist()):
        # turns * f mod 2^64 in two halves that int64 holds: the angle to 2^-53 of a turn
        low = turns * (f & 0xFFFFFFFF)
        high = turns * (f >> 32) + (low >> 32)
        angle = ((high & 0xFFFFFFFF).double() + (low & 0xFFFFFFFF).double() / 2 ** 32) / 2 ** 32
        angle = angle * 2 * math.pi
        for got, want in ((c[:, i], angle.cos()), (s[:, i], angle.sin())):
            off = (got - mscale * want).abs().max().item()
            assert off <= bound, (i, off / U)
