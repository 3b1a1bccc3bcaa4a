"""64-bit references of the training operators (layer norm, the norm backward
passes, the row softmax with a relative position bias) and the error bounds
their kernels are held to.

Bounds.  u = 2^-24 is half a step of fp32; an output of type t is rounded once,
off by at most finfo(t).eps / 2 of its value.  A sum of n terms whose longest
chain of additions is k long is off by at most k * u * (sum of |terms|).  The
chains of the kernels here are at most K = 160 long within a row: up to 137
elements per thread at the widest tested rows (70001 elements over 512
threads), then 5 levels of a warp and at most 16 warps.
"""
from fractions import Fraction

import torch

U = 2.0 ** -24
K = 160
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(t):
    return torch.finfo(t).eps / 2


def close(got, ref, tol, what=""):
    """|got - ref| <= tol element by element; NaN must meet NaN."""
    got, ref, tol = got.detach().double().cpu(), ref.double().cpu(), tol.double().cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} for {tuple(ref.shape)}"
    nan = ref.isnan()
    assert (got.isnan() == nan).all(), f"{what}: NaN in other places"
    bad = ((got - ref).abs() > tol) & ~nan & ~(got == ref)
    if bad.any():
        i = int(((got - ref).abs() / tol.clamp(min=1e-300)).where(bad, torch.zeros_like(ref))
                .flatten().argmax())
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: "
            f"{got.flatten()[i].item()!r} for {ref.flatten()[i].item()!r}, "
            f"allowed {tol.flatten()[i].item():.3g}")


def make(shape, t, seed, mean=0.0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (mean + std * torch.randn(shape, generator=g)).to(TYPES[t])


# ------------------------------------------------------------------- norms --

def layernorm(x, w, b, eps):
    """(y, mean, rstd) and their bounds."""
    x64 = x.double()
    mean = x64.mean(-1, keepdim=True)
    var = ((x64 - mean) ** 2).mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    w64 = w.double() if w is not None else torch.ones(x.shape[-1], dtype=torch.float64)
    b64 = b.double() if b is not None else torch.zeros(x.shape[-1], dtype=torch.float64)
    scaled = (x64 - mean) * rstd * w64
    y = scaled + b64
    top = x64.abs().amax(-1, keepdim=True)
    # the mean is off by at most K*u*max|x|; the sum of squares about the computed
    # mean by (K + 4)*u of itself and by that offset squared; rsqrt halves both
    off = K * U * top
    rel = (K / 2 + 4) * U + (off * rstd) ** 2 / 2
    tol_y = (w64.abs() * rstd * (off + U * top) + scaled.abs() * (rel + 4 * U) + 2 * U * y.abs()
             + half_step(x.dtype) * y.abs() * (1 + 2.0 ** -8))
    # bf16: the rounding is of the computed value
    tol_y = tol_y * (1 + half_step(x.dtype))
    return (y, mean[..., 0], rstd[..., 0]), (tol_y, off[..., 0] + U * mean[..., 0].abs(),
                                             (rstd * (rel + 4 * U))[..., 0])


def _bwd(dy, x, w, xh, rstd, layer, rel):
    """dx, dw, db and bounds; xh is off by rel of itself, rstd too."""
    w64 = w.double() if w is not None else torch.ones(x.shape[-1], dtype=torch.float64)
    d64 = dy.double()
    g = d64 * w64
    c1 = g.mean(-1, keepdim=True) if layer else torch.zeros_like(rstd)
    c2 = (g * xh).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    m1 = g.abs().mean(-1, keepdim=True) if layer else torch.zeros_like(rstd)
    m2 = (g * xh).abs().mean(-1, keepdim=True)
    parts = g.abs() + c1.abs() + (xh * c2).abs()
    tol = rstd * (4 * U * parts + (K + 4) * U * m1 + xh.abs() * m2 * ((K + 8) * U + 2 * rel)
                  + rel * parts)
    tol = tol + half_step(x.dtype) * (dx.abs() + tol)
    rows = x[..., 0].numel()
    chain = (rows + 40) * U             # no chain over rows is longer than they are
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    dw = flat(d64 * xh).sum(0)
    tol_w = flat((d64 * xh).abs()).sum(0) * (chain + 4 * U + rel)
    db = flat(d64).sum(0)
    tol_b = flat(d64.abs()).sum(0) * chain
    return (dx, dw, db), (tol, tol_w, tol_b)


def layernorm_bwd(dy, x, w, mean, rstd):
    """From the mean and rstd that the kernel is given."""
    xh = (x.double() - mean.double()[..., None]) * rstd.double()[..., None]
    return _bwd(dy, x, w, xh, rstd.double()[..., None], True, 3 * U)


def rmsnorm_bwd(dy, x, w, eps):
    x64 = x.double()
    rstd = ((x64 * x64).mean(-1, keepdim=True) + eps).rsqrt()
    (dx, dw, _), (tx, tw, _) = _bwd(dy, x, w, x64 * rstd, rstd, False, (K / 2 + 4) * U)
    return (dx, dw), (tx, tw)


# ------------------------------------------- softmax with a relative bias --

def bucket_edges(half, distance):
    """Smallest distance of each bucket of a direction, in whole numbers: n has
    reached bucket near + k when (n / near)^(half - near) >= (distance / near)^k."""
    near = half // 2
    edges = list(range(near))
    for k in range(half - near):
        bound = Fraction(distance, near) ** k
        lo, hi = 0, distance
        while lo < hi:
            n = (lo + hi) // 2
            if Fraction(n, near) ** (half - near) >= bound:
                hi = n
            else:
                lo = n + 1
        edges.append(lo)
    return edges


def bucket(r, num_buckets, distance, both):
    half = num_buckets // 2 if both else num_buckets
    n = abs(r) if both else max(-r, 0)
    k = max(i for i, e in enumerate(bucket_edges(half, distance)) if e <= n)
    return k + (half if both and r > 0 else 0)


class Rule:
    """A bias rule, as keyword arguments of the binding and as 64-bit arithmetic."""

    def __init__(self, num_buckets=32, max_distance=128, both=True, causal=False, scale=1.0,
                 q_offset=0, q_start=None, kv_len=None):
        self.num_buckets, self.max_distance, self.both = num_buckets, max_distance, both
        self.causal, self.scale, self.q_offset = causal, scale, q_offset
        self.q_start, self.kv_len = q_start, kv_len

    def kwargs(self, device="cuda"):
        at = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
        return dict(max_distance=self.max_distance, bidirectional=self.both, causal=self.causal,
                    scale=self.scale, q_offset=self.q_offset, q_start=at(self.q_start),
                    kv_len=at(self.kv_len))

    def places(self, b, q, k):
        """(buckets, valid): [b, q, k]."""
        start = torch.tensor(self.q_start or [0] * b, dtype=torch.int64)
        r = torch.arange(k) - (self.q_offset + start[:, None, None] + torch.arange(q)[:, None])
        half = self.num_buckets // 2 if self.both else self.num_buckets
        edges = torch.tensor(bucket_edges(half, self.max_distance))
        n = r.abs() if self.both else (-r).clamp(min=0)
        which = torch.searchsorted(edges, n, right=True) - 1
        if self.both:
            which = which + half * (r > 0)
        valid = torch.ones_like(r, dtype=torch.bool)
        if self.kv_len is not None:
            valid &= torch.arange(k) < torch.tensor(self.kv_len)[:, None, None]
        if self.causal:
            valid &= r <= 0
        return which, valid


def relbias(x, table, rule):
    """y and its bound."""
    b, h, q, k = x.shape
    which, valid = rule.places(b, q, k)
    valid = valid[:, None].expand(x.shape)
    bias = table.double()[which].permute(0, 3, 1, 2)
    sx = rule.scale * x.double()
    v = torch.where(valid, sx + bias, float("-inf"))
    top = v.amax(-1, keepdim=True)
    e = torch.exp(v - top)
    e = torch.where(valid, e, 0.0)
    y = torch.where(valid, e / e.sum(-1, keepdim=True), 0.0)
    # v is off by 2u(|sx| + |bias|), exp's argument by |v| and |top| roundings more;
    # 2^-21 covers the exponential (2^-22) twice, K*u the sum
    size = torch.where(valid & v.isfinite(), sx.abs() + bias.abs(), 0.0)
    rel = 16 * U * size.amax(-1, keepdim=True) + (K + 8) * U + 2.0 ** -21
    tol = y * (rel + half_step(x.dtype) * (1 + rel)) + 1e-37
    return y, tol


def relbias_bwd(dy, y, rule):
    """(dx, dtable) and bounds, from the y that the kernel is given."""
    b, h, q, k = y.shape
    which, valid = rule.places(b, q, k)
    valid = valid[:, None].expand(y.shape)
    y64 = torch.where(valid, y.double(), 0.0)
    d64 = torch.where(valid, dy.double(), 0.0)
    dot = (y64 * d64).sum(-1, keepdim=True)
    ds = y64 * (d64 - dot)
    tol = y64.abs() * (4 * U * (d64.abs() + dot.abs())
                       + (K + 4) * U * (y64 * d64).abs().sum(-1, keepdim=True))
    dx = rule.scale * ds
    tol_x = abs(rule.scale) * tol
    tol_x = tol_x + (half_step(y.dtype) + 2 * U) * (dx.abs() + tol_x)
    dt = torch.zeros((rule.num_buckets, h), dtype=torch.float64)
    tol_t = torch.zeros_like(dt)
    # a bucket's fp32 chains: 64 rows of a few vectors of a thread, their 8 elements, a
    # warp, the window's up to 16 groups; then fp64
    chain = 700 * U
    flat = which.reshape(-1)
    for src, dst in ((ds, dt), (tol + chain * ds.abs(), tol_t)):
        dst.index_add_(0, flat, src.permute(0, 2, 3, 1).reshape(-1, h))
    return (dx, dt), (tol_x, tol_t + 2 * U * dt.abs())
