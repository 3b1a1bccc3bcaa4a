"""64-bit references of the block boundary (norms, gate, residual scales) and of
rotary positions with head norms, and the error bounds that their kernels are held
to.

Bounds, with u = 2^-24 and the rules of _train64.  A row's sum of H terms is added in
chains of at most chain(H) = H / 256 + 40 additions: 256 threads at least share a row of
more than 256 elements (a warp a head of up to 1024), a thread's own terms are summed
vector by vector, then come 5 levels of a warp and at most 16 warps.  A factor
rsqrt(mean of squares + eps) is therefore off by rho(H) = (chain / 2 + 4) u of itself: half
of the sum's error, 4 u for the division by H, the addition of eps and rsqrt.  Every
following operation adds u of its result; the counts below are of those operations.
A column sum over n rows is off by at most (n + 60) u of the sum of |terms|.
"""
import math

import torch

from _train64 import U, half_step


def chain(h):
    return h / 256 + 40


def rho(h):
    return (chain(h) / 2 + 4) * U


def stored(v, tol, t):
    """The bound of a value that is off by tol before it is rounded to type t."""
    return tol + half_step(t) * (v.abs() + tol)


class Block:
    """A boundary's rule, as keyword arguments of the binding and in 64 bits."""

    def __init__(self, post=True, pre=True, rs=1.0, bs=1.0, post_eps=1e-6, pre_eps=1e-5):
        self.post, self.pre = post, pre
        # as the fp32 numbers that the kernels get
        self.rs, self.bs, self.post_eps, self.pre_eps = (
            torch.tensor(v, dtype=torch.float32).double().item() for v in (rs, bs, post_eps, pre_eps))

    def kwargs(self):
        return dict(post_norm=self.post, pre_norm=self.pre, residual_scale=self.rs,
                    branch_scale=self.bs, post_eps=self.post_eps, pre_eps=self.pre_eps)


def wide(w, h):
    return torch.ones(h, dtype=torch.float64) if w is None else w.double()


def gate_rows(gate, x):
    """The gate for every row of x, 64 bits."""
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    g = gate.double()
    return g.reshape(*g.shape[:-1], *[1] * (x.dim() - g.dim()), g.shape[-1]) if g.dim() > 1 else g


def norm_factor(v, eps):
    return ((v * v).mean(-1, keepdim=True) + eps).rsqrt()


def block_fwd(x, residual, post_w, pre_w, gate, rule):
    """(h, y) and their bounds; y None without a pre norm."""
    n, t = x.shape[-1], x.dtype
    x64, r64 = x.double(), residual.double()
    branch = x64 * norm_factor(x64, rule.post_eps) * wide(post_w, n) if rule.post else x64
    branch = rule.bs * gate_rows(gate, x) * branch
    h = rule.rs * r64 + branch
    # x * r * w * gate * bs: 4 products; the addition is one fma
    eh = branch.abs() * ((rho(n) if rule.post else 0) + 5 * U) + 2 * U * h.abs()
    if not rule.pre:
        return (h, None), (stored(h, eh, t), None)
    w = wide(pre_w, n)
    r = norm_factor(h, rule.pre_eps)
    y = h * r * w
    # the sum of squares is of values that are off by eh
    rel = rho(n) + (h.abs() * eh).mean(-1, keepdim=True) * r * r
    ey = (w * r).abs() * (eh * (1 + rel) + h.abs() * (rel + 3 * U))
    return (h, y), (stored(h, eh, t), stored(y, ey, t))


def block_bwd(dy, dh, x, h, post_w, pre_w, gate, rule):
    """(dx, dresidual, dpost_w, dpre_w, dgate) and bounds, from the x and h given."""
    n, t = x.shape[-1], x.dtype
    flat = lambda v: v.reshape(-1, n)  # noqa: E731
    x64 = x.double()
    rows = x64[..., 0].numel()
    add = (rows + 60) * U
    zero = torch.zeros_like(x64)
    d = zero if dh is None else dh.double()
    near = d.abs()                       # sizes of what D is added from
    dpre = tpre = None
    ek = kh = rh = 0.0
    g = h64 = zero
    if rule.pre:
        h64, dy64 = h.double(), dy.double()
        rh = norm_factor(h64, rule.pre_eps)
        g = dy64 * wide(pre_w, n)
        kh = (g * h64).mean(-1, keepdim=True) * rh * rh
        ek = (g * h64).abs().mean(-1, keepdim=True) * rh * rh * (chain(n) + 3) * U \
            + kh.abs() * (2 * rho(n) + 4 * U)
        d = d + rh * (g - h64 * kh)
        terms = dy64 * h64 * rh if pre_w is not None else None
        dpre = flat(terms).sum(0) if pre_w is not None else None
        tpre = flat(terms.abs()).sum(0) * (add + rho(n) + 3 * U) if pre_w is not None else None
    p = rh * (g.abs() + (h64 * kh).abs())
    ed = 2 * U * (near + p) + p * (rho(n) + 4 * U) + rh * h64.abs() * ek
    dres = rule.rs * d
    tres = stored(dres, abs(rule.rs) * ed + U * dres.abs(), t)
    gate64, w = gate_rows(gate, x), wide(post_w if rule.post else None, n)
    u = (gate64 * w).expand(x64.shape)
    f = rule.bs * d * u
    if rule.post:
        rx = norm_factor(x64, rule.post_eps)
        q = u * x64
        mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
        kx = mean(f * x64) * rx * rx
        m0 = mean((q * (zero if dh is None else dh.double())).abs())
        m1, m2 = mean((q * g).abs()) * rh, mean((q * h64).abs()) * rh
        edot = m0 * (chain(n) + 6) * U + m1 * ((chain(n) + 6) * U + rho(n)) \
            + m2 * (abs(kh) if rule.pre else 0.0) * ((chain(n) + 8) * U + rho(n)) + m2 * ek
        ekx = abs(rule.bs) * rx * rx * edot + kx.abs() * (2 * rho(n) + 6 * U)
        dx = rx * (f - x64 * kx)
        sizes = f.abs() + (x64 * kx).abs()
        tx = rx * ((rule.bs * u).abs() * ed + 5 * U * sizes + x64.abs() * ekx) \
            + rx * sizes * (rho(n) + 2 * U)
        xh, rel = x64 * rx, rho(n)
    else:
        dx, xh, rel = f, x64, 0.0
        tx = (rule.bs * u).abs() * ed + 4 * U * f.abs()
    tx = stored(dx, tx, t)
    a = rule.bs * d * xh
    ea = abs(rule.bs) * ed * xh.abs() + a.abs() * (add + rel + 6 * U)
    dpost = tpost = dgate = tgate = None
    if rule.post and post_w is not None:
        dpost = flat(a * gate64).sum(0)
        tpost = flat(ea * gate64.abs() + (a * gate64).abs() * add).sum(0)
    if gate is not None:
        shape = gate.shape[:-1]
        k = len(shape)
        while k and shape[k - 1] == 1:
            k -= 1
        over = tuple(range(k, x.dim() - 1))
        total = lambda v: (v.sum(over) if over else v).reshape(gate.shape)  # noqa: E731
        dgate, tgate = total(a * w), total((ea + U * a.abs()) * w.abs())
    return (dx, dres, dpost, dpre, dgate), (tx, tres, tpost, tpre, tgate)


# ------------------------------------------------------------------ rotation --

def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, low=None,
                     high=None, divisors=None):
    """Angles per position, 64 bits, and mscale."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2 * i / rot)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "base":
        f = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
    elif scaling == "ramp":
        low, high = low or 1.0, high or 32.0
        first, last = (rot * math.log(original_len / (b * 2 * math.pi)) / (2 * math.log(base))
                       for b in (high, low))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
        divided = ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        f = f / factor * divided + f * (1 - divided)
        mscale = 0.1 * math.log(factor) + 1
    elif scaling == "bands":
        low, high = low or 1.0, high or 4.0
        kept = ((original_len * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f / factor * (1 - kept) + f * kept
    if divisors is not None:
        f = f / torch.tensor(divisors, dtype=torch.float64)
    return f, mscale


class Rope:
    """A rule of turning: frequencies (whole numbers, 2^-64 turns a position), layout, norm,
    scale."""

    def __init__(self, freqs, interleaved=False, norm=True, mscale=1.0, eps=1e-6, start=0):
        self.freqs = [int(f) % 2 ** 64 for f in freqs]
        self.interleaved, self.norm, self.start = interleaved, norm, start
        self.mscale, self.eps = (torch.tensor(v, dtype=torch.float32).double().item()
                                 for v in (mscale, eps))
        self.rot = 2 * len(freqs)

    def kwargs(self):
        return dict(norm=self.norm, interleaved=self.interleaved, mscale=self.mscale, eps=self.eps,
                    start=self.start)

    def angles(self, positions, lead):
        """[*lead, 1, rot / 2]; positions None, [seq] or of shape lead."""
        if positions is None:
            positions = torch.arange(lead[-1])
        at = positions.long().expand(lead).flatten().tolist()
        # whole turns taken away in Python's integers: fp64 would lose far positions
        out = [[((p + self.start) * f % 2 ** 64) / 2 ** 64 * 2 * math.pi for f in self.freqs]
               for p in at]
        return torch.tensor(out, dtype=torch.float64).reshape(*lead, 1, len(self.freqs))

    def pairs(self, v):
        if self.interleaved:
            return v[..., 0:self.rot:2], v[..., 1:self.rot:2]
        return v[..., :self.rot // 2], v[..., self.rot // 2:self.rot]

    def joined(self, one, two, v):
        out = v.clone()
        a, b = self.pairs(out)
        a.copy_(one)
        b.copy_(two)
        return out

    def turn(self, v, angles, back=False):
        """The turned v, and for each element the size |one| + |two| of its pair times
        |mscale| (behind the turned part: zeros)."""
        c, s = self.mscale * angles.cos(), self.mscale * angles.sin()
        if back:
            s = -s
        one, two = self.pairs(v)
        size = (one.abs() + two.abs()) * abs(self.mscale)
        return (self.joined(one * c - two * s, two * c + one * s, v),
                self.joined(size, size, torch.zeros_like(v)))


# cos and sin are off by 6 u: the angle by an eighth of a turn's rounding (0.8 u), sincospi by
# 2 u, the product with mscale by u; two products and an addition more
TURN = 10 * U


def rope_fwd(x, w, rule, positions):
    """The output and its bound."""
    n = x.shape[-1]
    v = x.double()
    rel = 0.0
    if rule.norm:
        v = v * norm_factor(v, rule.eps) * wide(w, n)
        rel = rho(n) + 3 * U
    out, size = rule.turn(v, rule.angles(positions, x.shape[:-2]))
    plain = torch.where(size == 0, v.abs(), size)
    return out, stored(out, size * TURN + plain * rel, x.dtype)


def rope_bwd(dy, x, w, rule, positions):
    """(dx, dw) and bounds."""
    n = dy.shape[-1]
    g, size = rule.turn(dy.double(), rule.angles(positions, dy.shape[:-2]), back=True)
    eg = size * TURN
    if not rule.norm:
        return (g, None), (stored(g, eg, dy.dtype), None)
    x64, w64 = x.double(), wide(w, n)
    r = norm_factor(x64, rule.eps)
    gw = g * w64
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    k = mean(gw * x64) * r * r
    ek = r * r * (mean((w64 * x64).abs() * eg) + mean((gw * x64).abs()) * (chain(n) + 4) * U) \
        + k.abs() * (2 * rho(n) + 4 * U)
    dx = r * (gw - x64 * k)
    sizes = gw.abs() + (x64 * k).abs()
    tx = r * (w64.abs() * eg + 3 * U * sizes + x64.abs() * ek) + r * sizes * (rho(n) + U)
    terms = g * x64 * r
    rows = terms[..., 0].numel()
    flat = lambda v: v.reshape(-1, n).sum(0)  # noqa: E731
    tw = flat(eg * (x64 * r).abs() + terms.abs() * ((rows + 60) * U + rho(n) + 2 * U))
    return (dx, flat(terms)), (stored(dx, tx, dy.dtype), tw)
