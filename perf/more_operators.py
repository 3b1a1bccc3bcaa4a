"""Measured cases of what a transformer block does between its matrix products:
its boundary (the norm behind the branch, gate, residual scales, the norm before
the next branch) and the rotary positions of queries and keys with their
per-head norm, forward and backward.

``run`` computes each operator either in its plain form (elementary torch
operations in fp32, angles in 64 bits) or, with ``own`` true, through the
library's binding.
"""
import math

import torch

own = False

EPS = 1e-6
RESIDUAL, BRANCH = 0.875, 0.5      # scales of the residual and of the branch
MOST = 250_000_000                 # elements of a drawn case's arrays, at most
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


# --------------------------------------------------------------------- cases --

def _block(name, op, dtype, batch, seq, hidden, gate, post=True, pre=True):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "seq": seq, "hidden": hidden,
            "gate": gate, "post": post, "pre": pre}


def _rope(name, op, dtype, batch, seq, heads, kv_heads, dim, rot, interleaved, norm, scaling,
          factor, far, packed):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "seq": seq, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "interleaved": interleaved,
            "norm": norm, "scaling": scaling, "factor": factor, "far": far, "packed": packed}


def listed():
    return [
        # one decoding step of 64 sequences: latency counts
        _block("block_fwd_decode_bf16", "block_fwd", "bf16", 64, 1, 4096, "none"),
        # a ragged-width batch in fp32, a learned gate for each channel
        _block("block_fwd_ragged_f32", "block_fwd", "f32", 5, 511, 2050, "channel"),
        # a large training batch, a learned gate for each channel
        _block("block_fwd_batch_bf16", "block_fwd", "bf16", 16, 4096, 4096, "channel"),
        # one short sequence's backward pass: latency counts
        _block("block_bwd_sequence_bf16", "block_bwd", "bf16", 1, 128, 2048, "none"),
        # four sequences of 512 tokens in fp32, a gate for each sequence
        _block("block_bwd_step_f32", "block_bwd", "f32", 4, 512, 3584, "sequence"),
        # a large training batch of a wide model
        _block("block_bwd_batch_bf16", "block_bwd", "bf16", 16, 4096, 8192, "channel"),
        # one decoding step of 64 sequences, each at its own far position
        _rope("rope_fwd_decode_bf16", "rope_fwd", "bf16", 64, 1, 32, 8, 128, 128, False, True,
              "bands", 8.0, True, True),
        # ragged sequences in fp32: a part of the head, neighbouring pairs, no norm
        _rope("rope_fwd_part_f32", "rope_fwd", "f32", 5, 511, 16, 16, 80, 32, True, False,
              "linear", 4.0, False, False),
        # the prompt of a long context, q and k inside the projection's output
        _rope("rope_fwd_prompt_bf16", "rope_fwd", "bf16", 1, 65536, 32, 8, 128, 128, False, True,
              "ramp", 4.0, False, True),
        # one short sequence's backward pass: latency counts
        _rope("rope_bwd_sequence_bf16", "rope_bwd", "bf16", 1, 128, 16, 2, 128, 128, False, True,
              "none", 1.0, False, False),
        # ragged sequences in fp32, neighbouring pairs, half of the head
        _rope("rope_bwd_part_f32", "rope_bwd", "f32", 3, 777, 12, 4, 96, 48, True, True,
              "base", 2.0, False, False),
        # a large training batch
        _rope("rope_bwd_batch_bf16", "rope_bwd", "bf16", 16, 4096, 32, 8, 128, 128, False, True,
              "none", 1.0, False, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["block_fwd", "block_bwd", "rope_fwd", "rope_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("block_fwd", "block_bwd"):
        hidden = _log_int(rng, 64, 16384)
        if rng.random() < 0.7:
            hidden = max(64, hidden // 64 * 64)      # most widths are round, some are odd
        rows = _log_int(rng, 1, min(65536, MOST // hidden))
        batch = _log_int(rng, 1, min(64, rows))
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        return {"op": op, "dtype": dtype, "batch": batch, "seq": max(1, rows // batch),
                "hidden": hidden, "gate": rng.choice(["none", "channel", "sequence"]),
                "post": post, "pre": pre}
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 7])
    tokens = _log_int(rng, 1, min(65536, MOST // (dim * (heads + kv_heads))))
    batch = _log_int(rng, 1, min(64, tokens))
    scaling = rng.choice(["none", "linear", "base", "ramp", "bands"])
    return {"op": op, "dtype": dtype, "batch": batch, "seq": max(1, tokens // batch),
            "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rng.choice([dim, dim, dim // 2, dim // 4]),
            "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.6, "scaling": scaling,
            "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
            "far": rng.random() < 0.5, "packed": rng.random() < 0.5}


def _gates(case):
    return {"none": 0, "channel": 1, "sequence": case["batch"]}[case["gate"]]


def work(case):
    s = SIZES[case["dtype"]]
    if case["op"].startswith("block"):
        h, post, pre = case["hidden"], case["post"], case["pre"]
        n = case["batch"] * case["seq"] * h
        small = (post + pre + _gates(case)) * h
        if case["op"] == "block_fwd":
            return {"bytes": (3 + pre) * n * s + small * s, "flops": (4 + 4 * post + 4 * pre) * n}
        return {"bytes": (4 + 2 * pre) * n * s + small * (s + 4),
                "flops": (4 + 10 * post + 10 * pre) * n}
    tokens = case["batch"] * case["seq"]
    n = tokens * (case["heads"] + case["kv_heads"]) * case["dim"]
    turned = n // case["dim"] * case["rot"]
    seen = 8 * (tokens if case["far"] else case["seq"]) + 4 * case["rot"]
    if case["op"] == "rope_fwd":
        small = 2 * case["dim"] * s if case["norm"] else 0
        return {"bytes": 2 * n * s + seen + small, "flops": 3 * turned + 4 * n * case["norm"]}
    small = 2 * case["dim"] * (s + 4) if case["norm"] else 0
    return {"bytes": (2 + case["norm"]) * n * s + seen + small,
            "flops": 3 * turned + 10 * n * case["norm"]}


# -------------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(scale).add_(mean).to(t)

    if case["op"].startswith("block"):
        b, s, h = case["batch"], case["seq"], case["hidden"]
        st = {"case": case, "x": normal(b, s, h, scale=0.5), "gate": None,
              "post_w": normal(h, scale=0.1, mean=1.0) if case["post"] else None,
              "pre_w": normal(h, scale=0.1, mean=1.0) if case["pre"] else None}
        if case["gate"] != "none":
            shape = (h,) if case["gate"] == "channel" else (b, h)
            st["gate"] = normal(*shape, scale=0.3, mean=0.5)
        # a residual stream whose channels differ in size, a few of them large
        column = torch.rand((h,), generator=g, device="cuda").add_(0.5)
        column[torch.rand((h,), generator=g, device="cuda") < 0.01] *= 10
        residual = torch.randn((b, s, h), generator=g, device="cuda").mul_(column).to(t)
        if case["op"] == "block_fwd":
            st["residual"] = residual
            return st
        st["residual"] = residual
        st["h"] = _plain_block_fwd(st)[0]
        del st["residual"]
        st["dh"] = normal(b, s, h)
        st["dy"] = normal(b, s, h) if case["pre"] else None
        return st

    b, s, dim = case["batch"], case["seq"], case["dim"]
    heads, kv = case["heads"], case["kv_heads"]

    def pair():
        if case["packed"]:       # q, k and v side by side, as one projection writes them
            qkv = normal(b, s, heads + 2 * kv, dim)
            return qkv[:, :, :heads], qkv[:, :, heads:heads + kv]
        return normal(b, s, heads, dim), normal(b, s, kv, dim)

    st = {"case": case, "q_w": None, "k_w": None}
    if case["norm"]:
        st["q_w"], st["k_w"] = (normal(dim, scale=0.1, mean=1.0) for _ in range(2))
    if case["far"]:              # each token somewhere in a long context
        st["positions"] = torch.randint(0, 1 << 20, (b, s), generator=g, device="cuda")
    else:                        # the same for every sequence
        st["positions"] = torch.arange(s, device="cuda")
    if case["op"] == "rope_fwd" or case["norm"]:
        st["q"], st["k"] = pair()
    if case["op"] == "rope_bwd":
        st["dq"], st["dk"] = normal(b, s, heads, dim), normal(b, s, kv, dim)
    if own:
        from row_wise_rmsnorm_fwd_gb300 import binding
        st["freqs"], st["mscale"] = binding.rmsnorm_rope_freqs(
            case["rot"], base=BASE, scaling=case["scaling"], factor=case["factor"],
            original_len=TRAINED, device="cuda")
    else:
        st["freqs"], st["mscale"] = _frequencies(case)
    return st


# ----------------------------------------------------------------- frequencies --

BASE, TRAINED = 10000.0, 8192      # of the unscaled frequencies, and positions seen in training


def _frequencies(case):
    """Angle per position of each pair, fp64, and the scale of what is turned."""
    rot, kind, factor = case["rot"], case["scaling"], case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base = BASE * factor ** (rot / (rot - 2)) if kind == "base" else BASE
    f = base ** (-2 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ramp":
        # the pair that makes `turns` turns over the trained length
        where = [rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(BASE))
                 for turns in (32, 1)]
        low, high = max(math.floor(where[0]), 0), min(math.ceil(where[1]), rot - 1)
        share = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * share + f * (1 - share), 0.1 * math.log(factor) + 1
    if kind == "bands":
        turns = TRAINED * f / (2 * math.pi)
        share = ((turns - 1) / (4 - 1)).clamp(0, 1)
        return f / factor * (1 - share) + f * share, 1.0
    return f, 1.0


# --------------------------------------------------------------- plain forms --

def _gate_of(st):
    """The gate, to be multiplied with [batch, seq, hidden]."""
    gate = st["gate"]
    if gate is None:
        return 1.0
    return gate.float() if gate.dim() == 1 else gate.float()[:, None]


def _plain_block_fwd(st):
    x = st["x"].float()
    if st["case"]["post"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["post_w"].float()
    h = RESIDUAL * st["residual"].float() + BRANCH * (_gate_of(st) * x)
    out = h.to(st["x"].dtype)
    if not st["case"]["pre"]:
        return out, None
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["pre_w"].float()
    return out, y.to(st["x"].dtype)


def _plain_norm_bwd(g, xh, rstd):
    return (g - xh * (g * xh).mean(-1, keepdim=True)) * rstd


def _plain_block_bwd(st):
    case, t = st["case"], st["x"].dtype
    d, x, gate = st["dh"].float(), st["x"].float(), _gate_of(st)
    dpre = dpost = dgate = None
    if case["pre"]:
        h, dy = st["h"].float(), st["dy"].float()
        rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        h = h * rstd
        dpre = (dy * h).sum((0, 1))
        d = d + _plain_norm_bwd(dy * st["pre_w"].float(), h, rstd)
    e = BRANCH * d
    if case["post"]:
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * rstd
        n = xh * st["post_w"].float()
        dn = e * gate
        dpost = (dn * xh).sum((0, 1))
        dx = _plain_norm_bwd(dn * st["post_w"].float(), xh, rstd)
    else:
        n, dx = x, e * gate
    if st["gate"] is not None:
        dgate = (e * n).sum((0, 1) if st["gate"].dim() == 1 else 1)
    return dx.to(t), (RESIDUAL * d).to(t), dpost, dpre, dgate


def _angles(st):
    """cos and sin with their scale, fp32, [batch or 1, seq, 1, rot / 2]."""
    pos = st["positions"]
    a = (pos if pos.dim() == 2 else pos[None])[..., None, None].double() * st["freqs"]
    return (a.cos() * st["mscale"]).float(), (a.sin() * st["mscale"]).float()


def _turn(case, x, c, s):
    rot = case["rot"]
    out = x.clone()
    if case["interleaved"]:
        one, two = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = one * c - two * s, two * c + one * s
    else:
        one, two = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = one * c - two * s, two * c + one * s
    return out


def _plain_rope_fwd(st):
    case, (c, s) = st["case"], _angles(st)
    outs = []
    for x, w in ((st["q"], st["q_w"]), (st["k"], st["k_w"])):
        v = x.float()
        if case["norm"]:
            v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()
        outs.append(_turn(case, v, c, s).to(x.dtype))
    return tuple(outs)


def _plain_rope_bwd(st):
    case, (c, s) = st["case"], _angles(st)
    dxs, dws = [], []
    for n in ("q", "k"):
        dy = st["d" + n]
        g = _turn(case, dy.float(), c, -s)
        if case["norm"]:
            x = st[n].float()
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            x = x * rstd
            dws.append((g * x).sum((0, 1, 2)))
            g = _plain_norm_bwd(g * st[n + "_w"].float(), x, rstd)
        dxs.append(g.to(dy.dtype))
    return (*dxs, *dws) if case["norm"] else (*dxs, None, None)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"block_fwd": _plain_block_fwd, "block_bwd": _plain_block_bwd,
                "rope_fwd": _plain_rope_fwd, "rope_bwd": _plain_rope_bwd}[op](state)
    from row_wise_rmsnorm_fwd_gb300 import binding
    t, st = case["dtype"], state
    if op.startswith("block"):
        how = dict(post_norm=case["post"], pre_norm=case["pre"], residual_scale=RESIDUAL,
                   branch_scale=BRANCH, post_eps=EPS, pre_eps=EPS)
        if op == "block_fwd":
            fn = binding.rmsnorm_block_fwd_f32 if t == "f32" else binding.rmsnorm_block_fwd_bf16
            return fn(st["x"], st["residual"], st["post_w"], st["pre_w"], st["gate"], **how)
        fn = binding.rmsnorm_block_bwd_f32 if t == "f32" else binding.rmsnorm_block_bwd_bf16
        return fn(st["dy"], st["dh"], st["x"], st["h"], st["post_w"], st["pre_w"], st["gate"],
                  **how)
    how = dict(norm=case["norm"], interleaved=case["interleaved"], mscale=st["mscale"], eps=EPS)
    if op == "rope_fwd":
        fn = binding.rmsnorm_rope_fwd_f32 if t == "f32" else binding.rmsnorm_rope_fwd_bf16
        return fn(st["q"], st["k"], st["freqs"], st["positions"], st["q_w"], st["k_w"], **how)
    fn = binding.rmsnorm_rope_bwd_f32 if t == "f32" else binding.rmsnorm_rope_bwd_bf16
    if not case["norm"]:
        return fn(st["dq"], st["dk"], st["freqs"], st["positions"], **how)
    return fn(st["dq"], st["dk"], st["freqs"], st["positions"], st["q"], st["k"], st["q_w"],
              st["k_w"], **how)


# ------------------------------------------------------------------- 64 bits --

def _exact_norm(x, w):
    size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    return x / torch.sqrt(size ** 2 / x.shape[-1] + EPS) * w


def _exact_branch(case, x, post_w, gate):
    n = _exact_norm(x, post_w) if case["post"] else x
    if gate is None:
        return n
    return torch.einsum("bsh,h->bsh" if gate.dim() == 1 else "bsh,bh->bsh", n, gate)


def _exact_block(case, st):
    wide = {n: st[n].double() if st.get(n) is not None else None
            for n in ("x", "residual", "post_w", "pre_w", "gate", "h", "dh", "dy")}
    if case["op"] == "block_fwd":
        h = torch.add(wide["residual"] * RESIDUAL,
                      _exact_branch(case, wide["x"], wide["post_w"], wide["gate"]), alpha=BRANCH)
        return h, _exact_norm(h, wide["pre_w"]) if case["pre"] else None
    leaves = {n: wide[n].requires_grad_() for n in ("x", "post_w", "pre_w", "gate", "h")
              if wide[n] is not None}
    d, dpre = wide["dh"], None
    if case["pre"]:
        more, dpre = torch.autograd.grad(_exact_norm(leaves["h"], leaves["pre_w"]),
                                         (leaves["h"], leaves["pre_w"]), wide["dy"])
        d = d + more
    names = [n for n in ("x", "post_w", "gate") if n in leaves]
    got = dict(zip(names, torch.autograd.grad(
        _exact_branch(case, leaves["x"], leaves.get("post_w"), leaves.get("gate")),
        [leaves[n] for n in names], BRANCH * d)))
    return got["x"], RESIDUAL * d, got.get("post_w"), dpre, got.get("gate")


def _exact_turns(case, st):
    """What a pair is multiplied with, as a complex number: [batch or 1, seq, 1, rot / 2]."""
    rot, kind, k = case["rot"], case["scaling"], case["factor"]
    angle, mscale = [], 1.0
    for i in range(rot // 2):
        f = math.exp(-math.log(BASE) * 2 * i / rot)
        if kind == "linear":
            f /= k
        elif kind == "base":
            f *= math.exp(-math.log(k) * 2 * i / (rot - 2))
        elif kind == "ramp":
            mscale = 1 + math.log(k) / 10
            fast, slow = (rot / 2 * math.log(TRAINED / (2 * math.pi * b), BASE) for b in (32, 1))
            fast, slow = max(int(fast // 1), 0), min(-int(-slow // 1), rot - 1)
            keep = 1 - min(1.0, max(0.0, (i - fast) / (slow - fast if slow > fast else 0.001)))
            f *= keep + (1 - keep) / k
        elif kind == "bands":
            length = 2 * math.pi / f
            if length > TRAINED:
                f /= k
            elif length >= TRAINED / 4:
                keep = (TRAINED / length - 1) / 3
                f *= keep + (1 - keep) / k
        angle.append(f)
    pos = st["positions"].reshape(-1, case["seq"], 1, 1).double()
    angle = pos * torch.tensor(angle, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(angle, mscale), angle)


def _exact_rotate(case, x, turns):
    rot = case["rot"]
    if case["interleaved"]:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turns
        front = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turns
        front = torch.cat([z.real, z.imag], -1)
    return torch.cat([front, x[..., rot:]], -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("block"):
        return _exact_block(case, st)
    turns = _exact_turns(case, st)
    if case["op"] == "rope_fwd":
        return tuple(_exact_rotate(case, _exact_norm(st[n].double(), st[n + "_w"].double())
                                   if case["norm"] else st[n].double(), turns) for n in ("q", "k"))
    dxs, dws = [], []
    for n in ("q", "k"):
        g = _exact_rotate(case, st["d" + n].double(), turns.conj())   # the transpose turns back
        if not case["norm"]:
            dxs.append(g)
            dws.append(None)
            continue
        x, w = (st[m].double().requires_grad_() for m in (n, n + "_w"))
        dx, dw = torch.autograd.grad(_exact_norm(x, w), (x, w), g)
        dxs.append(dx)
        dws.append(dw)
    return (*dxs, *dws)
