"""Measured cases of the norm backward passes, layer norm, and the row softmax
with a learned relative position bias.

``run`` computes each operator either in its plain form (elementary torch
operations in fp32) or, with ``own`` true, through the library's binding.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
SCALE = 0.125
MOST = 250_000_000     # elements of a drawn case's tensors, at most
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


# --------------------------------------------------------------------- cases --

def _norm(name, op, dtype, rows, hidden):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "hidden": hidden}


def _bias(name, op, dtype, batch, heads, q, k, causal, ragged, buckets=32, distance=128):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "heads": heads, "q": q,
            "k": k, "causal": causal, "ragged": ragged, "buckets": buckets,
            "distance": distance}


def listed():
    return [
        # the norm of a short prompt: 32 tokens, latency counts
        _norm("ln_fwd_prompt_f32", "ln_fwd", "f32", 32, 2048),
        # a batch of ragged-width rows (8-byte vectors at best, odd row count)
        _norm("ln_fwd_ragged_bf16", "ln_fwd", "bf16", 8191, 2050),
        # a large training batch in fp32
        _norm("ln_fwd_batch_f32", "ln_fwd", "f32", 65536, 4096),
        # one short sequence's backward pass: latency counts
        _norm("ln_bwd_sequence_bf16", "ln_bwd", "bf16", 128, 2048),
        # four sequences of 512 tokens, fp32
        _norm("ln_bwd_step_f32", "ln_bwd", "f32", 2048, 3584),
        # a large training batch of a wide model
        _norm("ln_bwd_batch_bf16", "ln_bwd", "bf16", 65536, 8192),
        # one sequence of ragged-width rows
        _norm("rms_bwd_ragged_f32", "rms_bwd", "f32", 128, 2050),
        # a large training batch
        _norm("rms_bwd_batch_bf16", "rms_bwd", "bf16", 65536, 4096),
        # one decoding step of 64 sequences with caches of 0 to 4096 keys
        _bias("bias_fwd_decode_bf16", "bias_fwd", "bf16", 64, 32, 1, 4096, True, True),
        # encoder attention scores, 8 sequences of 512 tokens
        _bias("bias_fwd_encoder_bf16", "bias_fwd", "bf16", 8, 32, 512, 512, False, False),
        # a small ragged batch in fp32, odd sizes, padded keys
        _bias("bias_bwd_padded_f32", "bias_bwd", "f32", 5, 7, 77, 333, False, True),
        # decoder attention scores in training, causal
        _bias("bias_bwd_decoder_bf16", "bias_bwd", "bf16", 4, 32, 2048, 2048, True, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "rms_bwd", "bias_fwd", "bias_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("ln_fwd", "ln_bwd", "rms_bwd"):
        hidden = _log_int(rng, 64, 16384)
        if rng.random() < 0.7:
            hidden = max(64, hidden // 64 * 64)      # most widths are round, some are odd
        rows = _log_int(rng, 1, min(65536, MOST // hidden))
        return {"op": op, "dtype": dtype, "rows": rows, "hidden": hidden}
    k = _log_int(rng, 1, 8192)
    if rng.random() < 0.5:
        k = max(8, k // 8 * 8)
    causal = rng.random() < 0.5
    q = 1 if rng.random() < 0.25 else _log_int(rng, 1, min(4096, 2 * k))
    heads = _log_int(rng, 1, min(32, MOST // (q * k)))
    batch = _log_int(rng, 1, min(64, MOST // (q * k * heads)))
    return {"op": op, "dtype": dtype, "batch": batch, "heads": heads, "q": q, "k": k,
            "causal": causal, "ragged": rng.random() < 0.5,
            "buckets": rng.choice([16, 32, 64]), "distance": rng.choice([64, 128, 500])}


def _lengths(case):
    """Valid keys of each sequence, and where its first query stands."""
    b, q, k = case["batch"], case["q"], case["k"]
    if case["ragged"]:
        kv = [k * i // max(1, b - 1) if b > 1 else k for i in range(b)]
    else:
        kv = [k] * b
    q0 = [n - q if case["causal"] else 0 for n in kv]
    return kv, q0


def _valid(case):
    """Scores inside the mask, over the batch and heads."""
    kv, q0 = _lengths(case)
    kv, q0 = np.array(kv)[:, None], np.array(q0)[:, None]
    n = np.broadcast_to(kv, (case["batch"], case["q"]))
    if case["causal"]:
        n = np.clip(np.minimum(n, q0 + np.arange(case["q"]) + 1), 0, None)
    return int(n.sum()) * case["heads"]


def work(case):
    s = SIZES[case["dtype"]]
    op = case["op"]
    if op.startswith("bias"):
        n = _valid(case)
        every = case["batch"] * case["heads"] * case["q"] * case["k"]
        small = case["buckets"] * case["heads"]
        if op == "bias_fwd":
            return {"bytes": (n + every) * s + small * s, "flops": 8 * n}
        return {"bytes": (2 * n + every) * s + small * 4, "flops": 7 * n}
    r, h = case["rows"], case["hidden"]
    if op == "ln_fwd":
        return {"bytes": 2 * r * h * s + 2 * h * s + 8 * r, "flops": 8 * r * h}
    if op == "ln_bwd":
        return {"bytes": 3 * r * h * s + h * s + 8 * r + 8 * h, "flops": 14 * r * h}
    return {"bytes": 3 * r * h * s + h * s + 4 * h, "flops": 12 * r * h}


# -------------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(t)

    if case["op"].startswith("bias"):
        b, h, q, k = (case[n] for n in ("batch", "heads", "q", "k"))
        kv, q0 = _lengths(case)
        order = torch.randperm(b, generator=g, device="cuda")
        kv = torch.tensor(kv, device="cuda", dtype=torch.int32)[order]
        q0 = torch.tensor(q0, device="cuda", dtype=torch.int32)[order]
        st = {"case": case, "kv_len": kv if case["ragged"] else None,
              "q_start": q0 if case["ragged"] and case["causal"] else None,
              "q_offset": 0 if case["ragged"] or not case["causal"] else k - q}
        x = normal(b, h, q, k, scale=2.0)
        if case["op"] == "bias_fwd":
            st.update(x=x, table=normal(case["buckets"], h))
            return st
        p = x.float()
        mask = _mask(st, p)
        if mask is not None:
            p = p.masked_fill(~mask, float("-inf"))
        p = p.softmax(-1)
        st.update(y=p.nan_to_num_(nan=0.0).to(t), dy=normal(b, h, q, k))
        return st
    r, h = case["rows"], case["hidden"]
    # activations with a mean of their own in each column, a few columns large
    x = torch.randn((r, h), generator=g, device="cuda")
    column = torch.randn((h,), generator=g, device="cuda")
    large = torch.rand((h,), generator=g, device="cuda") < 0.01
    x = x.mul_(1 + 9 * large.float()).add_(column.mul_(0.5)).to(t)
    st = {"case": case, "x": x, "w": (1 + 0.1 * torch.randn((h,), generator=g, device="cuda")).to(t)}
    if case["op"] == "ln_fwd":
        st["b"] = normal(h, scale=0.1)
        return st
    st["dy"] = normal(r, h)
    if case["op"] == "ln_bwd":
        mean = x.mean(1, dtype=torch.float32)
        var = (x.float() - mean[:, None]).square_().mean(1)
        st.update(mean=mean, rstd=(var + EPS).rsqrt())
    return st


# --------------------------------------------------------------- plain forms --

def _mask(st, x):
    """True where a key is valid, broadcast over [batch, heads, q, k]; None without a mask."""
    case = st["case"]
    if not case["causal"] and not case["ragged"]:
        return None
    j = torch.arange(case["k"], device=x.device)
    mask = torch.ones((1, 1, 1, case["k"]), dtype=torch.bool, device=x.device)
    if st["kv_len"] is not None:
        mask = j < st["kv_len"].long()[:, None, None, None]
    if case["causal"]:
        mask = mask & (_relative(st, x) <= 0)[:, None, _place(case, x)]
    return mask


def _relative(st, x):
    """The positions that a key may have relative to a query, [batch or 1, q + k - 1]."""
    case = st["case"]
    rel = torch.arange(1 - case["q"], case["k"], device=x.device)[None] - st["q_offset"]
    return rel if st["q_start"] is None else rel - st["q_start"].long()[:, None]


def _place(case, x):
    """Where in _relative's answer the pair (query, key) stands, [q, k]."""
    i = torch.arange(case["q"], device=x.device)
    return torch.arange(case["k"], device=x.device) - i[:, None] + case["q"] - 1


def _buckets(rel, buckets, distance, both):
    """The bucket of each relative position: half of the small distances one by
    one, the others by their logarithm up to `distance`.  The logarithm is in
    64 bits and pushed over a border that it lands on."""
    n = -rel
    first = torch.zeros_like(rel)
    if both:
        buckets //= 2
        first = (rel > 0).long() * buckets
        n = n.abs()
    n = n.clamp(min=0)
    near = buckets // 2
    far = torch.log(n.clamp(min=near).double() / near) / math.log(distance / near)
    far = near + (far * (buckets - near) + 1e-9).floor().long()
    return first + torch.where(n < near, n, far.clamp(max=buckets - 1))


def _plain_bias_fwd(st):
    case, x = st["case"], st["x"]
    bucket = _buckets(_relative(st, x), case["buckets"], case["distance"], not case["causal"])
    bias = st["table"].float().t()[:, bucket].transpose(0, 1)[..., _place(case, x)]
    v = x.float() * SCALE + bias
    mask = _mask(st, x)
    if mask is not None:
        v = torch.where(mask, v, float("-inf"))
    top = v.amax(-1, keepdim=True)
    e = torch.exp(v - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(-1, keepdim=True)
    return (e / torch.where(total == 0, 1.0, total)).to(x.dtype)


def _plain_bias_bwd(st):
    case = st["case"]
    y, dy = st["y"].float(), st["dy"].float()
    mask = _mask(st, y)
    if mask is not None:
        dy = torch.where(mask, dy, 0.0)
    ds = y * (dy - (y * dy).sum(-1, keepdim=True))
    bucket = _buckets(_relative(st, y), case["buckets"], case["distance"], not case["causal"])
    # the rows shifted against each other, so that a column holds one relative position
    q, k = case["q"], case["k"]
    shifted = torch.nn.functional.pad(ds.flip(2), (0, q)).flatten(2)[..., :q * (q + k - 1)]
    each = shifted.unflatten(2, (q, q + k - 1)).sum(2, dtype=torch.float64)
    which = (bucket[..., None] == torch.arange(case["buckets"], device=y.device)).double()
    dt = torch.matmul(each, which).sum(0)
    return (ds * SCALE).to(st["y"].dtype), dt.t().float()


def _plain_ln_fwd(st):
    x = st["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * rstd * st["w"].float() + st["b"].float()
    return y.to(st["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_bwd(st):
    dy, x, w = st["dy"].float(), st["x"].float(), st["w"].float()
    layer = st["case"]["op"] == "ln_bwd"
    if layer:
        rstd = st["rstd"][:, None]
        xh = (x - st["mean"][:, None]) * rstd
    else:
        rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        xh = x * rstd
    g = dy * w
    inner = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        inner = inner - g.mean(1, keepdim=True)
    dx = (inner * rstd).to(st["x"].dtype)
    dw = (dy * xh).sum(0)
    return (dx, dw, dy.sum(0)) if layer else (dx, dw)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_bwd, "rms_bwd": _plain_bwd,
                "bias_fwd": _plain_bias_fwd, "bias_bwd": _plain_bias_bwd}[op](state)
    from row_wise_rmsnorm_fwd_gb300 import binding
    t = case["dtype"]
    if op == "ln_fwd":
        fn = binding.layernorm_fwd_f32 if t == "f32" else binding.layernorm_fwd_bf16
        return fn(state["x"], state["w"], state["b"], eps=EPS, stats=True)
    if op == "ln_bwd":
        fn = binding.layernorm_bwd_f32 if t == "f32" else binding.layernorm_bwd_bf16
        return fn(state["dy"], state["x"], state["w"], state["mean"], state["rstd"])
    if op == "rms_bwd":
        fn = binding.rmsnorm_bwd_f32 if t == "f32" else binding.rmsnorm_bwd_bf16
        return fn(state["dy"], state["x"], state["w"], eps=EPS)
    how = dict(max_distance=case["distance"], bidirectional=not case["causal"],
               causal=case["causal"], scale=SCALE, q_offset=state["q_offset"],
               q_start=state["q_start"], kv_len=state["kv_len"])
    if op == "bias_fwd":
        fn = binding.rowsoftmax_relbias_fwd_f32 if t == "f32" else \
            binding.rowsoftmax_relbias_fwd_bf16
        return fn(state["x"], state["table"], **how)
    fn = binding.rowsoftmax_relbias_bwd_f32 if t == "f32" else binding.rowsoftmax_relbias_bwd_bf16
    return fn(state["dy"], state["y"], case["buckets"], **how)


# ------------------------------------------------------------------- 64 bits --

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("bias"):
        return _exact_bias(case, st)
    x = st["x"].double()
    if op == "rms_bwd":
        x.requires_grad_()
        w = st["w"].double().requires_grad_()
        y = w * x / torch.sqrt(torch.einsum("rh,rh->r", x, x) / x.shape[1] + EPS)[:, None]
        return torch.autograd.grad(y, (x, w), st["dy"].double())
    if op == "ln_bwd":
        x.requires_grad_()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    w = st["w"].double().requires_grad_()
    b = (st["b"].double() if op == "ln_fwd" else torch.zeros_like(w)).requires_grad_()
    y = torch.addcmul(b, (x - mean) / torch.sqrt(var + EPS), w)
    if op == "ln_fwd":
        return y.detach(), mean[:, 0], 1 / torch.sqrt(var[:, 0] + EPS)
    return torch.autograd.grad(y, (x, w, b), st["dy"].double())


def _exact_edges(buckets, distance):
    """Smallest distance of each bucket of one direction: exact in whole numbers."""
    near = buckets // 2
    wide = buckets - near
    edges = list(range(near))
    n = near
    for step in range(wide):
        # log(n / near) / log(distance / near) * wide >= step
        while n ** wide * near ** step < distance ** step * near ** wide:
            n += 1
        edges.append(n)
    return edges


def _exact_bias(case, st):
    both = not case["causal"]
    one = case["buckets"] // 2 if both else case["buckets"]
    edges = np.array(_exact_edges(one, case["distance"]))
    kv = [case["k"]] * case["batch"] if st["kv_len"] is None else st["kv_len"].tolist()
    q0 = [st["q_offset"]] * case["batch"] if st["q_start"] is None else st["q_start"].tolist()
    rows, cols = np.arange(case["q"])[:, None], np.arange(case["k"])[None, :]
    outs = []
    dt = torch.zeros((case["buckets"], case["heads"]), dtype=torch.float64, device="cuda")
    for n in range(case["batch"]):
        rel = cols - rows - q0[n]
        away = np.abs(rel) if both else np.maximum(-rel, 0)
        bucket = np.searchsorted(edges, away, side="right") - 1 + (one * (rel > 0) if both else 0)
        keep = np.broadcast_to(cols < kv[n], rel.shape)
        if case["causal"]:
            keep = keep & (rel <= 0)
        keep = torch.from_numpy(np.array(keep)).cuda()
        bucket = torch.from_numpy(bucket).cuda()
        if case["op"] == "bias_fwd":
            v = SCALE * st["x"][n].double() + st["table"].double()[bucket].permute(2, 0, 1)
            total = torch.logsumexp(v.masked_fill(~keep, float("-inf")), -1, keepdim=True)
            outs.append(torch.where(keep, torch.exp(v - total), 0.0))
            continue
        y, dy = st["y"][n].double(), torch.where(keep, st["dy"][n].double(), 0.0)
        ds = y * dy - y * torch.einsum("hqk,hqk->hq", y, dy)[..., None]
        outs.append(SCALE * ds)
        for k in range(case["buckets"]):
            dt[k] += torch.einsum("hqk,qk->h", ds, (bucket == k).double())
    out = torch.stack(outs)
    return out if case["op"] == "bias_fwd" else (out, dt)
