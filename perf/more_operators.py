"""Timed cases of what surrounds a decoder layer's blocks and its head: dropout
from a counter-based generator, the join of a block's output with the residual
stream (norm after the block, gate, dropout, residual scale, norm before the
next block) with its gradient, and the log probabilities of given tokens with
entropy and top alternatives, on rows of logits or from hidden states and the
LM head's weights, with their gradients.

``listed()`` and ``draw()`` give cases, ``prepare()`` the data that a training
program has in hand, ``run()`` one pass: in the plain form (elementary torch
operations in 32 bits) or, when ``own`` is true, through the framework's kernel
API on device pointers.  ``exact()`` states the same results in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the embedding rows of a tiny model's step: nothing but latency
        dict(name="dropout-small", op="dropout", rows=256, d=256, dtype="fp32", p=0.1),
        # one 8B-shape layer's activations (batch 8 x 2048)
        dict(name="dropout-8b", op="dropout", rows=16384, d=4096, dtype="bf16", p=0.05),
        # a short prompt of a small model through one join: latency
        dict(name="join-fwd-small", op="join", dir="fwd", rows=8, d=384, h="bf16", post=True, gate=True,
             next=True, p=0.1, alpha=1.0, beta=1.0),
        # one 8B-shape layer with norms on both sides of its blocks and residual dropout
        dict(name="join-fwd-8b", op="join", dir="fwd", rows=16384, d=4096, h="bf16", post=True, gate=False,
             next=True, p=0.1, alpha=1.0, beta=1.0),
        # its gradient, with a gate for each channel too
        dict(name="join-bwd-8b", op="join", dir="bwd", rows=16384, d=4096, h="bf16", post=True, gate=True,
             next=True, p=0.1, alpha=1.0, beta=0.22),
        # a gated block without a norm after it, an odd token count, the block's output in 32 bits
        dict(name="join-bwd-odd", op="join", dir="bwd", rows=5003, d=2048, h="fp32", post=False, gate=True,
             next=True, p=0.05, alpha=1.0, beta=0.5),
        # the widest hidden size, no dropout
        dict(name="join-bwd-wide", op="join", dir="bwd", rows=4095, d=12288, h="bf16", post=True, gate=False,
             next=True, p=0.0, alpha=1.0, beta=1.0),
        # one token of a served request: its log probability and 20 alternatives
        dict(name="logprob-one", op="rows", dir="fwd", rows=1, vocab=128256, pad=0, z="fp32", k=20, scale=1.0),
        # a scored batch at the 8B vocabulary, with temperature
        dict(name="logprob-8b", op="rows", dir="fwd", rows=4096, vocab=128256, pad=0, z="fp32", k=20, scale=0.8),
        # the gradient of a policy loss with an entropy bonus, 16-bit logits, padded tokens
        dict(name="logprob-bwd", op="rows", dir="bwd", rows=4000, vocab=151936, pad=0, z="bf16", k=0, scale=1.0),
        # scoring a batch from its hidden states: 8B width and vocabulary, logits in chunks
        dict(name="lm-logprob-fwd-8b", op="lm", dir="fwd", rows=2048, d=4096, vocab=128256, chunk=1024, scale=1.0),
        # the gradient down to the hidden states and the head's weights, 1.3B width and vocabulary
        dict(name="lm-logprob-bwd", op="lm", dir="bwd", rows=4095, d=2048, vocab=32000, chunk=2048, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "join", "join", "rows", "rows", "lm"])
    p = rng.choice([0.0, 0.05, 0.1, 0.1, 0.5])
    if op == "dropout":
        d = _log(rng, 8, 16384)
        return dict(op=op, rows=_log(rng, 1, min(32768, 16384 * 4096 // d)), d=d,
                    dtype=rng.choice(["bf16", "fp32"]), p=p)
    if op == "join":
        d = 8 * _log(rng, 1, 2048)
        post, nxt = rng.random() < 0.6, rng.random() < 0.8
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), rows=_log(rng, 1, min(32768, 16384 * 4096 // d)), d=d,
                    h=rng.choice(["bf16", "bf16", "fp32"]), post=post, gate=rng.random() < 0.5, next=nxt, p=p,
                    alpha=rng.choice([1.0, 1.0, 0.8]), beta=rng.choice([1.0, 0.22]))
    if op == "rows":
        vocab = _log(rng, 50, 260000)
        way = rng.choice(["fwd", "bwd"])
        return dict(op=op, dir=way, rows=_log(rng, 1, min(16384, 4096 * 128256 // vocab)), vocab=vocab,
                    pad=rng.choice([0, 0, 64]), z=rng.choice(["fp32", "fp32", "bf16"]),
                    k=rng.choice([0, 1, 5, 20, 32]) if way == "fwd" else 0, scale=rng.choice([1.0, 1.0, 0.7, 1.6]))
    way = rng.choice(["fwd", "bwd"])
    d, vocab = 8 * _log(rng, 8, 512), 8 * _log(rng, 32, 16032)
    top = 2 * 2048 * 4096 * 128256 // (2 if way == "fwd" else 6)
    rows = _log(rng, 1, max(2, min(8192, top // (d * vocab))))
    return dict(op=op, dir=way, rows=rows, d=d, vocab=vocab, chunk=rng.choice([512, 1024, 2048]),
                scale=rng.choice([1.0, 0.7]))


def work(case):
    c = case
    if c["op"] == "dropout":
        n = c["rows"] * c["d"]
        return dict(bytes=n * (4 if c["dtype"] == "bf16" else 8), flops=n * 2)
    if c["op"] == "join":
        n, hb = c["rows"] * c["d"], 2 if c["h"] == "bf16" else 4
        gains = 2 * c["d"] * (c["post"] + c["gate"] + c["next"])
        stats = 4 * c["rows"] * (c["post"] + c["next"])
        if c["dir"] == "fwd":
            return dict(bytes=n * (4 + hb + 4 + 2 * c["next"]) + gains + stats, flops=n * 10)
        return dict(bytes=n * (8 + 2 * hb + 8 * c["next"]) + 2 * gains + stats, flops=n * 24)
    zb = 4 if c.get("z", "fp32") == "fp32" else 2
    if c["op"] == "rows":
        n = c["rows"] * c["vocab"]
        if c["dir"] == "fwd":
            return dict(bytes=n * zb + c["rows"] * (16 + 8 * c["k"]), flops=n * 5)
        # a tenth of the rows are padding: only their zeros are written
        live = c["rows"] - c["rows"] // 10
        return dict(bytes=live * c["vocab"] * zb + n * 2 + c["rows"] * 20, flops=live * c["vocab"] * 7)
    n, d, v = c["rows"], c["d"], c["vocab"]
    if c["dir"] == "fwd":
        return dict(bytes=2 * n * d + 2 * v * d + 16 * n, flops=2 * n * d * v + 5 * n * v)
    return dict(bytes=4 * n * d + 4 * v * d + 20 * n, flops=6 * n * d * v + 7 * n * v)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _sampled(z, g):
    """A token of each row, drawn from the softmax of its logits."""
    e = torch.empty(z.shape, device=DEV).exponential_(generator=g)
    return (z.float() - torch.log(e)).argmax(dim=1).int()


def _padding(rows):
    """Every tenth row is padding."""
    return torch.arange(rows, device=DEV) % 10 == 9


def prepare(case, seed):
    c, g = case, _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    new = lambda dt, *s: torch.empty(*s, device=DEV, dtype=dt)
    f32, b16, n = torch.float32, torch.bfloat16, c["rows"]
    st = dict(case=c, seed=(0x9E3779B97F4A7C15 * (seed + 1)) & (2 ** 64 - 1), offset=(5 << 32) + 77 * seed)
    if c["op"] == "dropout":
        st["x"] = rnd(n, c["d"]).to(_type(c["dtype"]))
        st["y"] = torch.empty_like(st["x"])
    elif c["op"] == "join":
        d = c["d"]
        chan = torch.ones(d, device=DEV)  # a residual stream: a few channels are far larger
        chan[torch.randint(0, d, (max(1, d // 512),), generator=g, device=DEV)] = 30.0
        st["x"] = rnd(n, d) * chan
        st["h"] = (0.5 * rnd(n, d)).to(_type(c["h"]))
        for name, there, mean in (("g_post", c["post"], 1.0), ("gate", c["gate"], 0.3), ("g_next", c["next"], 1.0)):
            st[name] = (mean + 0.1 * rnd(d)).bfloat16() if there else None
        st["y"] = new(b16, n, d)
        st["rstd_post"], st["rstd_next"] = new(f32, n), new(f32, n)
        if c["dir"] == "fwd":
            st["xout"] = new(f32, n, d)
        else:
            # what the forward left, and the gradients that come back
            st["xout"], _, st["rstd_post"], st["rstd_next"] = _join_fwd(st)
            del st["x"], st["y"]
            st["dy"] = 0.1 * rnd(n, d) if c["next"] else None
            st["dres"] = 0.1 * rnd(n, d)
            st["dx"], st["dh"] = new(f32, n, d), torch.empty_like(st["h"])
            st["dg_post"], st["dgate"], st["dg_next"] = new(b16, d), new(b16, d), new(b16, d)
    elif c["op"] == "rows":
        v = c["vocab"]
        z = torch.zeros(n, -(-v // 8) * 8 + c["pad"], device=DEV, dtype=_type(c["z"]))
        # logits of a model: broad, with a few candidates far above the rest
        raw = 1.5 * rnd(n, v)
        raw.scatter_add_(1, torch.randint(0, v, (n, 8), generator=g, device=DEV),
                         4.0 + 10.0 * torch.rand(n, 8, generator=g, device=DEV))
        z[:, :v] = raw
        del raw
        st["z"] = z
        st["tokens"] = _sampled(z[:, :v], g)
        st["tokens"][_padding(n)] = -100
        st["logp"], st["lse"], st["entropy"] = new(f32, n), new(f32, n), new(f32, n)
        if c["dir"] == "fwd":
            st["ids"], st["top"] = new(torch.int32, n, c["k"]), new(f32, n, c["k"])
        else:
            _, st["lse"], st["entropy"] = _logp(z[:, :v].float() * c["scale"], st["tokens"])
            _upstream(st, rnd, n)
            st["dz"] = torch.zeros(z.shape, device=DEV, dtype=b16)
    else:
        d, v = c["d"], c["vocab"]
        st["h"] = rnd(n, d).bfloat16()             # normed hidden states
        st["w"] = (1.3 / math.sqrt(d) * rnd(v, d)).bfloat16()
        st["tokens"] = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
        st["tokens"][_padding(n)] = -100
        st["logp"], st["lse"], st["entropy"] = new(f32, n), new(f32, n), new(f32, n)
        if c["dir"] == "bwd":
            _, st["lse"], st["entropy"] = _logp((st["h"].float() @ st["w"].float().t()) * c["scale"], st["tokens"])
            _upstream(st, rnd, n)
            st["dh"], st["dw"] = new(b16, n, d), new(b16, v, d)
    return st


def _upstream(st, rnd, n):
    """Advantages over the batch and an entropy bonus, none on padding."""
    live = (~_padding(n)).float()
    st["dlogp"] = rnd(n) * live / n
    st["dentropy"] = 0.05 * (1 + 0.2 * rnd(n)) * live / n


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the framework's calls
def _scratch(st, dtype, count):
    """Scratch, kept by the program that makes the calls."""
    if "scratch" not in st:
        st["scratch"] = torch.empty(max(1, count), device=DEV, dtype=dtype)
    return st["scratch"].data_ptr()


def _run_own(st):
    import offloaded_fine_tuning_gb300 as sf
    c, s, n = st["case"], torch.cuda.current_stream().cuda_stream, st["case"]["rows"]
    p = lambda k: st[k].data_ptr() if st.get(k) is not None else 0
    if c["op"] == "dropout":
        fmt = sf.F32 if c["dtype"] == "fp32" else sf.BF16
        rc = sf.op_dropout(p("x"), p("y"), fmt, n * c["d"], c["p"], st["seed"], st["offset"], stream=s)
        out = (st["y"],)
    elif c["op"] == "join":
        fmt = sf.F32 if c["h"] == "fp32" else sf.BF16
        drop = (c["alpha"], c["beta"], c["p"], st["seed"], st["offset"])
        if c["dir"] == "fwd":
            rc = sf.op_join_fwd(p("x"), p("h"), fmt, p("g_post"), p("gate"), p("g_next"), *drop, p("xout"),
                                p("y") if c["next"] else 0, p("rstd_post") if c["post"] else 0,
                                p("rstd_next") if c["next"] else 0, n, c["d"], EPS, stream=s)
            out = (st["xout"], st["y"] if c["next"] else None, st["rstd_post"] if c["post"] else None,
                   st["rstd_next"] if c["next"] else None)
        else:
            w = _scratch(st, torch.float32, sf.join_bwd_scratch(n, c["d"]))
            rc = sf.op_join_bwd(p("xout"), p("h"), fmt, p("g_post"), p("gate"), p("g_next"), *drop, p("rstd_post"),
                                p("rstd_next"), p("dy"), p("dres"), p("dx"), p("dh"),
                                p("dg_post") if c["post"] else 0, p("dgate") if c["gate"] else 0,
                                p("dg_next") if c["next"] else 0, w, n, c["d"], stream=s)
            out = (st["dx"], st["dh"], st["dg_post"] if c["post"] else None, st["dgate"] if c["gate"] else None,
                   st["dg_next"] if c["next"] else None)
    elif c["op"] == "rows":
        fmt, ld = sf.F32 if c["z"] == "fp32" else sf.BF16, st["z"].shape[1]
        if c["dir"] == "fwd":
            rc = sf.op_logprob_rows(p("z"), fmt, ld, p("tokens"), n, c["vocab"], c["scale"], p("logp"), p("lse"),
                                    p("entropy"), c["k"], p("ids"), p("top"), stream=s)
            out = (st["logp"], st["lse"], st["entropy"], *((st["ids"], st["top"]) if c["k"] else ()))
        else:
            rc = sf.op_logprob_rows_bwd(p("z"), fmt, ld, p("tokens"), n, c["vocab"], c["scale"], p("lse"),
                                        p("entropy"), p("dlogp"), p("dentropy"), p("dz"), ld, stream=s)
            out = (st["dz"],)
    else:
        d, v = c["d"], c["vocab"]
        if c["dir"] == "fwd":
            w = _scratch(st, torch.uint8, sf.lm_logprob_workspace_bytes(n, v, c["chunk"]))
            rc = sf.op_lm_logprob(p("h"), p("w"), p("tokens"), n, d, v, c["scale"], c["chunk"], w, p("logp"),
                                  p("lse"), p("entropy"), stream=s)
            out = (st["logp"], st["lse"], st["entropy"])
        else:
            w = _scratch(st, torch.uint8, sf.lm_logprob_bwd_workspace_bytes(n, d, v, c["chunk"]))
            rc = sf.op_lm_logprob_bwd(p("h"), p("w"), p("tokens"), n, d, v, c["scale"], c["chunk"], p("lse"),
                                      p("entropy"), p("dlogp"), p("dentropy"), w, p("dh"), p("dw"), stream=s)
            out = (st["dh"], st["dw"])
    if rc != 0:
        raise RuntimeError(f"{c['op']}: status {rc}")
    return [o for o in out if o is not None]


# ------------------------------------------------------------------ the plain form
def _run_plain(st):
    c = st["case"]
    if c["op"] == "dropout":
        return [_drop(st, st["x"].float()).to(st["x"].dtype)]
    if c["op"] == "join":
        out = _join_fwd(st) if c["dir"] == "fwd" else _join_bwd(st)
    elif c["op"] == "rows":
        t = st["z"][:, :c["vocab"]].float() * c["scale"]
        if c["dir"] == "bwd":
            dz = torch.zeros_like(st["dz"])
            dz[:, :c["vocab"]] = _logp_bwd(st, t).bfloat16()
            return [dz]
        logp, lse, entropy = _logp(t, st["tokens"])
        out = logp, lse, entropy
        if c["k"]:
            ids = _top(st["z"][:, :c["vocab"]].float(), c["k"])
            out += ids.int(), torch.gather(t, 1, ids) - lse[:, None]
    else:
        h, w = st["h"].float(), st["w"].float()
        t = (h @ w.t()) * c["scale"]
        if c["dir"] == "fwd":
            out = _logp(t, st["tokens"])
        else:
            dz = _logp_bwd(st, t)
            out = (dz @ w).bfloat16(), (dz.t() @ h).bfloat16()
    return [o for o in out if o is not None]


def _philox(octets, seed, offset):
    """The four 32-bit words of each octet's counter (Philox4x32-10, Salmon et al. 2011)."""
    c = [octets & M32, octets >> 32, torch.full_like(octets, offset & M32), torch.full_like(octets, offset >> 32)]
    key = [seed & M32, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # the low 64 bits; the shifts' masks drop the sign
        c = [((b >> 32) & M32) ^ c[1] ^ key[0], b & M32, ((a >> 32) & M32) ^ c[3] ^ key[1], a & M32]
        key = [(key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32]
    return c


def _threshold(p):
    return round(torch.tensor(p, dtype=torch.float32).item() * 65536)


def _kept(st, shape):
    """Which elements dropout keeps: 16 bits of each against the threshold."""
    n = math.prod(shape)
    words = _philox(torch.arange(-(-n // 8), device=DEV), st["seed"], st["offset"])
    bits = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], dim=1).reshape(-1)[:n]
    return (bits >= _threshold(st["case"]["p"])).reshape(shape)


def _drop(st, u):
    if _threshold(st["case"]["p"]) == 0:
        return u
    return torch.where(_kept(st, u.shape), u * (65536.0 / (65536 - _threshold(st["case"]["p"]))), torch.zeros_like(u))


def _join_fwd(st):
    c, u = st["case"], st["h"].float()
    r1 = y = r2 = None
    if c["post"]:
        r1 = torch.rsqrt((u * u).mean(dim=1) + EPS)
        u = u * r1[:, None] * st["g_post"].float()
    if c["gate"]:
        u = u * st["gate"].float()
    x = c["alpha"] * st["x"] + c["beta"] * _drop(st, u)
    if c["next"]:
        r2 = torch.rsqrt((x * x).mean(dim=1) + EPS)
        y = (x * r2[:, None] * st["g_next"].float()).bfloat16()
    return x, y, r1, r2


def _join_bwd(st):
    c, h = st["case"], st["h"].float()
    big, dgn, dgp, dgt = st["dres"], None, None, None
    if c["next"]:
        xh = st["xout"] * st["rstd_next"][:, None]
        gd = st["dy"] * st["g_next"].float()
        big = big + st["rstd_next"][:, None] * (gd - xh * (gd * xh).mean(dim=1, keepdim=True))
        dgn = (st["dy"] * xh).sum(dim=0, dtype=torch.float64).bfloat16()
    dv = c["beta"] * _drop(st, big)
    hh = h * st["rstd_post"][:, None] if c["post"] else h
    a = (dv * hh).sum(dim=0, dtype=torch.float64)
    w = torch.ones(c["d"], device=DEV)
    if c["gate"]:
        dgt = (a * st["g_post"].double() if c["post"] else a).bfloat16()
        w = w * st["gate"].float()
    if c["post"]:
        dgp = (a * st["gate"].double() if c["gate"] else a).bfloat16()
        w = w * st["g_post"].float()
    dh = w * dv
    if c["post"]:
        dh = st["rstd_post"][:, None] * (dh - hh * (dh * hh).mean(dim=1, keepdim=True))
    return c["alpha"] * big, dh.to(st["h"].dtype), dgp, dgt, dgn


def _logp(t, tokens):
    """Log probability of each row's token (0 where it is negative), lse and entropy."""
    m = t.amax(dim=1, keepdim=True)
    x = t - m
    e = torch.exp(x)
    s = e.sum(dim=1)
    ls = torch.log(s)
    at = torch.gather(x, 1, tokens.clamp(min=0).long()[:, None])[:, 0]
    logp = torch.where(tokens >= 0, at - ls, torch.zeros_like(ls))
    return logp, m[:, 0] + ls, ls - (e * x).sum(dim=1) / s


def _top(z, k):
    """Ids of the k largest of each row, ties by the lowest id: by one whole-number key."""
    bits = z.contiguous().view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)  # in the order of the values; -0 is 0
    key = order * 2 ** 31 + (2 ** 31 - 1 - torch.arange(z.shape[1], device=DEV))
    return torch.topk(key, k, dim=1).indices


def _logp_bwd(st, t):
    c = st["case"]
    lp = t - st["lse"][:, None]
    p = torch.exp(lp)
    dl = torch.where(st["tokens"] >= 0, st["dlogp"], torch.zeros_like(st["dlogp"]))
    d = -p * (dl[:, None] + st["dentropy"][:, None] * (lp + st["entropy"][:, None]))
    d.scatter_add_(1, st["tokens"].clamp(min=0).long()[:, None], dl[:, None])
    return d * c["scale"]


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The results in 64 bits, straight from the definitions."""
    c = case
    if c["op"] == "lm" and work(c)["flops"] > 7e12:  # at about 1 TFLOP/s in 64 bits
        return None
    st = prepare(c, seed)
    out = {"dropout": _exact_dropout, "join": _exact_join, "rows": _exact_rows, "lm": _exact_lm}[c["op"]](c, st)
    return [o for o in out if o is not None]


def _exact_keep(st, shape):
    """The kept elements as weights 0 or 1 / (1 - p): the generator on 16-bit limbs."""
    t = _threshold(st["case"]["p"])
    if t == 0:
        return torch.ones(shape, dtype=torch.float64, device=DEV)
    count = math.prod(shape)
    i = torch.arange((count + 7) // 8, device=DEV)

    def multiply(a, b):
        """High and low 32 bits of a (tensor) times b, by 16-bit limbs."""
        a0, a1, b0, b1 = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
        low = a0 * b0
        mid = a1 * b0 + (low >> 16)
        mid2 = a0 * b1 + (mid & 0xFFFF)
        return a1 * b1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    w0, w1 = i % 2 ** 32, i // 2 ** 32
    w2, w3 = torch.full_like(i, st["offset"] % 2 ** 32), torch.full_like(i, st["offset"] // 2 ** 32)
    for r in range(10):
        ka, kb = (st["seed"] + r * 0x9E3779B9) % 2 ** 32, (st["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        (ha, la), (hb, lb) = multiply(w0, 0xD2511F53), multiply(w2, 0xCD9E8D57)
        w0, w1, w2, w3 = hb ^ w1 ^ ka, lb, ha ^ w3 ^ kb, la
    keep = torch.empty(i.shape[0] * 8, dtype=torch.float64, device=DEV)
    for j, w in enumerate((w0, w1, w2, w3)):
        keep[2 * j::8] = (w % 65536 >= t).double()
        keep[2 * j + 1::8] = (w // 65536 >= t).double()
    return keep[:count].reshape(shape) / (1 - t / 65536)


def _exact_dropout(c, st):
    return (st["x"].double() * _exact_keep(st, st["x"].shape),)


def _exact_join(c, st):
    h, keep = st["h"].double(), _exact_keep(st, st["h"].shape)
    one = torch.ones(c["d"], dtype=torch.float64, device=DEV)
    gp, gt, gn = (st[k].double() if st[k] is not None else one for k in ("g_post", "gate", "g_next"))
    if c["dir"] == "fwd":
        r1 = 1.0 / torch.sqrt((h ** 2).sum(dim=1) / c["d"] + EPS)
        u = h * r1[:, None] * gp if c["post"] else h
        x = c["alpha"] * st["x"].double() + c["beta"] * keep * u * gt
        r2 = 1.0 / torch.sqrt((x ** 2).sum(dim=1) / c["d"] + EPS)
        y = x * r2[:, None] * gn
        return x, y if c["next"] else None, r1 if c["post"] else None, r2 if c["next"] else None
    total = st["dres"].double()
    dgn = None
    if c["next"]:
        r = st["rstd_next"].double()[:, None]
        u, w = st["xout"].double() * r, st["dy"].double() * gn
        total = total + r * (w - u * ((w * u).sum(dim=1, keepdim=True) / c["d"]))
        dgn = (st["dy"].double() * u).sum(dim=0)
    dv = c["beta"] * keep * total
    r = st["rstd_post"].double()[:, None] if c["post"] else 1.0
    u, w = h * r, dv * gp * gt
    dh = r * (w - u * ((w * u).sum(dim=1, keepdim=True) / c["d"])) if c["post"] else w
    sums = (dv * u).sum(dim=0)
    return (c["alpha"] * total, dh, sums * gt if c["post"] else None, sums * gp if c["gate"] else None, dgn)


def _exact_logp(t, tokens):
    lse = torch.logsumexp(t, dim=1)
    lp = t - lse[:, None]
    at = lp[torch.arange(t.shape[0], device=DEV), tokens.long().clamp(min=0)]
    return at * (tokens >= 0), lse, -(torch.exp(lp) * lp).sum(dim=1)


def _exact_grad(c, st, t):
    lp = t - st["lse"].double()[:, None]
    rows = torch.arange(t.shape[0], device=DEV)
    live = (st["tokens"] >= 0).double()
    g = torch.exp(lp)
    g *= -((st["dlogp"].double() * live)[:, None] +
           st["dentropy"].double()[:, None] * (lp + st["entropy"].double()[:, None]))
    g[rows, st["tokens"].long().clamp(min=0)] += st["dlogp"].double() * live
    return g * c["scale"]


def _exact_rows(c, st):
    t = st["z"][:, :c["vocab"]].double() * c["scale"]
    if c["dir"] == "bwd":
        dz = torch.zeros(st["dz"].shape, dtype=torch.float64, device=DEV)
        dz[:, :c["vocab"]] = _exact_grad(c, st, t)
        return (dz,)
    logp, lse, entropy = _exact_logp(t, st["tokens"])
    if not c["k"]:
        return logp, lse, entropy
    values, ids = torch.sort(t, dim=1, descending=True, stable=True)
    return logp, lse, entropy, ids[:, :c["k"]].int(), values[:, :c["k"]] - lse[:, None]


def _exact_lm(c, st):
    h, w = st["h"].double(), st["w"].double()
    t = (h @ w.t()) * c["scale"]
    if c["dir"] == "fwd":
        return _exact_logp(t, st["tokens"])
    g = _exact_grad(c, st, t)
    return g @ w, g.t() @ h
