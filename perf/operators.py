"""The operators around the MoE token path, as cases to be timed and compared:
the layer norm in front of the block, the router's balance loss, and the dense
products with their epilogue (router projection, shared expert), each in both
directions.

``run`` computes them in plain torch (``own`` false: elementary operations in
fp32, rounded once at the end) or through the library's entry points (``own``
true).  Inputs are drawn on the GPU from the seed alone.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one decoded token through the block's norm: latency only
        dict(name="norm fwd, one token", op="norm", dir="fwd", s=1, m=4096, dtype="bf16", affine="bf16", dres=False),
        # the norm of a large training batch, backward: the residual branch's gradient joins in
        dict(name="norm bwd, training batch", op="norm", dir="bwd", s=16384, m=4096, dtype="bf16", affine="bf16", dres=True),
        # a ragged batch of an odd width in fp32 (rows not of 16 bytes), fp32 weights
        dict(name="norm bwd, odd width", op="norm", dir="bwd", s=2791, m=2815, dtype="f32", affine="f32", dres=False),
        # an 8-expert router's loss over one training batch
        dict(name="balance fwd, 8 experts", op="balance", dir="fwd", s=8192, e=8, k=2, seqs=1, masked=0.0, zipf=0.0),
        # the largest router: 256 experts, packed ragged sequences with padding, skewed routing
        dict(name="balance fwd, packed", op="balance", dir="fwd", s=131072, e=256, k=8, seqs=37, masked=0.1, zipf=1.2),
        # the gradient into the router's logits, fine-grained experts, skewed, added to the gate's gradient
        dict(name="balance bwd, fine-grained", op="balance", dir="bwd", s=16384, e=128, k=8, seqs=4, masked=0.05, zipf=1.5),
        # one decoded token through a shared expert's second product, residual added: reads the weights once
        dict(name="linear fwd, one token", op="linear", dir="fwd", s=1, K=4096, N=4096, act="none", bias=True, res=True,
             out="bf16", save_z=False),
        # a serving batch of decoded tokens through the first product
        dict(name="linear fwd, decode batch", op="linear", dir="fwd", s=64, K=4096, N=4096, act="silu", bias=True, res=False,
             out="bf16", save_z=False),
        # the router's projection: few columns, fp32 logits out
        dict(name="linear fwd, router", op="linear", dir="fwd", s=16384, K=4096, N=128, act="none", bias=False, res=False,
             out="f32", save_z=False),
        # the shared expert's first product in training: activation, z kept for the backward pass
        dict(name="linear fwd, shared expert", op="linear", dir="fwd", s=8192, K=4096, N=16384, act="gelu", bias=True,
             res=False, out="bf16", save_z=True),
        # a ragged batch, odd number of columns, residual
        dict(name="linear fwd, ragged", op="linear", dir="fwd", s=2791, K=2816, N=2815, act="gelu_tanh", bias=True, res=True,
             out="bf16", save_z=False),
        # backward of a training product: three gradients
        dict(name="linear bwd, training", op="linear", dir="bwd", s=8192, K=4096, N=4096, act="silu", bias=True, res=False,
             out="bf16", save_z=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "balance", "balance", "linear", "linear", "linear"))
    if op == "norm":
        s = _log(rng, 1, 16384)
        m = _log(rng, 64, min(16384, 16384 * 4096 // s))
        if rng.random() < 0.5:
            m = max(64, m // 8 * 8)
        dtype = rng.choice(("bf16", "f32"))
        d = rng.choice(("fwd", "bwd"))
        return dict(op=op, dir=d, s=s, m=m, dtype=dtype, affine=rng.choice((dtype, "f32")),
                    dres=d == "bwd" and rng.random() < 0.5)
    if op == "balance":
        s, e = _log(rng, 1, 131072), rng.choice((2, 5, 8, 16, 24, 60, 64, 100, 128, 160, 255, 256))
        return dict(op=op, dir=rng.choice(("fwd", "bwd")), s=s, e=e, k=rng.randint(1, min(8, e)),
                    seqs=rng.choice((1, 1, _log(rng, 2, 64))), masked=rng.choice((0.0, 0.05, 0.3)),
                    zipf=rng.choice((0.0, 1.2, 1.5)))
    d = rng.choice(("fwd", "fwd", "bwd"))
    most = 8192 * 4096 * (4096 if d == "bwd" else 16384)
    s = _log(rng, 1, 16384)
    K = max(64, _log(rng, 64, 8192) // 8 * 8)
    N = max(1, min(_log(rng, 8, 16384), most // (s * K)))
    if rng.random() < 0.6:
        N = max(8, N // 8 * 8)
    act = rng.choice(ACTS)
    return dict(op=op, dir=d, s=s, K=K, N=N, act=act, bias=rng.random() < 0.7, res=d == "fwd" and rng.random() < 0.5,
                out=rng.choice(("bf16", "bf16", "f32")) if d == "fwd" else "bf16",
                save_z=(act != "none") if d == "bwd" else act != "none" and rng.random() < 0.5)


# ------------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _offsets(case, seed):
    """Packed sequences of uneven lengths covering all tokens, int32 [seqs + 1]."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, case["s"] + 1, (case["seqs"] - 1,), generator=g).sort().values
    ends = torch.tensor([case["s"]])
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, ends]).to(torch.int32).cuda()


def _sequence_of(offsets, s):
    return torch.searchsorted(offsets[1:].long().contiguous(), torch.arange(s, device=offsets.device), right=True)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "norm":
        s, m, dt = case["s"], case["m"], DTYPES[case["dtype"]]
        # residual-stream rows: a common offset, and a few channels far larger than the rest
        chan = 1.0 + 8.0 * (torch.rand(m, generator=g, device="cuda") < 0.01)
        st["x"] = (_randn(g, s, m) * chan + 0.25).to(dt)
        st["w"] = (1.0 + 0.2 * _randn(g, m)).to(DTYPES[case["affine"]])
        st["b"] = (0.1 * _randn(g, m)).to(DTYPES[case["affine"]])
        if case["dir"] == "bwd":
            xf = st["x"].float()
            st["mean"] = xf.mean(1)
            st["rstd"] = 1.0 / ((xf - st["mean"][:, None]).square().mean(1) + EPS).sqrt()
            st["dy"] = _randn(g, s, m).to(dt)
            st["res"] = _randn(g, s, m).to(dt) if case["dres"] else None
        return st
    if case["op"] == "balance":
        s, e, k = case["s"], case["e"], case["k"]
        bias = -case["zipf"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
        st["logits"] = _randn(g, s, e) + bias
        st["idx"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
        st["valid"] = ((torch.rand(s, generator=g, device="cuda") >= case["masked"]).to(torch.uint8)
                       if case["masked"] else None)
        st["offsets"] = _offsets(case, seed) if case["seqs"] > 1 else None
        if case["dir"] == "bwd":
            _, _, _, st["lse"], st["coef"], st["norm"] = _balance(st)
            st["dloss"] = torch.tensor([0.01, 0.001], device="cuda")
            st["dgate"] = 0.1 * _randn(g, s, e) / s  # the router's gradient from the gate, to be added
        return st
    s, K, N = case["s"], case["K"], case["N"]
    st["x"] = _randn(g, s, K).to(torch.bfloat16)
    st["W"] = (_randn(g, N, K) / math.sqrt(K)).to(torch.bfloat16)
    st["b"] = (0.5 * _randn(g, N)).to(torch.bfloat16) if case["bias"] else None
    if case["dir"] == "fwd":
        st["res"] = _randn(g, s, N).to(torch.bfloat16) if case["res"] else None
    else:
        st["dy"] = _randn(g, s, N).to(torch.bfloat16)
        st["z"] = _randn(g, s, N).to(torch.bfloat16) if case["save_z"] else None
    return st


# -------------------------------------------------------------- plain forms --

def _norm_fwd(st):
    x = st["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    y = (x - mean) * rstd * st["w"].float() + st["b"].float()
    return y.to(st["x"].dtype), mean[:, 0], rstd[:, 0]


def _norm_bwd(st):
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xh = (st["x"].float() - st["mean"][:, None]) * rstd
    g = dy * st["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if st["res"] is not None:
        dx = dx + st["res"].float()
    return dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _balance(st):
    """loss [2], counts [B, e], mean probabilities [B, e], and what the backward pass keeps."""
    logits, idx = st["logits"], st["idx"].long()
    s, e = logits.shape
    k, dev = idx.shape[1], logits.device
    live = torch.ones(s, device=dev) if st["valid"] is None else st["valid"].float()
    if st["offsets"] is None:
        B, seq = 1, torch.zeros(s, dtype=torch.int64, device=dev)
    else:
        B, seq = st["offsets"].numel() - 1, _sequence_of(st["offsets"], s)
    top = logits.max(1, keepdim=True).values
    ex = (logits - top).exp()
    tot = ex.sum(1, keepdim=True)
    p = ex / tot * live[:, None]
    lse = (top + tot.log())[:, 0] * live
    T = torch.zeros(B, device=dev).index_add_(0, seq, live)
    some = (T > 0).float()
    T1 = T.clamp(min=1.0)[:, None]
    mean_p = torch.zeros(B, e, device=dev).index_add_(0, seq, p) / T1
    counts = torch.zeros(B * e, dtype=torch.int64, device=dev).index_add_(
        0, (seq[:, None] * e + idx).reshape(-1), live.long()[:, None].expand(s, k).reshape(-1)).view(B, e)
    frac = counts.float() / (k * T1)
    per_seq, inv_tokens = 1.0 / some.sum().clamp(min=1.0), 1.0 / T.sum().clamp(min=1.0)
    loss = torch.stack([e * (frac * mean_p).sum() * per_seq, lse.square().sum() * inv_tokens])
    return loss, counts.to(torch.int32), mean_p, lse, e * frac / T1, torch.stack([per_seq, inv_tokens])


def _balance_bwd(st):
    logits, lse, coef = st["logits"], st["lse"], st["coef"]
    s = logits.shape[0]
    p = (logits - lse[:, None]).exp()
    c = coef * (st["dloss"][0] * st["norm"][0])
    c = c if st["offsets"] is None else c[_sequence_of(st["offsets"], s)]
    d = p * (c - (c * p).sum(1, keepdim=True) + (2.0 * st["dloss"][1] * st["norm"][1]) * lse[:, None])
    if st["valid"] is not None:
        d = torch.where(st["valid"][:, None] != 0, d, torch.zeros_like(d))
    return st["dgate"] + d


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    sg = 1.0 / (1.0 + torch.exp(-z))
    return sg * (1.0 + z * (1.0 - sg))


def _linear_fwd(st):
    z = st["x"].float() @ st["W"].float().t()
    if st["b"] is not None:
        z = z + st["b"].float()
    y = _act(z, st["act"])
    if st["res"] is not None:
        y = y + st["res"].float()
    y = y.to(DTYPES[st["out"]])
    return (y, z.to(torch.bfloat16)) if st["save_z"] else (y,)


def _linear_bwd(st):
    dz = st["dy"].float()
    if st["act"] != "none":
        dz = dz * _act_slope(st["z"].float(), st["act"])
    dx, dW = dz @ st["W"].float(), dz.t() @ st["x"].float()
    return (dx.to(torch.bfloat16), dW.to(torch.bfloat16)) + ((dz.sum(0),) if st["bias"] else ())


# --------------------------------------------------------------------- runs --

def run(state):
    st = state
    if not own:
        if st["op"] == "norm":
            return _norm_fwd(st) if st["dir"] == "fwd" else _norm_bwd(st)
        if st["op"] == "balance":
            return _balance(st)[:4] if st["dir"] == "fwd" else _balance_bwd(st)
        return _linear_fwd(st) if st["dir"] == "fwd" else _linear_bwd(st)

    from combine_moe_topk_gb300 import binding as B

    if st["op"] == "norm":
        if st["dir"] == "fwd":
            return B.moe_layernorm(st["x"], st["w"], st["b"], EPS)
        return B.moe_layernorm_bwd(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], dres=st["res"])
    if st["op"] == "balance":
        if st["dir"] == "fwd":
            r = B.moe_balance_loss(st["logits"], st["idx"], valid=st["valid"], seq_offsets=st["offsets"])
            return r.loss, r.counts, r.mean_prob, r.lse
        return B.moe_balance_loss_bwd(st["logits"], st["lse"], st["coef"], st["norm"], st["dloss"], valid=st["valid"],
                                      seq_offsets=st["offsets"], add=st["dgate"])
    if st["dir"] == "fwd":
        out = B.moe_linear(st["x"], st["W"], bias=st["b"], act=st["act"], residual=st["res"], out_dtype=DTYPES[st["out"]],
                           save_z=st["save_z"])
        return out if st["save_z"] else (out,)
    dx, dW, db = B.moe_linear_bwd(st["dy"], st["x"], st["W"], z=st["z"], act=st["act"], need_db=st["bias"])
    return (dx, dW, db) if st["bias"] else (dx, dW)


# --------------------------------------------------------------------- work --

def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "norm":
        s, m, n, a = case["s"], case["m"], size[case["dtype"]], size[case["affine"]]
        if case["dir"] == "fwd":
            return {"bytes": 2 * s * m * n + 2 * m * a + 8 * s, "flops": 8 * s * m}
        return {"bytes": (3 + case["dres"]) * s * m * n + m * a + 8 * m + 8 * s, "flops": 14 * s * m}
    if case["op"] == "balance":
        s, e, k, B = case["s"], case["e"], case["k"], case["seqs"]
        mask = s if case["masked"] else 0
        if case["dir"] == "fwd":
            return {"bytes": s * (4 * e + 4 * k + 4) + 8 * B * e + mask, "flops": 6 * s * e}
        return {"bytes": s * (12 * e + 4) + 4 * B * e + mask, "flops": 8 * s * e}
    s, K, N = case["s"], case["K"], case["N"]
    if case["dir"] == "fwd":
        out = s * N * (size[case["out"]] + 2 * case["res"] + 2 * case["save_z"])
        return {"bytes": 2 * s * K + 2 * N * K + 2 * N * case["bias"] + out, "flops": 2 * s * K * N}
    return {"bytes": 2 * s * N * (1 + case["save_z"]) + 4 * s * K + 4 * N * K + 4 * N * case["bias"], "flops": 4 * s * K * N}


# -------------------------------------------------------------------- exact --

def exact(case, seed):
    """The same outputs from the definitions in 64 bits; gradients by differentiating them."""
    st = prepare(case, seed)
    d = lambda t: t.double()  # noqa: E731
    if case["op"] == "norm":
        x = d(st["x"]).requires_grad_(case["dir"] == "bwd")
        w, b = d(st["w"]).requires_grad_(case["dir"] == "bwd"), d(st["b"]).requires_grad_(case["dir"] == "bwd")
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(b, (x - mean) * rstd, w)
        if case["dir"] == "fwd":
            return y, mean[:, 0], rstd[:, 0]
        dx, dw, db = torch.autograd.grad(y, (x, w, b), d(st["dy"]))
        return (dx if st["res"] is None else dx + d(st["res"])), dw, db
    if case["op"] == "balance":
        s, e, k = case["s"], case["e"], case["k"]
        logits = d(st["logits"]).requires_grad_(case["dir"] == "bwd")
        lse, p = torch.logsumexp(logits, 1), torch.softmax(logits, 1)
        live = torch.ones(s, dtype=torch.bool, device="cuda") if st["valid"] is None else st["valid"].bool()
        ends = [0, s] if st["offsets"] is None else st["offsets"].tolist()
        counts, mean_p, terms = [], [], []
        for lo, hi in zip(ends[:-1], ends[1:]):
            at = live[lo:hi]
            n = max(1, int(at.sum()))
            c = torch.bincount(st["idx"][lo:hi][at].reshape(-1).long(), minlength=e)
            m = p[lo:hi][at].sum(0) / n
            counts.append(c)
            mean_p.append(m)
            if int(at.sum()):
                terms.append(e * (c.double() / (k * n) * m).sum())
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        loss = sum(terms, zero) / max(1, len(terms))
        z = lse[live].square().sum() / max(1, int(live.sum()))
        if case["dir"] == "fwd":
            return (torch.stack([loss, z]), torch.stack(counts).to(torch.int32), torch.stack(mean_p),
                    torch.where(live, lse, torch.zeros_like(lse)))
        if not terms:
            return d(st["dgate"])
        grad, = torch.autograd.grad(0.01 * loss + 0.001 * z, logits)
        return d(st["dgate"]) + grad
    x, W = d(st["x"]), d(st["W"])
    fn = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"), "silu": torch.nn.functional.silu}[case["act"]]
    if case["dir"] == "fwd":
        z = torch.einsum("sk,nk->sn", x, W)
        z = z if st["b"] is None else z + d(st["b"])
        y = fn(z) if st["res"] is None else fn(z) + d(st["res"])
        return (y, z) if case["save_z"] else (y,)
    dz = d(st["dy"])
    if case["act"] != "none":
        z = d(st["z"]).requires_grad_(True)
        dz, = torch.autograd.grad(fn(z), z, dz)
    dx, dW = torch.einsum("sn,nk->sk", dz, W), torch.einsum("sn,sk->nk", dz, x)
    return (dx, dW, dz.sum(0)) if case["bias"] else (dx, dW)
