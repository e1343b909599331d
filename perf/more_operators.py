"""The operators that train and serve gated experts, as cases to be timed and
compared: the gated projection act(x Wg^T) * (x Wu^T) of a shared expert, the same
over the rows of routed experts, the experts' second product backward, and the
global gradient norm with clipping.

``run`` computes them in plain torch (``own`` false: elementary operations in
fp32, rounded once at the end) or through the library's entry points (``own``
true).  Inputs are drawn on the GPU from the seed alone.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one decoded token through a shared expert: both halves of the weights read once
        dict(name="gated fwd, one token", op="gated", dir="fwd", s=1, K=4096, N=4096, act="silu", bias=False, save_z=False),
        # a serving batch of decoded tokens
        dict(name="gated fwd, decode batch", op="gated", dir="fwd", s=64, K=4096, N=4096, act="silu", bias=False, save_z=False),
        # a shared expert in training: both projections kept for the backward pass
        dict(name="gated fwd, training", op="gated", dir="fwd", s=8192, K=4096, N=8192, act="silu", bias=False, save_z=True),
        # backward of a ragged training batch with biases: gradients of the input, of both halves, of the biases
        dict(name="gated bwd, training", op="gated", dir="bwd", s=6001, K=4096, N=4096, act="gelu_tanh", bias=True, save_z=True),
        # eight decoded tokens through 64 experts, six each, straight from the token rows
        dict(name="experts fwd, decode", op="experts", dir="fwd", s=8, e=64, k=6, K=2048, N=1408, act="silu", zipf=0.0,
             cap=0, gather=True, save_z=False),
        # eight large experts in training, dispatched rows, both projections kept
        dict(name="experts fwd, training", op="experts", dir="fwd", s=8192, e=8, k=2, K=4096, N=4096, act="silu", zipf=0.0,
             cap=0, gather=False, save_z=True),
        # 128 fine-grained experts under skewed routing, backward: segments from a few rows to one for each token
        dict(name="experts bwd, fine-grained skewed", op="experts", dir="bwd", s=16384, e=128, k=8, K=4096, N=512, act="silu",
             zipf=1.5, cap=0, gather=False, save_z=True),
        # the second product of 64 experts in capacity slots, backward: slots past an expert's count hold no route
        dict(name="expert product bwd, capacity", op="product", dir="bwd", s=8192, e=64, k=6, K=1408, N=2048, zipf=1.2, cap=768),
        # the same for a ragged batch without capacity: 128 short segments of odd lengths
        dict(name="expert product bwd, ragged", op="product", dir="bwd", s=2791, e=128, k=8, K=704, N=2816, zipf=0.0, cap=0),
        # the gradients of a router, norms and biases: latency only
        dict(name="clip, small tensors", op="clip", tensors=12, numel=40000, odd=False, dtypes="f32"),
        # a block's gradients as odd pieces of two buckets, bf16 weights and fp32 vectors, none on 16 bytes
        dict(name="clip, odd pieces", op="clip", tensors=301, numel=50000001, odd=True, dtypes="both"),
        # the gradients of several layers of experts
        dict(name="clip, expert weights", op="clip", tensors=48, numel=1200000000, odd=False, dtypes="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eight(v, least=64):
    return max(least, v // 8 * 8)


def draw(rng):
    op = rng.choice(("gated", "gated", "experts", "experts", "product", "clip"))
    if op == "clip":
        numel = _log(rng, 300, 600000000)
        return dict(op=op, tensors=min(_log(rng, 1, 600), numel), numel=numel, odd=rng.random() < 0.5,
                    dtypes=rng.choice(("f32", "bf16", "both")))
    if op == "gated":
        d = rng.choice(("fwd", "fwd", "bwd"))
        s, K = _log(rng, 1, 16384), _eight(_log(rng, 64, 8192))
        N = min(_eight(_log(rng, 64, 16384)), _eight((6001 if d == "bwd" else 8192) * 4096 * 4096 // (s * K)))
        return dict(op=op, dir=d, s=s, K=K, N=N, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                    save_z=d == "bwd" or rng.random() < 0.5)
    e = rng.choice((4, 8, 16, 60, 64, 100, 128, 256))
    k = rng.randint(1, min(8, e))
    s = _log(rng, 1, 16384)
    K = _eight(_log(rng, 64, 4096))
    N = min(_eight(_log(rng, 64, 4096)), _eight(131072 * 4096 * 512 // (s * k * K)), _eight(400000000 // (e * K)))
    zipf = rng.choice((0.0, 0.0, 1.2, 1.5))
    cap = max(1, s * k // e) if rng.random() < 0.3 else 0
    if op == "product":
        return dict(op=op, dir="bwd", s=s, e=e, k=k, K=K, N=N, zipf=zipf, cap=cap)
    d = rng.choice(("fwd", "fwd", "bwd"))
    return dict(op=op, dir=d, s=s, e=e, k=k, K=K, N=N, act=rng.choice(ACTS), zipf=zipf, cap=cap,
                gather=d == "fwd" and rng.random() < 0.5, save_z=d == "bwd" or rng.random() < 0.5)


# ------------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _routes(case, g):
    """idx i32 [s, k] of a router with an expert bias, the row of each kept route's token in expert order, and the
    experts' segments of rows: (first, end) on the host."""
    s, e, k, cap = case["s"], case["e"], case["k"], case["cap"]
    bias = -case["zipf"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    idx = (_randn(g, s, e, dtype=torch.float32) + bias).topk(k, dim=1).indices
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices  # token order within an expert
    counts = torch.bincount(flat, minlength=e).tolist()
    token, segs, at = [], [], 0
    for x in range(e):
        n = min(counts[x], cap) if cap else counts[x]
        token.append(order[at:at + n] // k)
        lo = x * cap if cap else at
        segs.append((lo, lo + n))
        at += counts[x]
    return idx.to(torch.int32).contiguous(), token, segs, e * cap if cap else s * k


def _cut(total, n, odd, seed):
    """n sizes that add up to total: alike, or uneven ones."""
    if odd and total >= 8 * n:
        g = torch.Generator().manual_seed(seed)
        w = torch.empty(n, dtype=torch.float64).uniform_(-3.0, 3.0, generator=g).exp()
        sizes = ((total - n) * w / w.sum()).long() + 1
    else:
        sizes = torch.full((n,), total // n, dtype=torch.int64)
    sizes[-1] += total - int(sizes.sum())
    return sizes.tolist()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "clip":
        # gradients as views of one bucket for each type; channels of different scales
        names = {"f32": ["f32"], "bf16": ["bf16"], "both": ["bf16", "f32"]}[case["dtypes"]]
        names = names[:case["tensors"]]
        st["grads"], st["clipped"], st["flat"], st["flat_out"] = [], [], [], []
        left = case["numel"]
        for i, name in enumerate(names):
            total = left if i == len(names) - 1 else left * 9 // 10
            n = case["tensors"] // len(names) if i else case["tensors"] - (len(names) - 1) * (case["tensors"] // len(names))
            left -= total
            skip = 1 if case["odd"] else 0  # the bucket begins off 16 bytes
            flat = _randn(g, total + skip, dtype=DTYPES[name])[skip:]
            for piece in flat.split(max(1, total // 7)):
                piece.mul_(float(torch.empty(1).uniform_(-4.0, 0.0, generator=torch.Generator().manual_seed(seed + piece.numel()))
                                 .exp()) * 1e-2)
            out = torch.empty(total + skip, device="cuda", dtype=DTYPES[name])[skip:]
            sizes = _cut(total, n, case["odd"], seed)
            st["flat"].append(flat)
            st["flat_out"].append(out)
            st["grads"] += flat.split(sizes)
            st["clipped"] += out.split(sizes)
        st["max_norm"] = 1e-3
        if own:
            from combine_moe_topk_gb300 import binding as B

            st["grads"], st["clipped"] = B.GradList(st["grads"]), B.GradList(st["clipped"])
        return st
    K, N, fwd = case["K"], case["N"], case["dir"] == "fwd"
    if case["op"] == "gated":
        s = case["s"]
        st["x"] = _randn(g, s, K)
        st["W"] = _randn(g, 2 * N, K).mul_(1.0 / math.sqrt(K))
        st["b"] = 0.5 * _randn(g, 2 * N) if case["bias"] else None
        if not fwd:
            st["dh"], st["z"] = _randn(g, s, N), _randn(g, s, 2 * N)
        return st
    idx, token, st["segs"], rows = _routes(case, g)
    x = _randn(g, case["s"], K)
    st["X"] = torch.zeros(rows, K, device="cuda", dtype=torch.bfloat16)  # slots without a route are zeros
    for t, (lo, hi) in zip(token, st["segs"]):
        st["X"][lo:hi] = x[t]
    wide = 2 * N if case["op"] == "experts" else N
    st["W"] = _randn(g, case["e"], wide, K).mul_(1.0 / math.sqrt(K))
    if fwd:
        st["x"] = x
        # rows without a route are left as they were
        st["H"] = torch.zeros(rows, N, device="cuda", dtype=torch.bfloat16)
        st["Z"] = torch.zeros(rows, 2 * N, device="cuda", dtype=torch.bfloat16) if case["save_z"] else None
    else:
        st["dY"] = _randn(g, rows, N)
        st["Z"] = _randn(g, rows, 2 * N) if case["op"] == "experts" else None
        st["dX"] = torch.zeros(rows, K, device="cuda", dtype=torch.bfloat16)
    if own:
        from combine_moe_topk_gb300 import binding as B

        st["h"] = B.moe_dispatch_layout(idx, case["e"], case["cap"])
    return st


# -------------------------------------------------------------- plain forms --

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
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    return torch.ones_like(z)


def _dz(dh, z, act):
    """Gradients of both projections [.., 2N] from that of their product."""
    N = dh.shape[1]
    dh, gate, up = dh.float(), z[:, :N].float(), z[:, N:].float()
    return torch.cat([dh * up * _act_slope(gate, act), dh * _act(gate, act)], 1)


def _gated_fwd(st):
    z = st["x"].float() @ st["W"].float().t()
    if st["b"] is not None:
        z = z + st["b"].float()
    N = st["N"]
    h = (_act(z[:, :N], st["act"]) * z[:, N:]).to(torch.bfloat16)
    return (h, z.to(torch.bfloat16)) if st["save_z"] else (h,)


def _gated_bwd(st):
    dz = _dz(st["dh"], st["z"], st["act"])
    dx, dW = dz @ st["W"].float(), dz.t() @ st["x"].float()
    return (dx.to(torch.bfloat16), dW.to(torch.bfloat16)) + ((dz.sum(0),) if st["bias"] else ())


def _experts_fwd(st):
    N, H, Z = st["N"], st["H"], st["Z"]
    for W, (lo, hi) in zip(st["W"], st["segs"]):
        if hi > lo:
            z = st["X"][lo:hi].float() @ W.float().t()
            H[lo:hi] = _act(z[:, :N], st["act"]) * z[:, N:]
            if Z is not None:
                Z[lo:hi] = z
    return (H,) if Z is None else (H, Z)


def _product_bwd(st):
    """Gradients of the rows and of the weights of Y[r] = X[r] W[x]^T, or of the gated projections."""
    dX, dW = st["dX"], torch.zeros_like(st["W"])
    for x, (lo, hi) in enumerate(st["segs"]):
        if hi > lo:
            d = st["dY"][lo:hi].float() if st["op"] == "product" else _dz(st["dY"][lo:hi], st["Z"][lo:hi], st["act"])
            dX[lo:hi] = d @ st["W"][x].float()
            dW[x] = d.t() @ st["X"][lo:hi].float()
    return dX, dW


def _clip(st):
    f32 = [f.float() for f in st["flat"]]
    norm = sum((f * f).sum(dtype=torch.float64) for f in f32).sqrt().float()
    coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for out, f in zip(st["flat_out"], f32):
        out.copy_(f * coef)
    return (norm.reshape(1), *st["flat_out"])


# --------------------------------------------------------------------- runs --

def run(state):
    st = state
    if not own:
        if st["op"] == "clip":
            return _clip(st)
        if st["op"] == "gated":
            return _gated_fwd(st) if st["dir"] == "fwd" else _gated_bwd(st)
        return _experts_fwd(st) if st["dir"] == "fwd" else _product_bwd(st)

    from combine_moe_topk_gb300 import binding as B

    if st["op"] == "clip":
        return (B.moe_clip_grad_norm(st["grads"], st["max_norm"], out=st["clipped"]), *st["flat_out"])
    if st["op"] == "gated":
        if st["dir"] == "fwd":
            out = B.moe_gated_linear(st["x"], st["W"], st["b"], st["act"], save_z=st["save_z"])
            return out if st["save_z"] else (out,)
        dx, dW, db = B.moe_gated_linear_bwd(st["dh"], st["x"], st["W"], st["z"], st["act"], need_db=st["bias"])
        return (dx, dW, db) if st["bias"] else (dx, dW)
    if st["dir"] == "fwd":
        f, x = (B.moe_dispatch_grouped_gated, st["x"]) if st["gather"] else (B.moe_grouped_gated, st["X"])
        out = f(st["h"], x, st["W"], st["act"], H=st["H"], Z=st["Z"], save_z=st["save_z"])
        return out if st["save_z"] else (out,)
    if st["op"] == "experts":
        return B.moe_grouped_gated_bwd(st["h"], st["dY"], st["X"], st["W"], st["Z"], st["act"], dX=st["dX"])
    return B.moe_grouped_gemm_bwd(st["h"], st["dY"], st["X"], st["W"], dX=st["dX"])


# --------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "clip":
        size = {"f32": 4.0, "bf16": 2.0, "both": 2.2}[case["dtypes"]]
        return {"bytes": 2 * size * case["numel"], "flops": 3 * case["numel"]}
    K, N, s = case["K"], case["N"], case["s"]
    if case["op"] == "gated":
        if case["dir"] == "fwd":
            return {"bytes": 2 * s * K + 4 * N * K + 2 * s * N * (3 if case["save_z"] else 1) + 4 * N * case["bias"],
                    "flops": 4 * s * K * N}
        return {"bytes": 6 * s * N + 4 * s * K + 8 * N * K + 8 * N * case["bias"], "flops": 8 * s * K * N}
    e, rows = case["e"], s * case["k"]
    if case["cap"]:
        rows = min(rows, e * case["cap"])
    active = e * (1.0 - (1.0 - case["k"] / e) ** s)  # experts that some token takes, under even routing
    if case["op"] == "experts" and case["dir"] == "fwd":
        x = min(s, rows) if case["gather"] else rows
        return {"bytes": 2 * x * K + 4 * active * N * K + 2 * rows * N * (3 if case["save_z"] else 1), "flops": 4 * rows * K * N}
    wide = 2 * N if case["op"] == "experts" else N
    dz = 6 * rows * N if case["op"] == "experts" else 2 * rows * N
    return {"bytes": dz + 4 * rows * K + 2 * (active + e) * wide * K, "flops": 4 * rows * K * wide}


# -------------------------------------------------------------------- exact --

def exact(case, seed):
    """The same outputs from the definitions in 64 bits; gradients by differentiating them.  None where the products
    would take too long in 64 bits."""
    if case["op"] != "clip" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    d = lambda t: t.double()  # noqa: E731
    if case["op"] == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for f in st["flat"]:
            for part in f.split(1 << 26):
                total = total + torch.dot(d(part), d(part))
        norm = torch.sqrt(total)
        scale = min(1.0, st["max_norm"] / (float(norm) + 1e-6))
        return (norm.reshape(1), *(torch.mul(d(f), scale) for f in st["flat"]))
    fn = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"), "silu": torch.nn.functional.silu}

    def glu(z):
        gate, up = z.chunk(2, dim=1)
        return fn[case["act"]](gate) * up

    if case["op"] == "gated":
        if case["dir"] == "fwd":
            z = torch.einsum("sk,nk->sn", d(st["x"]), d(st["W"]))
            z = z if st["b"] is None else z + d(st["b"])
            return (glu(z), z) if case["save_z"] else (glu(z),)
        z = d(st["z"]).requires_grad_(True)
        dz, = torch.autograd.grad(glu(z), z, d(st["dh"]))
        dx, dW = torch.einsum("sn,nk->sk", dz, d(st["W"])), torch.einsum("sn,sk->nk", dz, d(st["x"]))
        return (dx, dW, dz.sum(0)) if case["bias"] else (dx, dW)
    if case["dir"] == "fwd":
        Z = torch.zeros(st["X"].shape[0], 2 * case["N"], dtype=torch.float64, device="cuda")
        for x, (lo, hi) in enumerate(st["segs"]):
            Z[lo:hi] = torch.einsum("rk,nk->rn", d(st["X"][lo:hi]), d(st["W"][x]))
        return (glu(Z), Z) if case["save_z"] else (glu(Z),)
    if case["op"] == "experts":
        z = d(st["Z"]).requires_grad_(True)
        D, = torch.autograd.grad(glu(z), z, d(st["dY"]))
    else:
        D = d(st["dY"])
    dX, dW = torch.zeros(st["X"].shape, dtype=torch.float64, device="cuda"), []
    for x, (lo, hi) in enumerate(st["segs"]):
        dX[lo:hi] = torch.einsum("rn,nk->rk", D[lo:hi], d(st["W"][x]))
        dW.append(torch.einsum("rn,rk->nk", D[lo:hi], d(st["X"][lo:hi])))
    return dX, torch.stack(dW)
