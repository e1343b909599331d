"""The gated products, the experts' backward pass and clipping without a GPU: what
the library refuses before anything touches CUDA, the binding's own checks, the
autograd wrappers over plain torch forms, and clipping over gloo ranks."""
import ctypes
import os

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300 import build as cuda_build
from combine_moe_topk_gb300 import ep as EP

P = ctypes.c_void_p
OK, ARG, DTYPE, MISMATCH = 0, 1, 3, 4
AT = 0x10000  # an address that only the checks see


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return B.lib()


def gated(lib, x=AT, W=AT, bias=None, h=AT, z=None, status=None, **kw):
    d = dict(s=4, K=64, N=32, act=4, bias_dtype=0, ldx=64, ldw=64)
    d.update(kw)
    return lib.moe_gated_linear(B.GatedDesc(**d), x, W, bias, h, z, status, None)


@pytest.mark.parametrize("bad", [dict(s=-1), dict(K=4), dict(K=60), dict(K=0), dict(K=(1 << 18) + 8), dict(N=0), dict(N=12),
                                 dict(N=(1 << 29) + 8), dict(s=(1 << 30) + 1), dict(act=5), dict(act=-1), dict(ldx=56),
                                 dict(ldx=68), dict(ldw=60), dict(x=None), dict(x=AT + 8), dict(W=None), dict(h=None),
                                 dict(h=AT + 4), dict(z=AT + 2), dict(bias=AT + 4), dict(status=AT + 2)])
def test_gated_linear_refuses(lib, bad):
    assert gated(lib, **bad) == ARG
    assert lib.moe_last_error()


def test_gated_linear_takes_no_rows_and_refuses_a_bias_type(lib):
    assert gated(lib, s=0, x=None, W=None, h=None) == OK
    assert gated(lib, bias=AT, bias_dtype=2) == DTYPE
    assert lib.moe_gated_linear(None, AT, AT, None, AT, None, None, None) == ARG


def gated_bwd(lib, dh=AT, x=AT, W=AT, z=AT, dx=AT, dW=AT, db=AT, ws=AT, size=1 << 30, status=None, **kw):
    d = dict(s=4, K=64, N=32, act=4, dh_dtype=1, dx_dtype=1, dw_dtype=1, lddh=32, ldx=64, ldw=64, ldz=64)
    d.update(kw)
    return lib.moe_gated_linear_bwd(B.GatedBwdDesc(**d), dh, x, W, z, dx, dW, db, ws, size, status, None)


@pytest.mark.parametrize("bad", [dict(lddh=24), dict(lddh=36), dict(ldz=56), dict(ldz=68), dict(ldx=56), dict(ldw=60),
                                 dict(dh=None), dict(x=None), dict(W=None), dict(z=None), dict(dx=AT + 2), dict(dW=AT + 8),
                                 dict(db=AT + 4), dict(ws=None), dict(ws=AT + 8), dict(size=100), dict(N=20), dict(act=9)])
def test_gated_linear_bwd_refuses(lib, bad):
    assert gated_bwd(lib, **bad) == ARG


@pytest.mark.parametrize("bad", [dict(dh_dtype=2), dict(dx_dtype=2), dict(dw_dtype=-1)])
def test_gated_linear_bwd_refuses_types(lib, bad):
    assert gated_bwd(lib, **bad) == DTYPE


def test_gated_linear_bwd_with_nothing_to_do(lib):
    assert gated_bwd(lib, dx=None, dW=None, db=None, dh=None, x=None, W=None, z=None, ws=None, size=0) == OK
    assert gated_bwd(lib, s=0, dW=None, db=None, ws=None, size=0) == OK


def test_workspaces(lib):
    def size(dx=1, dW=1, db=1, **kw):
        d = dict(s=100, K=64, N=32, act=4, dh_dtype=1, dx_dtype=1, dw_dtype=1, lddh=32, ldx=64, ldw=64, ldz=64)
        d.update(kw)
        return lib.moe_gated_linear_bwd_workspace(B.GatedBwdDesc(**d), dx, dW, db)

    assert size(db=0) == 100 * 64 * 2
    assert size(db=0, dx_dtype=0) == 2 * 100 * 64 * 2  # dz in two terms
    assert size(dx=0, dW=0, db=0) == 0 and size(s=0) == 0
    assert 0 < size(dx=0, dW=0) < size()
    assert lib.moe_grouped_gated_bwd_workspace(10, 32) == 10 * 64 * 2 and lib.moe_grouped_gated_bwd_workspace(0, 32) == 0
    assert lib.moe_grad_norm_workspace(0) > 0
    assert lib.moe_grad_norm_workspace(1025) == 2 * lib.moe_grad_norm_workspace(1024) == 2 * lib.moe_grad_norm_workspace(1)


def test_handles_are_looked_up(lib):
    for h, want in ((None, ARG), (P(AT), MISMATCH)):
        assert lib.moe_grouped_gated(h, 4, 64, 32, 4, AT, AT, AT, None, None) == want
        assert lib.moe_dispatch_grouped_gated(h, 4, 4, 64, 32, 4, AT, AT, AT, None, None) == want
        assert lib.moe_grouped_gemm_bwd(h, 4, 64, 32, AT, AT, AT, AT, AT, None) == want
        assert lib.moe_grouped_gated_bwd(h, 4, 64, 32, 4, AT, AT, AT, AT, AT, AT, AT, 1 << 20, None) == want


def create(lib, *tensors, count=None):
    spec = (B.Tensor * max(1, len(tensors)))(*(B.Tensor(*t) for t in tensors))
    out = P()
    return lib.moe_tensor_list_create(spec, len(tensors) if count is None else count, ctypes.byref(out)), out


@pytest.mark.parametrize("t,want", [((None, 4, 0), ARG), ((AT, -1, 0), ARG), ((AT, 1 << 43, 0), ARG), ((AT + 2, 4, 0), ARG),
                                    ((AT + 1, 4, 1), ARG), ((AT, 4, 2), DTYPE), ((AT, 4, -1), DTYPE)])
def test_lists_refuse(lib, t, want):
    assert create(lib, t)[0] == want
    assert create(lib, (None, 0, 0), t)[0] == want


def test_lists_without_tensors_and_their_end(lib):
    assert create(lib, count=-1)[0] == ARG
    assert lib.moe_tensor_list_create(None, 1, ctypes.byref(P())) == ARG
    assert lib.moe_tensor_list_create(None, 0, None) == ARG
    rc, raw = create(lib)
    assert rc == OK
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None), dict(norm=AT + 2)):
        kw = dict(max_norm=1.0, norm=AT) | bad
        assert lib.moe_clip_grad_norm(raw, None, kw["max_norm"], kw["norm"], AT, 1 << 20, None, None) == ARG
        assert lib.moe_grad_clip(raw, None, kw["norm"], kw["max_norm"], None) == ARG
    assert lib.moe_tensor_list_destroy(raw) == OK
    assert lib.moe_tensor_list_destroy(raw) == MISMATCH
    assert lib.moe_grad_norm(raw, AT, AT, 1 << 20, None, None) == MISMATCH
    assert lib.moe_grad_clip(None, None, AT, 1.0, None) == MISMATCH


def test_the_binding_checks_shapes_and_types():
    bf = torch.bfloat16
    x, W = torch.zeros(4, 64, dtype=bf), torch.zeros(64, 64, dtype=bf)
    for call in (lambda: B.moe_gated_linear(x, W[:63]), lambda: B.moe_gated_linear(x, W[:, :56]),
                 lambda: B.moe_gated_linear(x.float(), W), lambda: B.moe_gated_linear(x, W, act="tanh"),
                 lambda: B.moe_gated_linear(x, W, torch.zeros(32)), lambda: B.moe_gated_linear(x, W, h=torch.zeros(4, 32)),
                 lambda: B.moe_gated_linear_bwd(torch.zeros(4, 31, dtype=bf), x, W, torch.zeros(4, 64, dtype=bf)),
                 lambda: B.moe_gated_linear_bwd(torch.zeros(4, 32, dtype=bf), x, W, torch.zeros(4, 32, dtype=bf)),
                 lambda: B.moe_gated_linear(x, W)):  # host memory
        with pytest.raises(B.MoEError):
            call()
    with pytest.raises(ValueError):
        B.moe_gated_linear(x[None], W)
    with pytest.raises(ValueError):
        B.moe_gated_linear(x[:1].expand(4, 64), W)


class FakeHandle:
    s, e, rows, raw = 4, 3, 8, None


def test_the_binding_checks_the_experts_operands():
    bf, h = torch.bfloat16, FakeHandle()
    x, X, W, H = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, dtype=bf), torch.zeros(3, 32, 64, dtype=bf), torch.zeros(8, 16, dtype=bf)
    Z = torch.zeros(8, 32, dtype=bf)
    for call in (lambda: B.moe_grouped_gated(h, X, W[:2]), lambda: B.moe_grouped_gated(h, X, W[:, :31]),
                 lambda: B.moe_grouped_gated(h, x, W), lambda: B.moe_dispatch_grouped_gated(h, X, W),
                 lambda: B.moe_grouped_gated(h, X.float(), W), lambda: B.moe_grouped_gated(h, X, W, "swish"),
                 lambda: B.moe_grouped_gated(h, X, W, H=Z), lambda: B.moe_grouped_gated(h, X, W, save_z=True, Z=H),
                 lambda: B.moe_grouped_gemm_bwd(h, H, X, W), lambda: B.moe_grouped_gemm_bwd(h, Z.float(), X, W),
                 lambda: B.moe_grouped_gemm_bwd(h, Z, X, W, dX=x), lambda: B.moe_grouped_gemm_bwd(h, Z, X, W, dW=W[:2]),
                 lambda: B.moe_grouped_gated_bwd(h, Z, X, W, Z), lambda: B.moe_grouped_gated_bwd(h, H, X, W, H)):
        with pytest.raises(B.MoEError):
            call()


def test_lists_of_the_binding_check_memory(lib):
    t = torch.zeros(4, 6)
    for bad in (t[:, ::2], t[:1].expand(4, 6), torch.zeros(3).to_sparse()):
        with pytest.raises(ValueError):
            B.GradList([bad])
    for bad in ([t], [t.half()], [t.long()]):  # host memory; types
        with pytest.raises(B.MoEError):
            B.GradList(bad)
    assert B._dense(t.t()) and B._dense(torch.zeros(2, 3, 4).permute(1, 2, 0)) and B._dense(torch.zeros(()))
    assert not B._dense(torch.as_strided(t, (3, 3), (2, 1)))


# ---- autograd over plain torch forms ----------------------------------------------

def _gated(x, W, act):
    g, u = (x.float() @ W.float().transpose(-1, -2)).chunk(2, -1)
    return torch.relu(g) * u, torch.cat([g, u], -1).bfloat16()


def _gated_bwd(dh, x, W, z):
    g, u = z.float().chunk(2, -1)
    dz = torch.cat([dh.float() * u * (g > 0), dh.float() * torch.relu(g)], -1)
    return dz


@pytest.fixture
def calls(monkeypatch):
    """One expert whose rows are all of them, so that the experts' calls are the dense ones."""
    log = []

    def fake(name, fn):
        def call(*args, **kw):
            log.append((name, args, kw))
            return fn(*args, **kw)

        monkeypatch.setattr(B, name, call)

    def fwd(x, W, bias=None, act="silu", save_z=False, **kw):
        h, z = _gated(x, W, act)
        return (h.to(x.dtype), z) if save_z else h.to(x.dtype)

    def bwd(dh, x, W, z, act="silu", need_dx=True, need_dw=True, need_db=True, **kw):
        dz = _gated_bwd(dh, x, W, z)
        return ((dz @ W.float()).to(x.dtype) if need_dx else None, (dz.t() @ x.float()).to(W.dtype) if need_dw else None,
                dz.sum(0) if need_db else None)

    def products(dY, X, W, need_dx, need_dw):
        return ((dY.float() @ W[0].float()).to(X.dtype) if need_dx else None,
                (dY.float().t() @ X.float()).to(W.dtype)[None] if need_dw else None)

    fake("moe_gated_linear", fwd)
    fake("moe_gated_linear_bwd", bwd)
    for name in ("moe_grouped_gated", "moe_dispatch_grouped_gated"):
        fake(name, lambda h, x, W, act="silu", save_z=False: fwd(x, W[0], act=act, save_z=save_z))
    fake("moe_grouped_gated_bwd", lambda h, dH, X, W, Z, act="silu", need_dx=True, need_dw=True:
         products(_gated_bwd(dH, X, W, Z), X, W, need_dx, need_dw))
    fake("moe_grouped_gemm", lambda h, X, W: (X.float() @ W[0].float().t()).to(X.dtype))
    fake("moe_grouped_gemm_bwd", lambda h, dY, X, W, need_dx=True, need_dw=True: products(dY, X, W, need_dx, need_dw))
    fake("moe_dispatch", lambda h, x: x * 1.0)
    fake("moe_dispatch_bwd", lambda h, dX: dX * 1.0)
    return log


def leaf(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).requires_grad_()


CALLS = {
    "gated_linear": lambda x, W: A.gated_linear(x, W[0], act="relu"),
    "grouped_gated": lambda x, W: A.grouped_gated(x, W, None, "relu"),
    "dispatch_grouped_gated": lambda x, W: A.dispatch_grouped_gated(x, W, None, "relu"),
    "grouped_gemm": lambda x, W: A.grouped_gemm(x, W, None),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_first_derivatives_and_no_second(calls, name):
    x, W = leaf(4, 8), leaf(1, 12, 8, seed=1)
    y = CALLS[name](x, W).float().square().sum()
    dx, dW = torch.autograd.grad(y, (x, W))
    assert dx.shape == x.shape and dW.shape == W.shape and torch.isfinite(dx).all()
    y = CALLS[name](x, W).float().square().sum() + x.square().sum()
    g, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.square().sum(), x)


def test_inference_keeps_no_projections(calls):
    x, W = leaf(4, 8).detach(), leaf(1, 12, 8, seed=1)
    for name in sorted(CALLS)[:3]:
        saved = []
        for grad in (True, False):
            calls.clear()
            with torch.set_grad_enabled(grad):
                CALLS[name](x, W)
            saved += [kw["save_z"] for n, _, kw in calls if "save_z" in kw]
        assert saved == [True, False], name
    W.requires_grad_(False)
    calls.clear()
    A.gated_linear(x, W[0])
    assert not calls[0][2]["save_z"]


def test_only_the_gradients_that_are_needed(calls):
    for name, at in (("grouped_gated", 5), ("dispatch_grouped_gated", 5), ("grouped_gemm", 4)):
        x, W = leaf(4, 8).detach(), leaf(1, 12, 8, seed=1)
        calls.clear()
        CALLS[name](x, W).float().sum().backward()
        back = [a for n, a, _ in calls if n.endswith("_bwd") and "dispatch_bwd" not in n]
        assert len(back) == 1 and back[0][-2:] == (False, True), name
        assert not any(n == "moe_dispatch_bwd" for n, _, _ in calls)


# ---- clipping over ranks ------------------------------------------------------------

class _List(list):
    tensors = property(lambda self: list(self))


def _rank(rank, R, port, q):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=R)
    try:
        B.GradList = _List
        B.moe_grad_norm = lambda g: torch.stack([t.double().square().sum() for t in g]).sum().sqrt().float().view(1)

        def clip(g, norm, max_norm, out=None):
            for t in g:
                t.mul_(min(1.0, max_norm / (float(norm) + 1e-6)))

        B.moe_grad_clip = clip
        g = torch.Generator().manual_seed(rank)
        own, common = [torch.randn(5, generator=g), torch.randn(3, 2, generator=g)], [torch.arange(4.0)]
        before = [t.clone() for t in own + common]
        norm = EP.clip_grad_norm(own, common, 0.5)
        q.put((rank, float(norm), [b.numpy() for b in before], [t.numpy() for t in own + common]))
    finally:
        dist.destroy_process_group()


def test_one_norm_over_ranks():
    R, ctx = 2, mp.get_context("spawn")
    q = ctx.Queue()
    port = 30700 + os.getpid() % 1000
    procs = [ctx.Process(target=_rank, args=(r, R, port, q)) for r in range(R)]
    for p in procs:
        p.start()
    got = sorted(q.get(timeout=300) for _ in procs)
    for p in procs:
        p.join(timeout=120)
        assert p.exitcode == 0
    total = sum(float((b.astype("f8") ** 2).sum()) for r in got for b in r[2][:2]) + float((got[0][2][2].astype("f8") ** 2).sum())
    for _, norm, before, after in got:
        assert abs(norm - total ** 0.5) < 1e-5
        for b, a in zip(before, after):
            assert abs(a - b * (0.5 / (total ** 0.5 + 1e-6))).max() < 1e-6
