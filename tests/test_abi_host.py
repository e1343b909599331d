"""Host-side checks of the C ABI that need no GPU: the library loads and
exports every entry point the header declares, the host-only helpers
compute what they say, and invalid arguments are rejected before anything
touches CUDA.  Also the activation-checkpoint recorder's bookkeeping, with
fake handles."""
import ctypes
import os
import re

import pytest

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300 import build as cuda_build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_gb300.h")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return B.lib()


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text)))


def test_header_symbols_are_exported(lib):
    names = declared_functions()
    assert len(names) >= 14
    assert sorted(B.EXPORTS) == names
    for n in names:
        assert hasattr(lib, n), f"{n} declared in the header but not exported"


def test_capacity_formula(lib):
    # ceil(cf * s * k / e): the two capacity workloads, and edge cases
    assert B.moe_capacity(1.25, 256, 2, 8) == 80
    assert B.moe_capacity(1.0, 32768, 6, 64) == 3072
    assert B.moe_capacity(1.0, 5000, 6, 64) == 469
    assert B.moe_capacity(1.0, 1, 1, 8) == 1
    assert B.moe_capacity(2.0, 0, 2, 8) == 0
    assert B.moe_capacity(0.0, 10, 2, 8) == 0
    assert B.moe_capacity(-1.0, 10, 2, 8) == 0
    assert B.moe_capacity(1.0, 10, 0, 8) == 0


def test_status_strings(lib):
    for code, name in B.STATUS.items():
        assert isinstance(B.moe_status_string(code), str) and B.moe_status_string(code)
    assert "fp32" in B.moe_status_string(3)


P = ctypes.c_void_p


def rc_name(rc):
    return B.STATUS[rc]


def test_gate_rejects_bad_sizes_without_a_gpu(lib):
    fake = P(0x10000)
    assert rc_name(lib.moe_topk_gate(fake, 4, 8, 9, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # k > e
    assert rc_name(lib.moe_topk_gate(fake, 4, 0, 1, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # e = 0
    assert rc_name(lib.moe_topk_gate(fake, 4, 300, 2, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # e > 256
    assert rc_name(lib.moe_topk_gate(fake, 4, 32, 17, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # k > 16
    assert rc_name(lib.moe_topk_gate(fake, 4, 8, 2, 2, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # renorm
    assert rc_name(lib.moe_topk_gate(None, 4, 8, 2, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # NULL
    assert rc_name(lib.moe_topk_gate(P(0x10004), 4, 8, 2, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"  # align
    assert rc_name(lib.moe_topk_gate(fake, -1, 8, 2, 1, fake, fake, None, None)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_topk_gate(fake, 0, 8, 2, 1, fake, fake, None, None)) == "MOE_OK"  # empty: nothing to do
    assert "min(e, 16)" in lib.moe_last_error().decode()


def test_layout_rejects_bad_sizes_without_a_gpu(lib):
    fake = P(0x10000)
    out = P()
    assert rc_name(lib.moe_dispatch_layout(fake, 4, 8, 2, 0, 3, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"  # R | e
    assert rc_name(lib.moe_dispatch_layout(fake, 4, 8, 2, -1, 0, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch_layout(fake, 4, 256, 2, 0, 128, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch_layout(fake, 4, 8, 9, 0, 0, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch_layout(fake, 2**30, 8, 4, 0, 0, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch_layout(fake, 4, 8, 2, 2**29, 0, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch_layout(fake, 4, 8, 2, 0, 0, None, None)) == "MOE_ERR_INVALID_ARG"
    assert out.value is None
    # send slots need virtual ranks; the flag is 0 or 1
    opt = B.LayoutOptions(0, 0, 0, 1, 1)
    assert rc_name(lib.moe_dispatch_layout_ex(fake, 4, 8, 2, ctypes.byref(opt), None, ctypes.byref(out))) \
        == "MOE_ERR_INVALID_ARG"
    assert "num_virtual_ranks" in lib.moe_last_error().decode()
    opt = B.LayoutOptions(0, 2, 0, 1, 2)
    assert rc_name(lib.moe_dispatch_layout_ex(fake, 4, 8, 2, ctypes.byref(opt), None, ctypes.byref(out))) \
        == "MOE_ERR_INVALID_ARG"
    assert out.value is None
    # an empty handle for in-place builds: the same checks, before any CUDA call
    assert rc_name(lib.moe_layout_create(4, 8, 2, ctypes.byref(B.LayoutOptions(0, 3, 0, 1, 0)), None,
                                         ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_layout_create(4, 8, 9, ctypes.byref(B.LayoutOptions(0, 0, 0, 1, 0)), None,
                                         ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_layout_create(4, 8, 2, None, None, ctypes.byref(out))) == "MOE_ERR_INVALID_ARG"
    assert out.value is None


def test_unknown_handles_are_rejected_without_a_gpu(lib):
    bogus = P(0xdead0)
    fake = P(0x10000)
    assert rc_name(lib.moe_dispatch(None, 4, 8, 8, 0, fake, fake, None)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch(bogus, 4, 8, 8, 0, fake, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_combine(bogus, 4, 8, 8, 1, fake, fake, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_combine_bwd(bogus, 4, 8, 8, 1, fake, fake, fake, fake, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_dispatch_bwd(bogus, 4, 8, 8, 1, fake, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_combine_gate_bwd(bogus, 4, 8, 8, 1, fake, fake, fake, None, 1, fake, fake, fake,
                                            None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_combine_gate_bwd(None, 4, 8, 8, 1, fake, fake, fake, None, 1, fake, fake, fake,
                                            None)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_layout_rebuild(bogus, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_layout_rebuild(None, fake, None)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_topk_gate_layout(bogus, fake, 1, fake, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_grouped_gemm(None, 8, 64, 64, fake, fake, fake, None)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_grouped_gemm(bogus, 8, 64, 64, fake, fake, fake, None)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_dispatch_grouped_gemm(None, 4, 8, 64, 64, fake, fake, fake, None)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_dispatch_grouped_gemm(bogus, 4, 8, 64, 64, fake, fake, fake, None)) \
        == "MOE_ERR_HANDLE_MISMATCH"
    info = B.LayoutInfo()
    assert rc_name(lib.moe_handle_info(bogus, ctypes.byref(info))) == "MOE_ERR_HANDLE_MISMATCH"
    st = ctypes.c_int32()
    assert rc_name(lib.moe_handle_status(bogus, None, ctypes.byref(st))) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_handle_destroy(bogus)) == "MOE_ERR_HANDLE_MISMATCH"
    assert rc_name(lib.moe_handle_destroy(None)) == "MOE_ERR_INVALID_ARG"


def test_debug_hook_arguments(lib):
    assert rc_name(lib.moe_debug_hold_layout_tile(1, 0)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_debug_hold_layout_tile(1, 20000)) == "MOE_ERR_INVALID_ARG"
    assert rc_name(lib.moe_debug_hold_layout_tile(-1, 100)) == "MOE_OK"


def test_launch_counters_exist(lib):
    for name in B.KERNELS:
        assert B.moe_launch_count(name) >= 0
    assert lib.moe_launch_count(99) == 0


# ------------------------------------------------------------- recorder --

class FakeIdx:
    def __init__(self, shape, tag):
        self.shape = shape
        self.tag = tag

    def detach(self):
        return self


def test_recorder_replays_in_call_order_and_falls_back():
    built = []

    def build(idx, e, cap, R):
        h = ("handle", len(built), idx.tag)
        built.append(h)
        return h

    rec = A.HandleRecorder(build=build)
    a, b, c = FakeIdx((8, 2), "a"), FakeIdx((8, 2), "b"), FakeIdx((8, 2), "c")
    fwd = [rec.layout(a, 4), rec.layout(b, 4), rec.layout(c, 4)]
    assert rec.recorded == 3 and len(built) == 3
    rec.replay()
    assert [rec.layout(a, 4), rec.layout(b, 4), rec.layout(c, 4)] == fwd
    assert rec.replayed == 3 and len(built) == 3, "replay must not build layouts"
    extra = rec.layout(a, 4)  # outran the log: a fresh build, not a stale handle
    assert rec.fallbacks == 1 and extra == built[-1] and len(built) == 4


def test_recorder_refuses_a_mismatched_call():
    built = []

    def build(idx, e, cap, R):
        built.append(idx.tag)
        return idx.tag

    rec = A.HandleRecorder(build=build)
    rec.layout(FakeIdx((8, 2), "a"), 4, capacity=3)
    rec.replay()
    # same call position, but a different capacity: never replay a mismatched layout
    assert rec.layout(FakeIdx((8, 2), "z"), 4, capacity=5) == "z"
    assert rec.fallbacks == 1 and rec.replayed == 0


def test_per_call_recorders_keep_passes_apart():
    """One recorder per checkpointed call: three passes through the same block
    route differently and must each replay their own handles."""
    built = []

    def build(idx, e, cap, R):
        built.append(idx.tag)
        return idx.tag

    recs = [A.HandleRecorder(build=build) for _ in range(3)]
    for p, rec in enumerate(recs):
        for layer in range(4):
            rec.layout(FakeIdx((8, 2), f"p{p}l{layer}"), 4)
    n = len(built)
    for p in (2, 0):  # recompute order: later passes first
        recs[p].replay()
        assert [recs[p].layout(FakeIdx((8, 2), "?"), 4) for _ in range(4)] == [f"p{p}l{l}" for l in range(4)]
    assert len(built) == n


def test_recorder_keys_on_layout_options():
    """A replay must match the logged call's layout options too: k-major,
    padding and send slots are part of what was built."""
    built = []

    def build(idx, e, cap, R, **opts):
        built.append((idx.tag, opts))
        return idx.tag

    rec = A.HandleRecorder(build=build)
    rec.layout(FakeIdx((8, 2), "a"), 4, capacity=3, priority="kmajor")
    rec.layout(FakeIdx((8, 2), "b"), 4, pad_multiple=8, send_slots=False)
    assert built[0][1] == {"priority": "kmajor", "pad_multiple": 1, "send_slots": False}
    rec.replay()
    assert rec.layout(FakeIdx((8, 2), "?"), 4, capacity=3, priority="kmajor") == "a"
    # same call position, but token priority this time: rebuilt, not replayed
    assert rec.layout(FakeIdx((8, 2), "c"), 4, pad_multiple=1) == "c"
    assert rec.replayed == 1 and rec.fallbacks == 1


def test_block_calls_reject_bad_arguments_without_a_gpu(lib):
    fake = P(0x10000)
    # layer norm: sizes, dtypes, strides, eps
    ln = lambda s=4, m=8, dt=0, ldx=8, wd=0, eps=1e-5, x=fake: rc_name(
        lib.moe_layernorm(s, m, dt, x, ldx, wd, fake, fake, eps, fake, None, None, None))
    assert ln(s=-1) == ln(m=0) == ln(ldx=7) == ln(eps=0.0) == ln(eps=float("nan")) == ln(x=None) == "MOE_ERR_INVALID_ARG"
    assert ln(dt=2) == ln(wd=2) == ln(dt=-1) == "MOE_ERR_DTYPE"
    assert ln(s=0) == "MOE_OK"
    assert lib.moe_layernorm_bwd_workspace(0, 64) == 0
    assert lib.moe_layernorm_bwd_workspace(5, 64) == 5 * 64 * 8
    bwd = lambda ws: rc_name(lib.moe_layernorm_bwd(4, 8, 0, fake, 8, fake, 8, 0, fake, fake, fake, None, 0, fake, fake, fake,
                                                   fake, ws, None))
    assert bwd(4 * 8 * 8 - 1) == "MOE_ERR_INVALID_ARG" and "workspace" in lib.moe_last_error().decode()
    # balance loss
    bl = lambda s=4, e=8, k=2, n=1, off=None, ws=1 << 30: rc_name(
        lib.moe_balance_loss(fake, fake, None, off, s, e, k, n, fake, fake, fake, fake, fake, fake, fake, ws, None, None))
    assert bl(s=-1) == bl(e=0) == bl(e=257) == bl(k=0) == bl(k=17) == bl(n=0) == bl(n=2) == bl(ws=8) == "MOE_ERR_INVALID_ARG"
    assert lib.moe_balance_loss_workspace(300, 1) == 0 and lib.moe_balance_loss_workspace(8, 4) > 0
    # products
    d = B.LinearDesc(4, 64, 8, 0, 1, 1, 1, 64, 64, 8)
    call = lambda dd: rc_name(lib.moe_linear(ctypes.byref(dd), fake, fake, None, None, fake, None, None, None))
    for field, value in (("s", -1), ("K", 4), ("K", 12), ("N", 0), ("act", 5), ("act", -1), ("ldx", 32), ("ldx", 68), ("ldw", 60)):
        bad = B.LinearDesc(*[value if f == field else getattr(d, f) for f, _ in B.LinearDesc._fields_])
        assert call(bad) == "MOE_ERR_INVALID_ARG", field
    assert call(B.LinearDesc(4, 64, 8, 0, 2, 1, 1, 64, 64, 8)) == "MOE_ERR_DTYPE"
    assert call(B.LinearDesc(0, 64, 8, 0, 1, 1, 1, 64, 64, 8)) == "MOE_OK"
    assert rc_name(lib.moe_linear(None, fake, fake, None, None, fake, None, None, None)) == "MOE_ERR_INVALID_ARG"
    b = B.LinearBwdDesc(4, 64, 8, 0, 2, 1, 1, 8, 64, 64, 8)
    assert rc_name(lib.moe_linear_bwd(ctypes.byref(b), fake, fake, fake, None, fake, fake, fake, fake, 1 << 30, None,
                                      None)) == "MOE_ERR_DTYPE"
    assert lib.moe_linear_bwd_workspace(0, 8) == 0 and lib.moe_linear_bwd_workspace(16, 8) > 0


@pytest.mark.parametrize("dtype", ["uint8", "bool", "int16"])
def test_a_status_word_that_is_too_small_is_refused(lib, dtype):
    # the kernels set bits of four bytes
    import torch

    st = torch.zeros(1, dtype=getattr(torch, dtype))
    x, W = torch.zeros(4, 8).bfloat16(), torch.zeros(3, 8).bfloat16()
    logits, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: B.moe_linear(x, W, device_status=st),
                 lambda: B.moe_linear_bwd(torch.zeros(4, 3).bfloat16(), x, W, device_status=st),
                 lambda: B.moe_balance_loss(logits, idx, device_status=st),
                 lambda: B.moe_topk_gate(logits, 2, device_status=st)):
        with pytest.raises(B.MoEError, match="device_status"):
            call()


def test_a_product_backward_asks_for_the_workspace_it_uses(lib):
    s, N = 512, 264
    need = lambda act=0, dy=1, lddy=N, dx=1, dW=1, db=1: lib.moe_linear_bwd_workspace_for(  # noqa: E731
        ctypes.byref(B.LinearBwdDesc(s, 64, N, act, dy, 1, 1, lddy, 64, 64, N)), dx, dW, db)
    most = lib.moe_linear_bwd_workspace(s, N)
    dz = s * N * 2
    assert need(db=0) == 0 and need(act=4, dx=0, dW=0, db=0) == 0
    assert 0 < need() < dz, "a bf16 dy without an activation is dz itself"
    assert need(act=4, dx=0, dW=0) == need()
    assert need(act=4, db=0) >= dz and need(dy=0, db=0) >= dz and need(lddy=N + 3, db=0) >= dz
    assert need(act=4) == need(act=4, db=0) + need() <= most
    two = lib.moe_linear_bwd_workspace_for(ctypes.byref(B.LinearBwdDesc(s, 64, N, 4, 1, 0, 1, N, 64, 64, N)), 1, 1, 1)
    assert two == need(act=4) + dz == most, "an fp32 result takes dz in two terms"
    assert lib.moe_linear_bwd_workspace_for(None, 1, 1, 1) == 0
    fake = P(0x10000)
    d = B.LinearBwdDesc(s, 64, N, 4, 1, 1, 1, N, 64, 64, N)
    assert rc_name(lib.moe_linear_bwd(ctypes.byref(d), fake, fake, fake, fake, fake, fake, fake, fake, need(act=4) - 1, None,
                                      None)) == "MOE_ERR_INVALID_ARG"
    assert "workspace" in lib.moe_last_error().decode()
