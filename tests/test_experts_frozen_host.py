"""The gathering experts' product with frozen weights: its backward pass needs no dispatched
rows.  Without a GPU: the library's calls are replaced."""
import pytest
import torch

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B


class FakeHandle:
    s, e, rows, raw, gaps = 4, 3, 8, None, False


@pytest.mark.parametrize("need_x,need_w", [(True, False), (False, True), (True, True)])
def test_rows_are_dispatched_again_only_for_the_weights(monkeypatch, need_x, need_w):
    log, bf = [], torch.bfloat16
    h = FakeHandle()

    def fwd(h, x, W, act, save_z=False):
        return torch.zeros(8, 16, dtype=bf), torch.zeros(8, 32, dtype=bf)

    def bwd(h, dH, X, W, Z, act="silu", need_dx=True, need_dw=True):
        log.append(("bwd", X is None, need_dx, need_dw))
        return torch.zeros(8, 64, dtype=bf) if need_dx else None, torch.zeros(3, 32, 64, dtype=bf) if need_dw else None

    monkeypatch.setattr(B, "moe_dispatch_grouped_gated", fwd)
    monkeypatch.setattr(B, "moe_grouped_gated_bwd", bwd)
    monkeypatch.setattr(B, "moe_dispatch", lambda h, x: log.append(("dispatch",)) or torch.zeros(8, 64, dtype=bf))
    monkeypatch.setattr(B, "moe_dispatch_bwd", lambda h, dX: log.append(("dispatch_bwd",)) or torch.zeros(4, 64, dtype=bf))
    x = torch.zeros(4, 64, dtype=bf, requires_grad=need_x)
    W = torch.zeros(3, 32, 64, dtype=bf, requires_grad=need_w)
    A.dispatch_grouped_gated(x, W, h).float().sum().backward()
    want = [("dispatch",)] * need_w + [("bwd", not need_w, need_x, need_w)] + [("dispatch_bwd",)] * need_x
    assert log == want


def test_the_binding_takes_no_rows_where_only_their_gradient_is_needed(monkeypatch):
    """X may be None without dW: rows come from the handle, K from W."""
    seen, bf, h = [], torch.bfloat16, FakeHandle()

    class Lib:
        moe_grouped_gated_bwd_workspace = staticmethod(lambda rows, N: 0)
        moe_grouped_gated_bwd = staticmethod(lambda raw, rows, K, N, act, dH, X, W, Z, dX, dW, *rest: seen.append((rows, K, N, X, dW)) or 0)
        moe_grouped_gemm_bwd = staticmethod(lambda raw, rows, K, N, dY, X, W, dX, dW, *rest: seen.append((rows, K, N, X, dW)) or 0)

    monkeypatch.setattr(B, "lib", lambda: Lib)
    W, dH, Z = torch.zeros(3, 32, 64, dtype=bf), torch.zeros(8, 16, dtype=bf), torch.zeros(8, 32, dtype=bf)
    dX, dW = B.moe_grouped_gated_bwd(h, dH, None, W, Z, need_dw=False)
    assert dX.shape == (8, 64) and dX.dtype == bf and dW is None
    dX, dW = B.moe_grouped_gemm_bwd(h, Z, None, W, need_dw=False)
    assert dX.shape == (8, 64) and dW is None
    assert seen == [(8, 64, 16, None, None), (8, 64, 32, None, None)]
    for call in (lambda: B.moe_grouped_gated_bwd(h, dH, None, W, Z), lambda: B.moe_grouped_gemm_bwd(h, Z, None, W),
                 lambda: B.moe_grouped_gated_bwd(h, dH, None, W[:2], Z, need_dw=False),
                 lambda: B.moe_grouped_gated_bwd(h, dH, None, W.float(), Z, need_dw=False),
                 lambda: B.moe_grouped_gated_bwd(h, dH[:4], None, W, Z, need_dw=False)):
        with pytest.raises(B.MoEError):
            call()
    assert len(seen) == 2
