"""Kernels that may start before their forerunner has ended read nothing of it
too early: the expert-parallel steps and the router's gradients back to back in
a captured graph, replayed on new inputs, against the same calls with the
device idle between them."""
import pytest
import torch

from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s,e,k,R,m", [(64, 16, 2, 4, 128), (900, 64, 6, 8, 256), (4096, 128, 8, 8, 512)])
def test_exchange_and_router_gradients_in_a_graph(s, e, k, R, m):
    g = torch.Generator().manual_seed(s)
    rows = s * R  # as many sent rows as there can be
    logits = torch.randn(s, e, generator=g).cuda()
    x = torch.randn(s, m, generator=g).bfloat16().cuda()
    back = torch.randn(rows, k, generator=g).cuda()
    partial = torch.randn(rows, m, generator=g).bfloat16().cuda()
    dloss = torch.tensor([0.1, 0.01], device="cuda")
    h_graph, h_eager = (B.moe_layout_create(s, e, k, num_virtual_ranks=R, send_slots=True) for _ in range(2))

    def chain(h, wait):
        out = []

        def do(*r):
            out.extend(r)
            if wait:
                torch.cuda.synchronize()
            return r

        idx, gate = do(*B.moe_topk_gate_layout(h, logits))
        send_row, _, _ = B.moe_ep_pack(h, gate, rows)  # metadata past the rows sent is left as it was
        do(send_row)
        sent = torch.zeros(rows, m, dtype=x.dtype, device="cuda")
        do(B.moe_ep_dispatch(h, send_row, rows, x, sent))
        do(B.moe_ep_combine(h, send_row, rows, partial))
        dgate, = do(B.moe_ep_unpack_dgate(h, send_row, rows, back))
        dl, = do(B.moe_topk_gate_bwd(logits, idx, gate, dgate, e))
        dgate2, = do(B.moe_ep_unpack_dgate(h, send_row, rows, back * 2))
        do(B.moe_topk_gate_bwd(None, idx, gate, dgate2, e, 1))
        bl = B.moe_balance_loss(logits, idx)
        do(*bl)
        do(B.moe_balance_loss_bwd(logits, bl.lse, bl.coef, bl.norm, dloss, add=dl))
        X, = do(B.moe_dispatch(h, x))
        dY, dgate3 = do(*B.moe_combine_bwd(h, x, gate, X))
        do(B.moe_topk_gate_bwd(logits, idx, gate, dgate3, e))
        do(B.moe_dispatch_bwd(h, dY))
        return out

    chain(h_graph, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(h_graph, False)
    for seed in range(6):
        g = torch.Generator().manual_seed(1000 + seed)
        logits.copy_(torch.randn(s, e, generator=g))
        x.copy_(torch.randn(s, m, generator=g))
        back.copy_(torch.randn(rows, k, generator=g))
        partial.copy_(torch.randn(rows, m, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        want = chain(h_eager, True)
        assert len(have) == len(want)
        for i, (a, c) in enumerate(zip(have, want)):
            assert torch.equal(a, c), i
