"""The smoke run launches every kernel family that it stands for."""
import pytest

import __graft_entry__ as G
from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu
FAMILIES = ["topk_gate", "layout", "dispatch", "combine", "combine_bwd", "dispatch_bwd", "topk_gate_bwd", "grouped_gemm",
            "dispatch_gemm", "layernorm", "layernorm_bwd", "balance", "balance_bwd", "linear", "linear_bwd"]


def test_smoke_runs_the_token_path_and_what_stands_around_it():
    before = {k: B.moe_launch_count(k) for k in FAMILIES}
    G.smoke()
    assert all(B.moe_launch_count(k) > n for k, n in before.items()), before
