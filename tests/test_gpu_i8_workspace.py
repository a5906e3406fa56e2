"""A workspace sized for the largest batch in calls with smaller ones."""
import pytest

from test_gpu_i8 import mpq, ops, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("F,K,Ms", [(9728, 16384, (2, 1, 40, 300, 600)), (1371, 2003, (16, 17, 1, 64, 200, 1100)),
                                    (19100, 600, (16, 2, 33, 90, 400))])
def test_largest_batch_first(mpq, F, K, Ms):
    import torch
    top = max(Ms)
    sizes = {"linear": mpq.i8_linear_workspace_size, "gated": mpq.i8_gated_workspace_size,
             "gated_backward": mpq.i8_gated_backward_workspace_size,
             "linear_backward": mpq.i8_linear_backward_workspace_size}
    spaces = {n: torch.zeros(f(top, F, K), dtype=torch.uint8, device="cuda") for n, f in sizes.items()}
    for M in (top,) + Ms:
        for name, call in ops(mpq, M, F, K, M):
            assert same(call(ws=spaces[name]), call()), (name, M)
            mpq.check(spaces[name])


@pytest.mark.parametrize("M,F,K", [(1, 1371, 1001), (9, 2000, 4096), (2, 9728, 2048), (40, 3000, 700), (300, 4001, 1000)])
def test_scratch_may_hold_anything(mpq, M, F, K):
    """Only the first bytes of a workspace have to be zero."""
    import torch
    from block_wise_mixed_b200 import _lib
    for name, call in ops(mpq, M, F, K, 3):
        want = call()
        ws = torch.full((getattr(mpq, "i8_%s_workspace_size" % name)(M, F, K),), 0xFF, dtype=torch.uint8, device="cuda")
        ws[:_lib.I8_WS_ZERO] = 0
        assert same(call(ws=ws), want) and same(call(ws=ws), want), name
        mpq.check(ws)
