"""linear_blocks detects warps that stop early: bounded waits run out, the kernel ends, and the context stays usable."""
import time

import pytest

from w4a16_compact_expert_gb300 import moe_w4a16 as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K,which", [(T, N, K, i) for T, N, K in ((3, 256, 16384), (16, 130, 5120), (200, 300, 1024),
                                                                      (600, 1000, 2048), (3000, 1500, 512))
                                         for i in range(4 if T > 64 else 3)])
def test_linear_blocks_gives_up_and_the_context_survives(which, T, N, K):
    import torch

    from tests import test_gpu_block_scaled as S
    from w4a16_compact_expert_gb300 import block as B
    act = "swiglu" if T > 64 else "none"
    x, w, xs, ws, _, _ = S.make_linear(T, N, K, act, seed=T)
    assert B.status() == M.OK
    t0 = time.monotonic()
    B.selftest_blocks_timeout(x, w, xs, ws, which, 2_000_000)     # about a millisecond of SM cycles
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 20
    assert B.status() == M.ERR_TIMEOUT
    assert B.status() == M.OK                                     # reported once, then cleared
    pick = [0, T // 2, T - 1]
    out = B.linear_blocks(x, w, xs, ws, act=act, out_dtype=S.E4 if T > 64 else S.F16)
    out = tuple(o[pick] for o in out) if T > 64 else out[pick]
    S.check_linear(x[pick], w, xs[pick], ws, None, None, act, out)
    assert B.status() == M.OK


def test_selftest_refusals():
    from tests import test_gpu_block_scaled as S
    from w4a16_compact_expert_gb300 import block as B
    for T, act, which, limit in ((20, "none", 0, 2000), (3, "none", 3, 2000), (3, "none", -1, 2000), (70, "swiglu", 4, 2000),
                                 (3, "none", 0, 10), (3, "none", 0, (1 << 31) + 1)):
        x, w, xs, ws, _, _ = S.make_linear(T, 128, 1024, act)
        with pytest.raises(M.MoEError):
            B.selftest_blocks_timeout(x, w, xs, ws, which, limit)
