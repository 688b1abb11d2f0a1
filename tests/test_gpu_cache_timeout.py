"""The bounded waits of spec_cache_attend give up cleanly (GPU, through the C ABI).

Every wait between the launch's warps is bounded. With a limit of a few polls nearly every one runs out while copies and
products are under way: the launch still returns, sets SV_ERR_TIMEOUT and nothing else, and the next call on the same
workspace is as it always was. Outputs of a launch that gave up are undefined, but stay within their rows. No fault is
injected: the waits simply stop early.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache import Batch, tree

pytestmark = pytest.mark.gpu

TIMEOUT = 1 << 7


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


# every CTA has several items of 12 tiles: the next one's queries wait for longer than a poll lasts (4 us)
@pytest.mark.parametrize("limit", [1, 2, 5])
@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("B,tokens,group,trees", [(140, 1, 4, False), (140, 6, 4, False), (70, 8, 8, False), (60, 40, 4, False),
                                                  (60, 32, 4, True)])
def test_waits_that_run_out_end_the_launch(sc, B, tokens, group, trees, kind, cache, limit):
    from speculative_decoding_verification_35_gb300.specverify import SvDebug
    rng = np.random.default_rng(1)
    par = [tree(rng, tokens) for _ in range(B)] if trees else None
    b = Batch(sc, [tokens] * B, [1500] * B, 8 * group, 8, 128, 32, kind, cache, parents=par)
    want, wl = b.attend()
    torch.cuda.synchronize()
    assert b.cache.status_bits() == 0
    room = torch.full((want.numel() + 2 * 4096,), 7.0, dtype=want.dtype, device="cuda")
    out = room[4096:-4096].view(want.shape)
    lse = torch.empty_like(wl)
    debug = SvDebug()
    debug.spin_limit = limit
    c = b.cache
    code = {"bf16": sc.SV_BF16, "fp16": sc.SV_F16}[kind]
    gave_up = 0
    for _ in range(3):
        assert sc.spec_cache_attend_ex(c.struct, 0, b.chunk.struct, code, b.hq, b.q.data_ptr(), b.q.stride(0), b.D ** -0.5, 0,
                                       out.data_ptr(), lse.data_ptr(), c.status.data_ptr(), c.workspace.data_ptr(), c.ws_bytes,
                                       debug, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()  # the launch returned
        st = c.status_bits()
        assert st & ~TIMEOUT == 0
        gave_up += st != 0
        c.status.zero_()
        if not st:  # nothing ran out
            assert torch.equal(out, want) and torch.equal(lse, wl)
        assert (room[:4096] == 7).all() and (room[-4096:] == 7).all()
        again, al = b.attend()
        torch.cuda.synchronize()
        assert c.status_bits() == 0 and torch.equal(again, want) and torch.equal(al, wl)
    assert gave_up == 3 or limit > 1
