"""The give-up path of the shared-prefix attention's kernel, run on a healthy GPU.

Every wait of its warps on one another is bounded.  rmsattn_set_wait_limit(-1)
makes each wait give up where it would go on waiting, so that waits run out while
all that they are for goes on normally; small limits let some through.  The kernel
must then return, give its tensor memory back and set bit 0 of the status word,
and calls with the default bound are right again."""
import pytest
import torch

from test_gpu_attn import make_cache, rand
from test_gpu_step import owns, prefix_state, rn  # noqa: F401  (rn: a fixture)

pytestmark = pytest.mark.gpu

CASES = [([(6, 256)], 4, 1, 64), ([(70, 1024), (3, 64)], 8, 2, 64), ([(6, 256)], 4, 1, 128), ([(65, 1040)], 16, 4, 128),
         ([(40, 320), (9, 640)], 8, 2, 256)]


@pytest.mark.parametrize("limit", [-1, 1000, 2500, 5000])
@pytest.mark.parametrize("groups,Hq,Hk,D", CASES)
def test_wait_that_runs_out_stops_cleanly(rn, groups, Hq, Hk, D, limit):  # noqa: F811
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, 16, D)
    cache = make_cache(rn, t)
    q = rand((lengths.shape[0], Hq, D), 3, torch.bfloat16).cuda()
    want = rn.kv_cache_prefix_attention(q, cache, table, lengths, P, cu)
    torch.cuda.synchronize()
    assert rn.rmsattn_read_status(clear=True) == 0
    hits = 0
    try:
        assert rn.rmsattn_set_wait_limit(limit) == rn.RMSN_OK
        for _ in range(4):
            got = rn.kv_cache_prefix_attention(q, cache, table, lengths, P, cu)
            torch.cuda.synchronize()
            status = rn.rmsattn_read_status(clear=True)
            assert status in (0, rn.RMSATTN_WAIT_RAN_OUT)
            hits += status
            if status == 0:  # nothing gave up: the result is whole
                assert torch.equal(got, want)
    finally:
        rn.rmsattn_set_wait_limit(0)
        rn.rmsattn_read_status(clear=True)
    if limit < 0:
        assert hits == 4
    for _ in range(2):
        assert torch.equal(rn.kv_cache_prefix_attention(q, cache, table, lengths, P, cu), want)
    torch.cuda.synchronize()
    assert rn.rmsattn_read_status() == 0
