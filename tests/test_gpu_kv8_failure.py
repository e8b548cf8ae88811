"""Failure detection of the 8-bit cache's attention and weights, without a fault, as
for the indexer in test_gpu_failure: their waits are bounded far below the latency
of their copies, so the roles give up, what they have in flight ends, and the host
reads DSA_ERR_TIMEOUT. The same calls at the default bound then give the same bits
as before."""
import pytest
import torch

from test_gpu_kv8 import Paged, SCALE, _attend, _q, _selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_tcgen05_b200 import _build
    _build.build()
    from sparse_attention_long_tcgen05_b200 import dsa
    yield dsa
    dsa.dsa_set_wait_limit_ns(0)


@pytest.mark.parametrize("H,k", [(16, 0), (32, 300), (64, 0), (128, 300), (128, 0)])
def test_waits_that_run_out_are_reported_and_the_context_recovers(dsa, H, k):
    lens = [700, 64, 3000, 129]
    p = Paged(lens, seed=45)
    q = _q(4, H, 130)
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    idx = torch.from_numpy(_selection([n - 1 for n in lens], k, 12)).cuda() if k else None
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))

    def weights(lse):
        acc = torch.zeros(4, p.table.shape[1] * 64, device="cuda")
        dsa.dsa_kv8_accumulate(att, p.d_exps, idx, k, lse, 1.0, acc, ws)
        return acc

    out, lse = _attend(dsa, att, p.d_exps, idx, k, 4, H)
    acc = weights(lse)
    assert dsa.dsa_check_status() == dsa.DSA_OK
    for call in (lambda: _attend(dsa, att, p.d_exps, idx, k, 4, H), lambda: weights(lse)):
        try:
            dsa.dsa_set_wait_limit_ns(1)      # every wait that is not complete at once runs out
            call()
            st = dsa.dsa_check_status()
        finally:
            dsa.dsa_set_wait_limit_ns(0)      # back to the 1 s default
        assert st == dsa.DSA_ERR_TIMEOUT, dsa.status_string(st)
        assert dsa.dsa_check_status() == dsa.DSA_OK
    again, lse2 = _attend(dsa, att, p.d_exps, idx, k, 4, H)
    assert torch.equal(again, out) and torch.equal(lse2, lse) and torch.equal(weights(lse), acc)
    assert dsa.dsa_check_status() == dsa.DSA_OK
