"""The 8-bit latent cache at the edges of its ranges, on the GPU: queries up to
the largest bf16 value.

Where two calls must give the same bits, a power of two has only been moved from
one factor to another. Other tolerances are those of test_gpu_kv8."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K
from test_gpu_kv8 import Paged, _attend, _close, _q, _selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_tcgen05_b200 import _build
    _build.build()
    from sparse_attention_long_tcgen05_b200 import dsa
    return dsa


def _weights(dsa, att, exps, idx, k, lse, n_seq, width):
    acc = torch.zeros(n_seq, width, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))
    dsa.dsa_kv8_accumulate(att, exps, idx, k, lse, 1.0, acc, ws)
    return acc


def _expected(q, keysets, scale):
    """Output, lse and sum p|v| of each query, and the largest logit that counts
    (the others are past e^-60 of the query's largest)."""
    got, zm = [], 0.0
    for qi, rows in zip(q, keysets):
        o, l, p = K.attend(qi, rows, scale)
        got.append((o, l, p @ np.abs(rows[:, :512])))
        if len(rows):
            z = scale * (qi @ rows.T)
            zm = max(zm, float(np.abs(z[z > z.max(axis=1, keepdims=True) - 60]).max()))
    return (*(np.stack(x) for x in zip(*got)), zm)


@pytest.mark.parametrize("H,k", [(16, 0), (32, 100), (64, 0), (128, 100)])
def test_queries_up_to_the_largest_bf16(dsa, H, k):
    """A head whose largest element is 2^125, 2^126, 2^127 or 255/256 * 2^128, with
    the softmax scale as much smaller: the bits of the ordinary head."""
    lens = [130, 700, 65]
    p = Paged(lens, seed=40, gain=1 / 16)
    q = _q(3, H, 110)
    q[0, 0, 5], q[1, H - 1, 575] = 7.96875, -7.96875
    d_idx = torch.from_numpy(_selection([n - 1 for n in lens], k, 7)).cuda() if k else None
    width = p.table.shape[1] * 64
    ref = None
    for g in (0, 122, 123, 124, 125):
        big = (q.float() * 2.0 ** g).to(torch.bfloat16)
        assert torch.isfinite(big).all()
        att = dsa.attn_in(big, p.d_codes, 2.0 ** (-1 - g), 512, kv_layout=p.layout(dsa))
        out, lse = _attend(dsa, att, p.d_exps, d_idx, k, 3, H)
        acc = _weights(dsa, att, p.d_exps, d_idx, k, lse, 3, width)
        assert dsa.dsa_check_status() == 0
        if ref is None:
            ref = out, lse, acc
            sets = [p.rows(b, d_idx[b].cpu().numpy()[d_idx[b].cpu().numpy() >= 0] if k else np.arange(n))
                    for b, n in enumerate(lens)]
            _close(out, lse, *_expected(q.double().cpu().numpy(), sets, 0.5))
        for a, b in zip(ref, (out, lse, acc)):
            assert torch.equal(a, b), g
