"""The 8-bit latent cache's calls as a server makes them, on the GPU: a whole step in
one captured graph, replayed as the sequences grow; pages beyond 4 GiB; a chunk of a
prompt that takes several passes; rows that hold NaN. Tolerances are those of
test_gpu_kv8."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K
from test_gpu_kv8 import Paged, SCALE, _attend, _close, _q, _reference, _selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_tcgen05_b200 import _build
    _build.build()
    from sparse_attention_long_tcgen05_b200 import dsa
    return dsa


@pytest.mark.parametrize("k", [0, 64])
def test_a_captured_step_follows_the_lengths(dsa, k):
    """Store, attention and weights of a step, captured once on a side stream: each
    replay gives the bits of the same calls made one by one at those lengths."""
    lens, H, steps = [126, 640, 63, 1], 32, 4
    n = len(lens)
    state = []
    for _ in range(2):
        p = Paged([x + steps for x in lens], seed=50)
        p.d_ctx.copy_(torch.tensor(lens))
        state.append((p, torch.zeros(n, p.table.shape[1] * 64, device="cuda")))
    rows, q = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda"), _q(n, H, 0)
    idx = torch.empty(n, max(k, 1), dtype=torch.int32, device="cuda")
    out = [torch.empty(n, H, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lse = [torch.empty(n, H, device="cuda") for _ in range(2)]

    def att_of(p):
        return dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))

    ws = [dsa.workspace(max(dsa.dsa_workspace_size(op, None, att_of(state[0][0]), 0, 0, k)
                            for op in (dsa.DSA_OP_KV8_MQA, dsa.DSA_OP_KV8_ACCUMULATE))) for _ in range(2)]

    def step(i):
        p, acc = state[i]
        p.d_ctx.add_(1)
        dsa.dsa_kv8_store(dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa)), rows)
        att = att_of(p)
        dsa.dsa_kv8_mqa_fwd(att, p.d_exps, idx if k else None, k, out[i], lse[i], ws[i])
        dsa.dsa_kv8_accumulate(att, p.d_exps, idx if k else None, k, lse[i], 0.9, acc, ws[i])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):                         # (captured, not run)
        step(0)
    for t in range(steps):
        rows.copy_(_q(n, 1, 60 + t, gain=2.0 ** t)[:, 0])
        q.copy_(_q(n, H, 70 + t))
        if k:
            idx.copy_(torch.from_numpy(_selection([x + t for x in lens], k, t)))
        graph.replay()
        step(1)
        assert dsa.dsa_check_status() == 0
        (a, acc_a), (b, acc_b) = state
        assert torch.equal(a.d_codes, b.d_codes) and torch.equal(a.d_exps, b.d_exps) and torch.equal(a.d_ctx, b.d_ctx)
        assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1]) and torch.equal(acc_a, acc_b)
        assert torch.isfinite(out[0]).all() and torch.isfinite(lse[0]).all()


def test_a_captured_eviction(dsa):
    lens, budget = [300, 64, 900], 128
    p = Paged(lens, seed=51, extra=6)
    dst = torch.tensor([p.free[0:2], p.free[2:4], p.free[4:6]], dtype=torch.int32, device="cuda")
    acc = torch.zeros(3, p.table.shape[1] * 64, device="cuda")
    kept = torch.empty(3, budget, dtype=torch.int32, device="cuda")
    acc_out, n = torch.zeros(3, budget, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    cache = dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dsa.dsa_kv8_evict(cache, acc, budget, 4, 20, dst, n, kept, acc_out)
    for t in range(3):
        acc.copy_(torch.rand(acc.shape, generator=torch.Generator().manual_seed(t)))
        graph.replay()
        assert dsa.dsa_check_status() == 0
        for b, x in enumerate(lens):
            keep = K.keep(acc[b].cpu().numpy(), x, budget, 4, 20)
            assert kept[b].tolist() == keep + [-1] * (budget - len(keep)) and n[b].item() == len(keep)


def test_pages_beyond_4_gib(dsa):
    """A pool of 120,000 pages (4.4 GB): the rows of the last pages are written, read,
    weighed and moved at byte offsets past 2^32."""
    total, lens, H = 120000, [200, 70], 16
    p = Paged(lens, seed=52, extra=4)
    used = p.num_pages
    shift = total - used                                  # the same pages, at the pool's end
    codes = torch.zeros(total, 64, 576, dtype=torch.uint8, device="cuda")
    exps = torch.zeros(total, dtype=torch.int8, device="cuda")
    codes[shift:], exps[shift:] = p.d_codes, p.d_exps
    table = p.d_table + torch.where(p.d_table >= 0, shift, 0).to(torch.int32)
    lay = dsa.paged_layout(table, p.d_ctx, total)
    rows = torch.randn(2, 576, generator=torch.Generator().manual_seed(1))
    want_c, want_e = K.store(p.codes, p.exps, rows.double().numpy(), [0, 1], [x - 1 for x in lens], p.table)
    dsa.dsa_kv8_store(dsa.kv8_cache(codes, exps, lay), rows.cuda())
    assert dsa.dsa_check_status() == 0
    assert np.array_equal(codes[shift:].cpu().numpy(), want_c) and np.array_equal(exps[shift:].cpu().numpy(), want_e)
    p.codes, p.exps = want_c, want_e
    q = _q(2, H, 140)
    att = dsa.attn_in(q, codes, SCALE, 512, kv_layout=lay)
    out, lse = _attend(dsa, att, exps, None, 0, 2, H)
    sets = [p.rows(b, np.arange(n)) for b, n in enumerate(lens)]
    _close(out, lse, *_reference(q.double().cpu().numpy(), sets))
    acc = torch.zeros(2, table.shape[1] * 64, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, 0))
    dsa.dsa_kv8_accumulate(att, exps, None, 0, lse, 1.0, acc, ws)
    assert abs(acc.sum().item() - 2) < 1e-3
    dst = torch.tensor([[f + shift for f in p.free[2 * b:2 * b + 2]] for b in range(2)], dtype=torch.int32, device="cuda")
    kept = torch.empty(2, 100, dtype=torch.int32, device="cuda")
    acc_out, n = torch.zeros(2, 128, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    dsa.dsa_kv8_evict(dsa.kv8_cache(codes, exps, lay), acc, 100, 4, 10, dst, n, kept, acc_out)
    assert dsa.dsa_check_status() == 0
    for b, x in enumerate(lens):
        keep = np.array(K.keep(acc[b].cpu().numpy(), x, 100, 4, 10))
        src = p.table[b, keep // 64].astype(np.int64) * 64 + keep % 64
        moved, eo = K.move(p.codes, p.exps, src, [f for f in p.free[2 * b:2 * b + 2]])
        for j in range(-(-len(keep) // 64)):
            m = min(64, len(keep) - 64 * j)
            f = p.free[2 * b + j]
            assert np.array_equal(codes[shift + f, :m].cpu().numpy(), moved[f, :m]) and exps[shift + f].item() == eo[f]


@pytest.mark.parametrize("H,n_q,k", [(128, 1300, 0), (128, 1300, 24), (8, 2500, 7)])
def test_a_prompt_chunk_in_several_passes(dsa, H, n_q, k):
    """More queries of a contiguous cache than one pass takes (1184 at 128 heads, 2368 at
    up to 64), the chunk being the whole prompt: every position from 0 on."""
    p = Paged([n_q], seed=53, extra=0)
    codes, exps = p.codes[p.table[0, :p.num_pages]], p.exps[p.table[0, :p.num_pages]]
    d_c, d_e = torch.from_numpy(codes).cuda().view(-1, 576)[:n_q], torch.from_numpy(exps).cuda()
    q = _q(n_q, H, 150)
    idx = torch.from_numpy(_selection(range(n_q), k, 13)).cuda() if k else None
    att = dsa.attn_in(q, d_c, SCALE, 512)
    out, lse = _attend(dsa, att, d_e, idx, k, n_q, H)
    assert dsa.dsa_check_status() == 0
    x = torch.from_numpy(K.values(codes, exps)[:n_q]).cuda()
    keep = torch.arange(n_q, device="cuda")[None] <= torch.arange(n_q, device="cuda")[:, None]
    if k:
        chosen = torch.zeros(n_q, n_q + 1, dtype=torch.bool, device="cuda")
        chosen.scatter_(1, torch.where(idx >= 0, idx, n_q).long(), True)
        keep &= chosen[:, :n_q]
    for h in range(0, H, 37):
        z = (SCALE * (q[:, h].double() @ x.T)).masked_fill(~keep, -float("inf"))
        pr = torch.softmax(z, dim=1)
        _close(out[:, h:h + 1], lse[:, h:h + 1], *(t[:, None].cpu().numpy() for t in
               (pr @ x[:, :512], torch.logsumexp(z, dim=1), pr @ x[:, :512].abs())),
               z.masked_fill(~keep, 0).abs().max().item())


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("column", [3, 570])
def test_a_nan_row_reaches_the_queries_that_see_it(dsa, H, column):
    """A NaN that the store kept, in a latent or a rope column: NaN in every head of
    the queries that attend to the row, nothing in the others."""
    lens = [300, 300, 2000]
    p = Paged(lens, seed=54)
    for b in (0, 2):
        p.codes[p.table[b, 1], 9, column] = 0x7F
    p.d_codes.copy_(torch.from_numpy(p.codes))
    q_seq, q_pos = [0, 0, 1, 2, 2], [72, 299, 299, 73, 1999]
    q = _q(5, H, 160)
    s, t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (q_seq, q_pos))
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa, s, t))
    out, lse = _attend(dsa, att, p.d_exps, None, 0, 5, H)
    assert dsa.dsa_check_status() == 0
    seen = torch.tensor([False, True, False, True, True], device="cuda")
    assert torch.equal(torch.isnan(out).all(dim=2).all(dim=1), seen) and torch.equal(torch.isnan(out).any(dim=2).any(dim=1), seen)
    assert torch.equal(torch.isnan(lse).all(dim=1), seen) and torch.equal(torch.isnan(lse).any(dim=1), seen)
