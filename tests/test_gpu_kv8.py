"""The 8-bit latent cache on the GPU against the 64-bit oracle: the store, the
attention over a selection and over every key, the accumulated weights, the
eviction, and a serving loop of all four.

Tolerances, from the arithmetic (u = 2^-8, half a bf16 step):
  codes, exponents, kept positions, moved rows: equal.
  output: each probability enters the product with relative error at most 2^-7
    (a sum of two 8-bit floats; the largest error of the second one), the output
    is rounded to bf16 once, and fp32 accumulation adds less than 2^-10 of the
    largest partial sum: |g - o| <= u |o| + 2^-7 sum_s p|v| + 2^-10 max|o|, and
    in the rms, where independent rounding errors average to 0.3 of their
    bounds, at most 4e-3 of the output's.
  lse: logits are exact products summed in fp32 with truncation: at most 40
    additions of relative error 2^-22 on sums as large as |q| |k| scale; with
    these inputs that bound is below 4e-5 (1 + max |z|).
  weights: the logit's and the lse's error enter the exponential: relative
    1e-4 (1 + max |z|) at most, and 1e-6 of the base that they are added to.
"""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_tcgen05_b200 import _build
    _build.build()
    from sparse_attention_long_tcgen05_b200 import dsa
    return dsa


class Paged:
    """Sequences of the given lengths in shuffled pages; rows that no token
    holds, and pages that no sequence holds, are NaN codes."""

    def __init__(self, lens, seed=0, extra=2, gain=1.0, ld=576, spread=3, empty=False):
        g = torch.Generator().manual_seed(seed)
        self.lens = list(lens)
        need = [max(1, -(-n // 64)) for n in lens]
        self.num_pages = sum(need) + extra
        perm = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
        off = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[off:off + n]
            off += n
        self.free = perm[off:]
        self.codes = np.full((self.num_pages, 64, 576), NAN_CODE, dtype=np.uint8)
        self.exps = torch.randint(-spread, spread + 1, (self.num_pages,), generator=g).numpy().astype(np.int8)
        if not empty:
            for b, n in enumerate(lens):
                for j in range(-(-n // 64)):
                    m = min(64, n - 64 * j)
                    pg = self.table[b, j]
                    x = torch.randn(m, 576, generator=g).double().numpy() * gain
                    e = K.block_exponent(x)
                    self.exps[pg] = e
                    self.codes[pg, :m] = K.encode_e4m3(K.round_e4m3(x * 2.0 ** -e))
        wide = torch.zeros(self.num_pages, 64, ld, dtype=torch.uint8)
        wide[:, :, :576] = torch.from_numpy(self.codes)
        self.d_codes = wide.cuda()[:, :, :576]
        self.d_exps = torch.from_numpy(self.exps).cuda()
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_ctx = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def layout(self, dsa, q_seq=None, q_pos=None):
        return dsa.paged_layout(self.d_table, self.d_ctx, self.num_pages, q_seq, q_pos)

    def rows(self, b, pos):
        pos = np.asarray(pos, dtype=np.int64)
        v = K.values(self.codes, self.exps)
        return v[self.table[b, pos // 64].astype(np.int64) * 64 + pos % 64]


def _attend(dsa, att, exps, idx, k, n_q, H, lse=True):
    out = torch.full((n_q, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((n_q, H), 7.0, device="cuda") if lse else None
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_MQA, None, att, 0, 0, k))
    ws.fill_(0xFF)
    dsa.dsa_kv8_mqa_fwd(att, exps, idx, k, out, l, ws)
    return out, l


def _close(out, lse, ref_out, ref_lse, absum, zmax):
    g, o = out.double().cpu().numpy(), ref_out
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), np.isneginf(ref_lse))
    fin = np.isfinite(ref_lse)
    assert np.all(np.abs(np.where(fin, lse.double().cpu().numpy() - np.where(fin, ref_lse, 0), 0)) <= 4e-5 * (1 + zmax))
    bound = 2.0 ** -8 * np.abs(o) + 2.0 ** -7 * absum + 2.0 ** -10 * np.abs(o).max(axis=-1, keepdims=True)
    err = np.abs(g - o)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-30)))
    if np.any(o):
        assert np.sqrt(np.mean((g - o) ** 2) / np.mean(o ** 2)) <= 4e-3


def _reference(q, keysets):
    out, lse, ab, zm = [], [], [], 0.0
    for qi, rows in zip(q, keysets):
        o, l, p = K.attend(qi, rows, SCALE)
        out.append(o)
        lse.append(l)
        ab.append(p @ np.abs(rows[:, :512]))
        if len(rows):
            zm = max(zm, float(np.abs(SCALE * (qi @ rows.T)).max()))
    return np.stack(out), np.stack(lse), np.stack(ab), zm


def _q(n, H, seed, gain=1.0, ld=None):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(n, H, 576, generator=g) * gain).to(torch.bfloat16)
    if ld is None:
        return q.cuda()
    wide = torch.zeros(n, ld, dtype=torch.bfloat16)
    wide[:, :H * 576] = q.view(n, -1)
    return wide.cuda().as_strided((n, H, 576), (ld, 576, 1))


def _selection(pos, k, seed):
    """Random distinct keys of each prefix in no order, with -1 anywhere."""
    rng = np.random.default_rng(seed)
    idx = np.full((len(pos), k), -1, dtype=np.int32)
    for i, p in enumerate(pos):
        n = min(k, p + 1)
        pick = rng.permutation(p + 1)[:n]
        idx[i, np.sort(rng.permutation(k)[:n])] = pick
    return idx


# ------------------------------------------------------------------------------------------ store

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("runs,lens", [
    ([1], [1]), ([1, 1, 1], [64, 65, 4000]), ([130, 0, 64, 7], [130, 50, 200, 71]),
    ([63, 1, 300], [64, 1, 364]), ([700], [901])])
def test_store_paged(dsa, dtype, runs, lens):
    p = Paged(lens, seed=3, ld=592)
    g = torch.Generator().manual_seed(4)
    rows = torch.randn(sum(runs), 576 + 16, generator=g) * torch.exp2(torch.randint(-4, 5, (sum(runs), 1), generator=g))
    rows[0, 3], rows[-1, 5] = 0.0, -1e-9
    rows = rows.to(dtype)
    cu = np.cumsum([0] + runs)
    seqs = [b for b, n in enumerate(runs) for _ in range(n)]
    pos = [lens[b] - runs[b] + i for b in range(len(runs)) for i in range(runs[b])]
    want_c, want_e = K.store(p.codes, p.exps, rows[:, :576].double().numpy(), seqs, pos, p.table)
    cache = dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa))
    d_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for _ in range(2):                                    # storing the same rows again changes nothing
        dsa.dsa_kv8_store(cache, rows.cuda()[:, :576], d_cu)
        assert dsa.dsa_check_status() == 0
        assert np.array_equal(p.d_exps.cpu().numpy(), want_e)
        assert np.array_equal(p.d_codes.cpu().numpy(), want_c)


def test_store_one_row_a_sequence_and_special_values(dsa):
    lens = [1, 65, 128, 500, 640, 77]
    p = Paged(lens, seed=5)
    rows = torch.randn(6, 576, generator=torch.Generator().manual_seed(6))
    rows[0] = 0                                           # the smallest exponent
    rows[1, 7], rows[1, 8], rows[1, 9] = float("nan"), float("inf"), -float("inf")
    rows[2] *= 1e30                                       # beyond 448 * 2^63: saturates
    rows[3] = 448.0                                       # exactly at a border
    rows[4, 0] = 448.5
    rows[5] *= 1e-30
    want_c, want_e = K.store(p.codes, p.exps, rows.double().numpy(), range(6), [n - 1 for n in lens], p.table)
    cache = dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa))
    dsa.dsa_kv8_store(cache, rows.cuda())
    assert dsa.dsa_check_status() == 0
    assert np.array_equal(p.d_exps.cpu().numpy(), want_e)
    assert np.array_equal(p.d_codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("n_keys,n", [(1, 1), (64, 64), (1000, 1000), (5003, 4966), (5003, 1)])
def test_store_contiguous(dsa, n_keys, n):
    p = Paged([n_keys], seed=7, extra=0)
    order = np.arange(p.num_pages)
    codes = p.codes[p.table[0, :p.num_pages]]
    exps = p.exps[p.table[0, :p.num_pages]]
    rows = (torch.randn(n, 576, generator=torch.Generator().manual_seed(8)) * 3).to(torch.bfloat16)
    want_c, want_e = K.store(codes, exps, rows.double().numpy(), [0] * n, list(range(n_keys - n, n_keys)), [order])
    d_c, d_e = torch.from_numpy(codes).cuda().view(-1, 576), torch.from_numpy(exps).cuda()
    dsa.dsa_kv8_store(dsa.kv8_cache(d_c[:n_keys], d_e), rows.cuda())
    assert dsa.dsa_check_status() == 0
    assert np.array_equal(d_e.cpu().numpy(), want_e)
    assert np.array_equal(d_c.cpu().numpy(), want_c.reshape(-1, 576))


def test_store_reports_and_skips_what_does_not_fit(dsa):
    lens = [10, 200, 70]
    p = Paged(lens, seed=9)
    p.table[1, 2] = p.num_pages + 5                       # rows 128..191 of sequence 1
    runs = [11, 100, 3]                                   # 11 rows into a sequence of 10
    rows = torch.randn(sum(runs), 576, generator=torch.Generator().manual_seed(1))
    keep = [i for i in range(11, 111) if not 128 <= 100 + i - 11 < 192] + [111, 112, 113]
    seqs = [1 if i < 111 else 2 for i in keep]
    pos = [100 + i - 11 if i < 111 else 67 + i - 111 for i in keep]
    want_c, want_e = K.store(p.codes, p.exps, rows[keep].double().numpy(), seqs, pos, p.table)
    p.d_table.copy_(torch.from_numpy(p.table))
    dsa.dsa_kv8_store(dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa)), rows.cuda(),
                      torch.tensor([0, 11, 111, 114], dtype=torch.int32, device="cuda"))
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    assert np.array_equal(p.d_exps.cpu().numpy(), want_e)
    assert np.array_equal(p.d_codes.cpu().numpy(), want_c)


# ------------------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("H", [1, 8, 16, 17, 32, 40, 64, 65, 100, 128])
def test_dense_heads(dsa, H):
    lens = [1, 63, 64, 129, 700]
    p = Paged(lens, seed=H, ld=608)
    q = _q(5, H, 20 + H, ld=H * 576 + 64)
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, None, 0, 5, H)
    assert dsa.dsa_check_status() == 0
    _close(out, lse, *_reference(q.double().cpu().numpy(), [p.rows(b, np.arange(n)) for b, n in enumerate(lens)]))


@pytest.mark.parametrize("lens,H", [([5000], 16), ([20011], 128), ([1, 30000, 2, 9000], 64), ([3000] * 9, 128)])
def test_dense_long_and_ragged(dsa, lens, H):
    """Keys of one query split over several CTAs, several queries on one CTA."""
    p = Paged(lens, seed=len(lens))
    q = _q(len(lens), H, 31)
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, None, 0, len(lens), H)
    assert dsa.dsa_check_status() == 0
    _close(out, lse, *_reference(q.double().cpu().numpy(), [p.rows(b, np.arange(n)) for b, n in enumerate(lens)]))
    again, lse2 = _attend(dsa, att, p.d_exps, None, 0, len(lens), H)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("k", [1, 2, 64, 127, 128, 129, 500, 2048])
def test_sparse_selections(dsa, k):
    lens = [1, 64, 200, 2500, 130]
    p = Paged(lens, seed=k)
    H = 128 if k % 2 == 0 else 48
    q = _q(5, H, 40 + k)
    idx = _selection([n - 1 for n in lens], k, k)
    d_idx = torch.from_numpy(np.pad(idx, ((0, 0), (0, 3)), constant_values=5)).cuda()[:, :k]
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, d_idx, k, 5, H)
    assert dsa.dsa_check_status() == 0
    _close(out, lse, *_reference(q.double().cpu().numpy(), [p.rows(b, idx[b][idx[b] >= 0]) for b in range(5)]))


@pytest.mark.parametrize("H,n_q,n_keys,k", [(128, 300, 333, 96), (16, 700, 700, 40), (64, 3, 5000, 2048), (128, 5, 5, 0),
                                            (32, 130, 200, 0)])
def test_contiguous_chunks(dsa, H, n_q, n_keys, k):
    p = Paged([n_keys], seed=11, extra=0)
    codes, exps = p.codes[p.table[0, :p.num_pages]], p.exps[p.table[0, :p.num_pages]]
    p.codes, p.exps, p.table = codes, exps, np.arange(p.num_pages)[None]
    q = _q(n_q, H, 50)
    pos = [n_keys - n_q + i for i in range(n_q)]
    d_c = torch.from_numpy(codes).cuda().view(-1, 576)[:n_keys]
    att = dsa.attn_in(q, d_c, SCALE, 512)
    idx = _selection(pos, k, 3) if k else None
    out, lse = _attend(dsa, att, torch.from_numpy(exps).cuda(), torch.from_numpy(idx).cuda() if k else None, k, n_q, H)
    assert dsa.dsa_check_status() == 0
    _close(out, lse, *_reference(q.double().cpu().numpy(),
                                 [p.rows(0, idx[i][idx[i] >= 0] if k else np.arange(pos[i] + 1)) for i in range(n_q)]))


@pytest.mark.parametrize("k", [0, 100])
def test_several_tokens_a_sequence(dsa, k):
    lens = [500, 70, 3, 260]
    p = Paged(lens, seed=12)
    q_seq, q_pos = [3, 0, 0, 2, 1, 1, 3, 2], [259, 499, 498, 0, 69, 10, 257, 2]
    q = _q(8, 128, 60)
    s, t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (q_seq, q_pos))
    idx = _selection(q_pos, k, 5) if k else None
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa, s, t))
    out, lse = _attend(dsa, att, p.d_exps, torch.from_numpy(idx).cuda() if k else None, k, 8, 128)
    assert dsa.dsa_check_status() == 0
    _close(out, lse, *_reference(q.double().cpu().numpy(), [p.rows(b, idx[i][idx[i] >= 0] if k else np.arange(x + 1))
                                                            for i, (b, x) in enumerate(zip(q_seq, q_pos))]))


def test_empty_rows_and_bad_entries(dsa):
    lens = [100, 300, 64, 10]
    p = Paged(lens, seed=13)
    idx = np.full((4, 130), -1, dtype=np.int32)           # query 0: nothing
    idx[1, [0, 70, 129]] = [5, 299, 300]                  # 300 is past the position
    idx[2, :64] = np.arange(64)
    idx[3, 1] = 2 ** 31 - 1
    q = _q(4, 128, 70)
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, torch.from_numpy(idx).cuda(), 130, 4, 128)
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    sets = [[], [5, 299], list(range(64)), []]
    _close(out, lse, *_reference(q.double().cpu().numpy(), [p.rows(b, s) for b, s in enumerate(sets)]))
    assert not out[0].any() and not out[3].any()
    # a page id out of range: its keys are skipped and reported, in both modes
    p.table[1, 1] = -3
    p.d_table.copy_(torch.from_numpy(p.table))
    out, lse = _attend(dsa, att, p.d_exps, None, 0, 4, 128)
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    sets = [np.arange(100), np.concatenate([np.arange(64), np.arange(128, 300)]), np.arange(64), np.arange(10)]
    p.table[1, 1] = 0
    _close(out, lse, *_reference(q.double().cpu().numpy(), [p.rows(b, s) for b, s in enumerate(sets)]))
    # a length out of range: an empty row
    p.d_ctx[2] = 0
    out, lse = _attend(dsa, att, p.d_exps, None, 0, 4, 128)
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    assert not out[2].any() and torch.all(torch.isneginf(lse[2])) and torch.isfinite(lse[0]).all()


def test_values_far_apart(dsa):
    """One key takes nearly all the probability and has a zero value, pages whose
    scales differ by 2^20, logits of hundreds: the small weights still count."""
    n = 3000
    p = Paged([n, n, n], seed=14)
    q = _q(3, 64, 80)
    q[1] *= 40
    # sequence 0: key 0 is a sink along the first 64 rope columns, with zero latent
    pg = p.table[0, 0]
    p.codes[pg, 0, :512] = 0
    p.codes[pg, 0, 512:] = K.encode_e4m3(np.full(64, 208.0))
    q[0, :, 512:] = 0.125
    # sequence 2: a few pages hold values 2^20 larger, and their keys' logits are low
    for j in (3, 20):
        p.exps[p.table[2, j]] += 20
    q[2] *= 2.0 ** -18
    p.d_codes.copy_(torch.from_numpy(p.codes))
    p.d_exps.copy_(torch.from_numpy(p.exps))
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, None, 0, 3, 64)
    assert dsa.dsa_check_status() == 0
    o, l, ab, zm = _reference(q.double().cpu().numpy(), [p.rows(b, np.arange(n)) for b in range(3)])
    _close(out, lse, o, l, ab, zm)
    for b in range(3):                                    # each sequence by itself: no large one hides a small one
        r = out[b].double().cpu().numpy()
        assert np.sqrt(np.mean((r - o[b]) ** 2) / np.mean(o[b] ** 2)) <= 4e-3, b


def test_nan_and_infinity_stay_in_their_head(dsa):
    p = Paged([300, 90], seed=15)
    q = _q(2, 128, 90)
    q[0, 3, 17], q[0, 100, 500], q[1, 127, 575] = float("nan"), float("inf"), float("nan")
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, None, 0, 2, 128)
    assert dsa.dsa_check_status() == 0
    bad = torch.isnan(out).all(dim=2)
    want = torch.zeros(2, 128, dtype=torch.bool, device="cuda")
    want[0, 3] = want[0, 100] = want[1, 127] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(out).any(dim=2), want)
    assert torch.isfinite(lse[~want]).all() and torch.isnan(lse[want]).all()


def test_no_lse_other_stream_and_graph(dsa):
    lens = [900, 40, 5000]
    p = Paged(lens, seed=16)
    q = _q(3, 128, 91)
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    ref, _ = _attend(dsa, att, p.d_exps, None, 0, 3, 128)
    out, none = _attend(dsa, att, p.d_exps, None, 0, 3, 128, lse=False)
    assert none is None and torch.equal(out, ref)
    ws = [dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_MQA, None, att, 0, 0, 0)) for _ in range(2)]
    outs = [torch.zeros_like(ref) for _ in range(2)]
    lse = torch.empty(3, 128, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):                                    # two calls at once, a workspace each
        for s, o, w in zip(streams, outs, ws):
            with torch.cuda.stream(s):
                dsa.dsa_kv8_mqa_fwd(att, p.d_exps, None, 0, o, None, w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_kv8_mqa_fwd(att, p.d_exps, None, 0, outs[0], lse, ws[0])
    q.copy_(_q(3, 128, 92))
    g.replay()
    want, _ = _attend(dsa, att, p.d_exps, None, 0, 3, 128)
    assert torch.equal(outs[0], want)
    assert dsa.dsa_check_status() == 0


# ------------------------------------------------------------------------------------------ weights

@pytest.mark.parametrize("decay", [1.0, 0.5])
@pytest.mark.parametrize("k,H,several", [(0, 128, False), (0, 16, True), (150, 128, False), (70, 24, True), (128, 65, False)])
def test_accumulate(dsa, decay, k, H, several):
    lens = [500, 70, 3, 260]
    p = Paged(lens, seed=17)
    q_seq = [3, 0, 0, 2, 1, 1, 3, 0] if several else [0, 1, 2, 3]
    q_pos = [259, 499, 498, 2, 69, 10, 257, 80] if several else [n - 1 for n in lens]
    n_q = len(q_seq)
    q = _q(n_q, H, 100)
    s, t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (q_seq, q_pos))
    idx = _selection(q_pos, k, 8) if k else None
    if k:
        idx[0, 0] = idx[0, 3] = idx[0, 5] = 7             # the same key three times
    d_idx = torch.from_numpy(idx).cuda() if k else None
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa, *((s, t) if several else ())))
    _, lse = _attend(dsa, att, p.d_exps, d_idx, k, n_q, H)
    width = p.table.shape[1] * 64
    base = torch.rand(4, width + 5, generator=torch.Generator().manual_seed(3)) * 1e-3
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))
    got = []
    for _ in range(2):
        ws.fill_(0xFF)
        acc = base.cuda()
        dsa.dsa_kv8_accumulate(att, p.d_exps, d_idx, k, lse, decay, acc, ws)
        assert dsa.dsa_check_status() == 0
        got.append(acc)
    assert torch.equal(got[0], got[1])
    want, w = base.double().numpy(), np.zeros(base.shape)
    zm = 0.0
    for b, n in enumerate(lens):
        want[b, :n] *= decay
    for i in range(n_q):
        keys = idx[i][idx[i] >= 0] if k else np.arange(q_pos[i] + 1)
        rows = p.rows(q_seq[i], keys)
        z = SCALE * (q[i].double().cpu().numpy() @ rows.T)
        zm = max(zm, float(np.abs(z).max()))
        np.add.at(w[q_seq[i]], keys, np.exp(z - lse[i].double().cpu().numpy()[:, None]).mean(axis=0))
    err = np.abs(got[0].double().cpu().numpy() - (want + w))
    assert np.all(err <= 1e-4 * (1 + zm) * w + 1e-6 * np.abs(want))
    for b, n in enumerate(lens):                          # behind the sequence: as it was
        assert np.array_equal(got[0][b, n:].cpu().numpy(), base[b, n:].numpy())


def test_accumulate_contiguous_and_empty(dsa):
    n_keys, n_q, H = 333, 41, 32
    p = Paged([n_keys], seed=18, extra=0)
    p.codes, p.exps = p.codes[p.table[0, :p.num_pages]], p.exps[p.table[0, :p.num_pages]]
    p.table = np.arange(p.num_pages)[None]
    q = _q(n_q, H, 101)
    pos = [n_keys - n_q + i for i in range(n_q)]
    idx = _selection(pos, 64, 9)
    idx[5] = -1                                           # nothing selected: lse is -inf, adds nothing
    d_exps, d_idx = torch.from_numpy(p.exps).cuda(), torch.from_numpy(idx).cuda()
    att = dsa.attn_in(q, torch.from_numpy(p.codes).cuda().view(-1, 576)[:n_keys], SCALE, 512)
    for k, di in ((64, d_idx), (0, None)):
        _, lse = _attend(dsa, att, d_exps, di, k, n_q, H)
        acc = torch.zeros(1, n_keys, device="cuda")
        ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))
        dsa.dsa_kv8_accumulate(att, d_exps, di, k, lse, 1.0, acc, ws)
        assert dsa.dsa_check_status() == 0
        want = np.zeros(n_keys)
        for i in range(n_q):
            keys = idx[i][idx[i] >= 0] if k else np.arange(pos[i] + 1)
            _, _, pr = K.attend(q[i].double().cpu().numpy(), p.rows(0, keys), SCALE)
            if len(keys):
                np.add.at(want, keys, pr.mean(axis=0))
        np.testing.assert_allclose(acc[0].double().cpu().numpy(), want, rtol=1e-3, atol=1e-9)
        assert abs(float(acc.sum()) - (n_q - (1 if k else 0))) < 1e-3 * n_q


@pytest.mark.parametrize("several", [False, True])
def test_more_queries_than_one_pass_takes(dsa, several):
    """2500 decode queries: attention in passes of 1184 (128 heads), weights in
    passes of 2048, over sequences of their own or 300 shared ones."""
    n_q, H, k = 2500, 66, 5
    n_seq = 300 if several else n_q
    g = torch.Generator().manual_seed(30)
    lens = torch.randint(1, 65, (n_seq,), generator=g).tolist()
    p = Paged(lens, seed=31)
    q_seq = torch.randint(0, n_seq, (n_q,), generator=g).tolist() if several else list(range(n_q))
    q_pos = [lens[b] - 1 for b in q_seq]
    s, t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (q_seq, q_pos))
    q = _q(n_q, H, 102)
    idx = _selection(q_pos, k, 10)
    rows = K.values(p.codes, p.exps)
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa, *((s, t) if several else ())))
    d_idx = torch.from_numpy(idx).cuda()
    out, lse = _attend(dsa, att, p.d_exps, d_idx, k, n_q, H)
    acc = torch.full((n_seq, p.table.shape[1] * 64), 2.0, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))
    dsa.dsa_kv8_accumulate(att, p.d_exps, d_idx, k, lse, 0.5, acc, ws)
    assert dsa.dsa_check_status() == 0
    qd, want = q.double().cpu().numpy(), np.full(acc.shape, 2.0)
    for b, n in enumerate(lens):
        want[b, :n] = 1.0
    refs = [[], [], []]
    for i in range(n_q):
        keys = idx[i][idx[i] >= 0]
        r = rows[p.table[q_seq[i], 0] * 64 + keys]
        o, l, pr = K.attend(qd[i], r, SCALE)
        np.add.at(want[q_seq[i]], keys, pr.mean(axis=0))
        for v, x in zip(refs, (o, l, pr @ np.abs(r[:, :512]))):
            v.append(x)
    _close(out, lse, *(np.stack(v) for v in refs), 10.0)
    np.testing.assert_allclose(acc.double().cpu().numpy(), want, rtol=1e-4)


def test_contiguous_weights_in_passes(dsa):
    """600 queries over 40,000 keys without a selection: passes of 419 queries,
    and a decay of the keys behind the first pass's."""
    n_keys, n_q, H = 40000, 600, 1
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n_keys, 576, generator=g, device="cuda")
    exps = torch.full((n_keys // 64,), -6, dtype=torch.int8, device="cuda")
    codes = (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    q = torch.randn(n_q, H, 576, generator=g, device="cuda").to(torch.bfloat16)
    att = dsa.attn_in(q, codes.view(torch.uint8), SCALE, 512)
    _, lse = _attend(dsa, att, exps, None, 0, n_q, H)
    acc = torch.ones(1, n_keys, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, 0))
    # 419 queries' weights (at most 64 MiB) and their operands: 2 x 16 padded heads x 576 bytes + 16 factors each
    assert ws.numel() <= (64 << 20) + 419 * (2 * 16 * 576 + 16 * 4) + 512
    dsa.dsa_kv8_accumulate(att, exps, None, 0, lse, 0.25, acc, ws)
    assert dsa.dsa_check_status() == 0
    z = q[:, 0].double() @ (codes.double() / 64).T * SCALE
    pos = torch.arange(n_keys - n_q, n_keys, device="cuda")[:, None]
    z = z.masked_fill(torch.arange(n_keys, device="cuda")[None] > pos, -float("inf"))
    assert torch.max((torch.logsumexp(z, 1) - lse[:, 0]).abs()) < 1e-4
    want = 0.25 + torch.exp(z - torch.logsumexp(z, 1, keepdim=True)).sum(dim=0)
    assert torch.max((acc[0].double() - want).abs() / want) < 1e-4


# ------------------------------------------------------------------------------------------ eviction

@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([1000], 100, 4, 20), ([5, 64, 65, 700], 64, 0, 0), ([300, 40, 2000], 256, 64, 192), ([129, 4000], 128, 1, 127),
    ([3000] * 3, 2999, 10, 100), ([70000], 9000, 16, 512), ([1], 1, 0, 1)])
@pytest.mark.parametrize("keys", [False, True])
def test_evict(dsa, lens, budget, sink, recent, keys):
    g = torch.Generator().manual_seed(19)
    m = [min(n, budget) for n in lens]
    need = [-(-x // 64) for x in m]
    p = Paged(lens, seed=20, extra=sum(need) + 1, ld=592, gain=2.0)
    width = p.table.shape[1] * 64
    acc = torch.rand(len(lens), width + 3, generator=g) ** 4
    acc[torch.rand(acc.shape, generator=g) < 0.4] = 0.0   # ties
    acc[0, 0], acc[-1, min(lens[-1], 40) - 1] = float("nan"), -0.0
    dst = np.full((len(lens), -(-budget // 64)), -1, dtype=np.int32)
    off = 0
    for b, n in enumerate(need):
        dst[b, :n] = p.free[off:off + n]
        off += n
    ik = torch.randint(0, 256, (p.num_pages, 64, 144), generator=g).to(torch.uint8)
    iks = torch.rand(p.num_pages, 64, generator=g)
    d_ik, d_iks = (ik.cuda()[:, :, :128], iks.cuda()) if keys else (None, None)
    lens_out = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    kept = torch.full((len(lens), budget + 2), -7, dtype=torch.int32, device="cuda")
    acc_out = torch.full((len(lens), budget + 1), -7.0, device="cuda")
    cache = dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa))
    dsa.dsa_kv8_evict(cache, acc.cuda(), budget, sink, recent, torch.from_numpy(dst).cuda(), lens_out, kept, acc_out,
                      d_ik, d_iks)
    assert dsa.dsa_check_status() == 0
    codes, exps = p.codes, p.exps
    want_ik, want_iks = ik[:, :, :128].numpy().copy(), iks.numpy().copy()
    for b, n in enumerate(lens):
        keep = K.keep(acc[b].numpy(), n, budget, sink, recent)
        assert lens_out[b].item() == len(keep) == m[b]
        row = kept[b].cpu().numpy()
        assert np.array_equal(row, keep + [-1] * (budget - len(keep)) + [-7, -7])
        assert np.array_equal(acc_out[b].cpu().numpy(), np.concatenate([acc[b].numpy()[keep], np.full(budget + 1 - len(keep), -7.0)]),
                              equal_nan=True)
        src = p.table[b, np.array(keep) // 64].astype(np.int64) * 64 + np.array(keep) % 64
        moved, eo = K.move(p.codes, p.exps, src, dst[b])
        pages = dst[b, :need[b]]
        codes, exps = codes.copy(), exps.copy()
        codes[pages], exps[pages] = moved[pages], eo[pages]
        to = dst[b, np.arange(len(keep)) // 64].astype(np.int64) * 64 + np.arange(len(keep)) % 64
        want_ik.reshape(-1, 128)[to], want_iks.reshape(-1)[to] = ik[:, :, :128].numpy().reshape(-1, 128)[src], iks.numpy().reshape(-1)[src]
    assert np.array_equal(p.d_codes.cpu().numpy(), codes)
    assert np.array_equal(p.d_exps.cpu().numpy(), exps)
    if keys:
        assert np.array_equal(d_ik.cpu().numpy(), want_ik) and np.array_equal(d_iks.cpu().numpy(), want_iks)


def test_evict_writes_the_lengths_in_place_and_reports_bad_ones(dsa):
    p = Paged([200, 300, 100], seed=21, extra=8)
    p.d_ctx[2] = 64 * p.table.shape[1] + 1                # more tokens than the table has
    dst = torch.tensor([p.free[0:2], p.free[2:4], p.free[4:6]], dtype=torch.int32, device="cuda")
    dst[1, 1] = p.num_pages                               # not a page
    kept = torch.full((3, 128), -7, dtype=torch.int32, device="cuda")
    acc = torch.rand(3, p.table.shape[1] * 64, device="cuda")
    acc_out = torch.zeros(3, 128, device="cuda")
    dsa.dsa_kv8_evict(dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa)), acc, 128, 2, 10, dst, p.d_ctx, kept, acc_out)
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    assert p.d_ctx.tolist() == [128, 128, 0]
    assert torch.all(kept[2] == -1) and kept[0, -1].item() == 199
    assert kept[1].tolist() == K.keep(acc[1].cpu().numpy(), 300, 128, 2, 10)


# ------------------------------------------------------------------------------------------ together

def test_a_serving_loop(dsa):
    """Prompts stored, decoded over the selection with running weights, evicted,
    and decoded on over the smaller cache: every step against the oracle."""
    H, k, budget = 32, 64, 192
    lens = [300, 150, 420]
    p = Paged([n + 8 for n in lens], seed=22, extra=3 * 4, empty=True)
    p.d_ctx.copy_(torch.tensor(lens))
    g = torch.Generator().manual_seed(23)
    rows = torch.randn(sum(lens), 576, generator=g).to(torch.bfloat16)
    cache = dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa))
    dsa.dsa_kv8_store(cache, rows.cuda(), torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda"))
    acc = torch.zeros(3, p.table.shape[1] * 64, device="cuda")

    def step(n, table, codes_exps, seed):
        """One decode step at lengths n: new rows in, attention, weights."""
        lay = dsa.paged_layout(table, p.d_ctx, p.num_pages)
        cache = dsa.kv8_cache(p.d_codes, p.d_exps, lay)
        new = torch.randn(3, 576, generator=g).to(torch.bfloat16)
        dsa.dsa_kv8_store(cache, new.cuda())
        c, e = K.store(*codes_exps, new.double().numpy(), range(3), [x - 1 for x in n], table.cpu().numpy())
        assert np.array_equal(p.d_codes.cpu().numpy(), c) and np.array_equal(p.d_exps.cpu().numpy(), e)
        q = _q(3, H, seed)
        idx = _selection([x - 1 for x in n], k, seed)
        att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=lay)
        d_idx = torch.from_numpy(idx).cuda()
        out, lse = _attend(dsa, att, p.d_exps, d_idx, k, 3, H)
        p.codes, p.exps, p.table = c, e, table.cpu().numpy()
        sets = [p.rows(b, idx[b][idx[b] >= 0]) for b in range(3)]
        _close(out, lse, *_reference(q.double().cpu().numpy(), sets))
        ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))
        before = acc.double().cpu().numpy()
        dsa.dsa_kv8_accumulate(att, p.d_exps, d_idx, k, lse, 0.9, acc, ws)
        for b in range(3):
            want = before[b].copy()
            want[:n[b]] *= np.float32(0.9)
            keys = idx[b][idx[b] >= 0]
            np.add.at(want, keys, K.attend(q[b].double().cpu().numpy(), sets[b], SCALE)[2].mean(axis=0))
            np.testing.assert_allclose(acc[b].cpu().numpy(), want, rtol=1e-3, atol=1e-9)
        return c, e

    pos = [i for n in lens for i in range(n)]
    seqs = [b for b, n in enumerate(lens) for _ in range(n)]
    state = K.store(p.codes, p.exps, rows.double().numpy(), seqs, pos, p.table)
    for t in range(3):
        p.d_ctx.add_(1)
        state = step([n + t + 1 for n in lens], p.d_table, state, 200 + t)
    n = [x + 3 for x in lens]
    dst = torch.tensor([p.free[4 * b:4 * b + 4] for b in range(3)], dtype=torch.int32, device="cuda")
    kept = torch.empty(3, budget, dtype=torch.int32, device="cuda")
    acc_out = torch.zeros(3, dst.shape[1] * 64, device="cuda")
    cache = dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa))
    dsa.dsa_kv8_evict(cache, acc, budget, 4, 16, dst, p.d_ctx, kept, acc_out)
    new = [min(budget, x) for x in n]
    assert p.d_ctx.tolist() == new
    codes, exps = state
    for b in range(3):
        keep = np.array(K.keep(acc[b].cpu().numpy(), n[b], budget, 4, 16))
        src = p.table[b, keep // 64].astype(np.int64) * 64 + keep % 64
        codes, exps = K.move(codes, exps, src, dst[b].tolist())
    acc = acc_out
    for t in range(2):
        p.d_ctx.add_(1)
        codes, exps = step([x + t + 1 for x in new], dst, (codes, exps), 300 + t)
    assert dsa.dsa_check_status() == 0
