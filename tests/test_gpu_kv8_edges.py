"""The 8-bit latent cache at the edges of its ranges, on the GPU: queries up to
the largest bf16 value, rows without latent values in blocks of a large scale,
logits far beyond one, exponents that the format does not have, calls in a row on
one workspace.

Where two calls must give the same bits, a power of two has only been moved from
one factor to another. Other tolerances are those of test_gpu_kv8."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K
from test_gpu_kv8 import Paged, _attend, _close, _q, _selection, SCALE

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
            zm = max(zm, float(np.abs(z[z >= z.max(axis=1, keepdims=True) - 60]).max()))
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


@pytest.mark.parametrize("H,k,sink", [(16, 0, 30), (128, 0, 70), (16, 1500, 70), (128, 1500, 30)])
def test_rows_without_latent_values_do_not_hide_the_others(dsa, H, k, sink):
    """Blocks whose scale an outlier token has raised by 2^28, so that their other
    rows hold zero codes (of both signs; with rope codes in sequence 1), and a sink
    with zero latent columns that takes all but e^-30 or e^-70 of the probability: the
    output is that of the keys in ordinary blocks, far below the zero rows' z + e."""
    lens = [1500, 1400, 1300, 1450]
    p = Paged(lens, seed=41)
    q = _q(4, H, 111)
    q[:, :, 512] = 0.0
    for b, blocks in ((0, (0, 9)), (1, (1, 20)), (2, (12,))):
        for j in blocks:
            pg = p.table[b, j]
            p.exps[pg] += 28
            p.codes[pg, :, :512] = np.where(np.arange(512) % 2, 0x80, 0x00)
            if b != 1:
                p.codes[pg, :, 512:] = 0x80
            # the outlier: small latent codes, a logit of about -3e8 for every head
            p.codes[pg, 17, :512] = K.encode_e4m3(K.round_e4m3(np.linspace(-3, 3, 512)))
            p.codes[pg, 17, 512:] = 0
            p.codes[pg, 17, 512] = 0xFE                   # -448
    q[:3, :, 512] = 8.0
    q[1, :, 513:] = 0.0                                   # sequence 1's rope codes count for nothing
    for b in range(3):                                    # the other rows do not see that column
        for j in range(-(-lens[b] // 64)):
            rows = np.arange(64) != 17 if p.exps[p.table[b, j]] > 10 else np.full(64, True)
            p.codes[p.table[b, j], rows, 512] = 0
    # sequence 3: the sink, the same z for every head
    pg = p.table[3, 4]
    p.codes[pg, 40] = 0
    p.codes[pg, 40, 512] = 0x7E                           # 448
    for j in range(-(-lens[3] // 64)):
        for r in range(64):
            if (j, r) != (4, 40):
                p.codes[p.table[3, j], r, 512] = 0
    q[3, :, 512] = sink / (SCALE * 448 * 2.0 ** float(p.exps[pg]))
    p.d_codes.copy_(torch.from_numpy(p.codes))
    p.d_exps.copy_(torch.from_numpy(p.exps))
    idx = _selection([n - 1 for n in lens], k, 9) if k else None
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, torch.from_numpy(idx).cuda() if k else None, k, 4, H)
    assert dsa.dsa_check_status() == 0
    sets = [p.rows(b, idx[b][idx[b] >= 0] if k else np.arange(lens[b])) for b in range(4)]
    qd = q.double().cpu().numpy()
    for b in range(4):                                    # each by itself: their outputs are of different sizes
        _close(out[b:b + 1], lse[b:b + 1], *_expected(qd[b:b + 1], sets[b:b + 1], SCALE))
        assert torch.all(out[b].abs().amax(dim=1) > 0), b


@pytest.mark.parametrize("H,k", [(16, 0), (128, 0), (32, 700), (128, 700)])
def test_logits_far_beyond_one(dsa, H, k):
    """Logits of up to 2^25, all the probability on the largest (two copies of a row
    in blocks whose scales differ by 2^8; a zero logit among very negative ones);
    past 2^26 fp32 has no room for the shift: NaN, unless a key inside decides."""
    lens = [700, 301, 700]
    p = Paged(lens, seed=43)
    q = _q(3, H, 113)
    q[:, :, 512], q[:, :, 0] = 512.0, 0.0
    value = np.where(np.arange(576) % 3, 80.0, -96.0)     # of the rows that win, in units of 2^e
    value[512], value[0] = 112.0, 0.0
    for b in range(3):
        for j in range(-(-lens[b] // 64)):
            p.codes[p.table[b, j], :, 512] = 0x00 if b == 0 else 0xF6    # -224
    e = int(p.exps[p.table[0, 5]])
    for j, slot, shift in ((5, 60, 0), (9, 3, 8)):
        pg = p.table[0, j]
        p.exps[pg] = e + shift
        if shift:
            p.codes[pg] = 0
        p.codes[pg, slot] = K.encode_e4m3(value * 2.0 ** -shift)
    p.codes[p.table[1, 4], 44] = 0                        # the last token of sequence 1
    p.codes[p.table[1, 4], 44, 0] = 0x38                  # 1.0
    p.codes[p.table[1, 4], :44] = p.codes[p.table[1, 3], :44]
    p.d_codes.copy_(torch.from_numpy(p.codes))
    p.d_exps.copy_(torch.from_numpy(p.exps))
    idx = _selection([n - 1 for n in lens], k, 11) if k else None
    d_idx = torch.from_numpy(idx).cuda() if k else None
    rows = [p.rows(b, np.arange(n)) for b, n in enumerate(lens)]
    for g in (12, 18, 24, 40, 90, 118):                   # logits of about 37, 0 and -70 times 2^g
        big = (q.float() * 2.0 ** g).to(torch.bfloat16)
        att = dsa.attn_in(big, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
        out, lse = _attend(dsa, att, p.d_exps, d_idx, k, 3, H)
        assert dsa.dsa_check_status() == 0
        o, l, _, _ = _expected(big.double().cpu().numpy(), rows, SCALE)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        inside = (0, 1) if g < 20 else (1,)
        for b in inside:                                  # one row's values, times weights exact to 2^-7, rounded to bf16
            assert np.all(np.abs(got[b] - o[b]) <= (2.0 ** -8 + 2.0 ** -7) * np.abs(o[b])), (g, b)
        assert np.all(gl[1] == 0), g
        if g < 20:                                        # fp32 logits of |q| |k| at most: 2^-20 of that
            norm = SCALE * np.linalg.norm(big[0].double().cpu().numpy(), axis=-1) * np.linalg.norm(value) * 2.0 ** e
            assert np.all(np.abs(gl[0] - l[0]) <= 2.0 ** -20 * norm + 1e-6), g
        else:
            assert np.isnan(got[[0, 2]]).all() and np.isnan(gl[[0, 2]]).all(), g


@pytest.mark.parametrize("H", [16, 128])
def test_calls_in_a_row_on_one_workspace(dsa, H):
    """Queries of very different sizes, call after call without a pause in one
    workspace: every call uses the operands and factors of its own queries."""
    lens = [65, 700, 130]
    p = Paged(lens, seed=44)
    qs = [_q(3, H, 120 + i, gain=2.0 ** (3 * i - 6)) for i in range(5)]
    atts = [dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa)) for q in qs]
    ref = [_attend(dsa, att, p.d_exps, None, 0, 3, H) for att in atts]
    width = p.table.shape[1] * 64
    ref_acc = [_weights(dsa, att, p.d_exps, None, 0, lse, 3, width) for att, (_, lse) in zip(atts, ref)]
    ws = dsa.workspace(max(dsa.dsa_workspace_size(op, None, atts[0], 0, 0, 0)
                           for op in (dsa.DSA_OP_KV8_MQA, dsa.DSA_OP_KV8_ACCUMULATE)))
    outs = [[torch.empty_like(ref[0][0]), torch.empty_like(ref[0][1]), torch.zeros_like(ref_acc[0])] for _ in range(200)]
    torch.cuda.synchronize()
    for i, (out, lse, acc) in enumerate(outs):
        dsa.dsa_kv8_mqa_fwd(atts[i % 5], p.d_exps, None, 0, out, lse, ws)
        dsa.dsa_kv8_accumulate(atts[i % 5], p.d_exps, None, 0, lse, 1.0, acc, ws)
    assert dsa.dsa_check_status() == 0
    for i, (out, lse, acc) in enumerate(outs):
        assert torch.equal(out, ref[i % 5][0]) and torch.equal(lse, ref[i % 5][1]) and torch.equal(acc, ref_acc[i % 5]), i


@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([20000, 100, 15001, 9000, 0, 5, 9001], 9000, 64, 512),       # a cluster a sequence, some within the budget
    ([20000, 19999, 64, 0, 300], 128, 0, 0), ([17000] * 3, 16999, 3, 5),
    ([700 + 37 * i for i in range(40)] + [0, 12000], 640, 16, 100)])   # one CTA a sequence
def test_eviction_of_many_ragged_sequences(dsa, lens, budget, sink, recent):
    """Selection by clusters and by single CTAs: kept positions, weights and rows of
    sequences far above the budget, within it, and without a token."""
    g = torch.Generator(device="cuda").manual_seed(6)
    m = [min(n, budget) for n in lens]
    pages, need = [-(-n // 64) for n in lens], [-(-n // 64) for n in m]
    total = sum(pages) + sum(need)
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(7)).to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    dst = torch.full((len(lens), -(-budget // 64)), -1, dtype=torch.int32)
    off = 0
    for b in range(len(lens)):
        table[b, :pages[b]] = perm[off:off + pages[b]]
        dst[b, :need[b]] = perm[off + pages[b]:off + pages[b] + need[b]]
        off += pages[b] + need[b]
    codes = torch.randint(0, 256, (total, 64, 576), generator=g, device="cuda").to(torch.uint8) & 0xF7
    exps = torch.full((total,), -6, dtype=torch.int8, device="cuda")
    acc = torch.rand(len(lens), table.shape[1] * 64, generator=g, device="cuda") ** 4
    acc[torch.rand(acc.shape, generator=g, device="cuda") < 0.4] = 0.0
    before = codes.clone()
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = torch.full_like(ctx, -7)
    kept = torch.full((len(lens), budget), -7, dtype=torch.int32, device="cuda")
    acc_out = torch.full((len(lens), budget), -7.0, device="cuda")
    cache = dsa.kv8_cache(codes, exps, dsa.paged_layout(table.cuda(), ctx, total))
    dsa.dsa_kv8_evict(cache, acc, budget, sink, recent, dst.cuda(), n, kept, acc_out)
    assert dsa.dsa_check_status() == 0
    assert n.tolist() == m
    want = before.cpu()
    for b in range(len(lens)):
        w = acc[b].cpu().numpy()
        keep = np.array(K.keep(w, lens[b], budget, sink, recent), dtype=np.int64)
        assert np.array_equal(kept[b].cpu().numpy(), np.concatenate([keep, np.full(budget - len(keep), -1)])), b
        assert np.array_equal(acc_out[b, :len(keep)].cpu().numpy(), w[keep]) and (acc_out[b, len(keep):] == -7).all(), b
        at = np.arange(len(keep))
        want[dst[b].numpy()[at // 64], at % 64] = before.cpu()[table[b].numpy()[keep // 64], keep % 64]
    assert torch.equal(codes.cpu(), want)


@pytest.mark.parametrize("H,k", [(16, 0), (128, 0), (128, 1400)])
@pytest.mark.parametrize("shift", [9, 13, 17])
def test_rows_far_below_their_blocks_scale(dsa, H, k, shift):
    """Blocks that an outlier has scaled up by 2^9 to 2^17: their other rows, of
    ordinary values, keep the small codes that are left of them, and their z + e
    lies as far above that of the other blocks' keys, which weigh as much."""
    lens = [1400, 1500]
    p = Paged(lens, seed=46)
    for b, j in ((0, 0), (1, 7)):
        p.codes[:, :, 512:] = 0
        pg = p.table[b, j]
        x = K.values(p.codes, p.exps).reshape(-1, 64, 576)[pg]
        p.exps[pg] += shift
        p.codes[pg] = K.encode_e4m3(K.round_e4m3(x * 2.0 ** -float(p.exps[pg])))
        p.codes[pg, 30] = K.encode_e4m3(np.full(576, 352.0))  # the outlier
    q = _q(2, H, 114)
    q[:, :, 512:] = -8.0                                  # only the outlier has rope codes
    p.d_codes.copy_(torch.from_numpy(p.codes))
    p.d_exps.copy_(torch.from_numpy(p.exps))
    idx = _selection([n - 1 for n in lens], k, 14) if k else None
    att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
    out, lse = _attend(dsa, att, p.d_exps, torch.from_numpy(idx).cuda() if k else None, k, 2, H)
    assert dsa.dsa_check_status() == 0
    sets = [p.rows(b, idx[b][idx[b] >= 0] if k else np.arange(lens[b])) for b in range(2)]
    qd = q.double().cpu().numpy()
    for b in range(2):
        _close(out[b:b + 1], lse[b:b + 1], *_expected(qd[b:b + 1], sets[b:b + 1], SCALE))


@pytest.mark.parametrize("bad", [-128, -65, 64, 127])
def test_exponents_outside_the_format(dsa, bad):
    """The keys of a block whose exponent is none are reported and skipped, the
    store leaves such a block as it is, eviction skips its rows."""
    lens = [300, 200, 70]
    p = Paged(lens, seed=42, extra=6)
    q = _q(3, 32, 112)
    p.exps[p.table[0, 2]] = p.exps[p.table[2, 1]] = bad
    p.d_exps.copy_(torch.from_numpy(p.exps))
    sets = [np.concatenate([np.arange(128), np.arange(192, 300)]), np.arange(200), np.arange(64)]
    idx = np.full((3, 300), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        idx[b, :n] = np.arange(n)
    for k, d_idx in ((0, None), (300, torch.from_numpy(idx).cuda())):
        att = dsa.attn_in(q, p.d_codes, SCALE, 512, kv_layout=p.layout(dsa))
        out, lse = _attend(dsa, att, p.d_exps, d_idx, k, 3, 32)
        assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
        qd = q.double().cpu().numpy()
        _close(out, lse, *_expected(qd, [p.rows(b, s) for b, s in enumerate(sets)], SCALE))
        acc = _weights(dsa, att, p.d_exps, d_idx, k, lse, 3, p.table.shape[1] * 64)
        assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
        for b, s in enumerate(sets):
            w = K.attend(qd[b], p.rows(b, s), SCALE)[2].mean(axis=0)
            assert np.abs(acc[b, s].double().cpu().numpy() - w).max() <= 1e-3 * w.max()
            rest = np.setdiff1d(np.arange(acc.shape[1]), s)
            assert not acc[b, rest].any()
    # the newest token of sequence 2 goes behind five rows of the bad block, sequence 0's into a sound one
    rows = torch.randn(3, 576, generator=torch.Generator().manual_seed(2))
    want_c, want_e = K.store(p.codes, p.exps, rows[:2].double().numpy(), [0, 1], [299, 199], p.table)
    dsa.dsa_kv8_store(dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa)), rows.cuda())
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    assert np.array_equal(p.d_exps.cpu().numpy(), want_e) and np.array_equal(p.d_codes.cpu().numpy(), want_c)
    p.codes, p.exps = want_c, want_e
    # eviction: the rows of sequence 0's bad block are left out, the others moved
    dst = torch.tensor([p.free[0:2], p.free[2:4], p.free[4:6]], dtype=torch.int32, device="cuda")
    kept = torch.empty(3, 128, dtype=torch.int32, device="cuda")
    acc = torch.rand(3, p.table.shape[1] * 64, generator=torch.Generator().manual_seed(3)).cuda()
    acc_out, n = torch.zeros(3, 128, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    dsa.dsa_kv8_evict(dsa.kv8_cache(p.d_codes, p.d_exps, p.layout(dsa)), acc, 128, 2, 10, dst, n, kept, acc_out)
    assert dsa.dsa_check_status() == dsa.DSA_ERR_DEVICE_BOUNDS
    codes, exps = p.d_codes.cpu().numpy(), p.d_exps.cpu().numpy()
    for b, (x, page) in enumerate(((0, 2), (1, None), (2, 1))):
        keep = np.array(K.keep(acc[b].cpu().numpy(), lens[b], 128, 2, 10))
        assert kept[b, :len(keep)].tolist() == keep.tolist()
        for j in range(0, len(keep), 64):
            src = keep[j:j + 64]
            ok = src // 64 != page
            to = int(dst[b, j // 64])
            e = int(p.exps[p.table[b, src[ok] // 64]].max()) if ok.any() else -64
            assert exps[to] == e
            flat = p.table[b, src // 64].astype(np.int64) * 64 + src % 64
            moved, _ = K.move(p.codes, p.exps, flat[ok], [to])
            assert np.array_equal(codes[to, np.flatnonzero(ok)], moved[to, :ok.sum()])
            assert np.array_equal(codes[to, np.flatnonzero(~ok)], p.codes[to, np.flatnonzero(~ok)])
