"""Pins of the 8-bit latent cache's oracle (CPU): its rounding against torch's
own e4m3 conversion, its exponents against the definition, its attention
against torch.softmax, its store and eviction against their invariants."""
import numpy as np
import torch

from oracle import kv8_oracle as K
from oracle.dsa_oracle import e4m3_decode


def test_round_and_encode_match_torch_cast():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * s for s in (1e-3, 0.05, 1.0, 100.0)])
    # every code, and every midpoint between neighbours (ties to even)
    v = e4m3_decode(np.arange(127, dtype=np.uint8))
    mid = torch.tensor((v[1:] + v[:-1]) / 2, dtype=torch.float32)
    x = torch.cat([x, mid, -mid, torch.tensor(v, dtype=torch.float32)]).clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(K.encode_e4m3(K.round_e4m3(x.numpy())), want)
    assert np.array_equal(K.round_e4m3([1e9, -1e9, np.inf]), [448.0, -448.0, 448.0])
    assert K.encode_e4m3(K.round_e4m3([np.nan]))[0] == 0x7F


def test_block_exponent_is_the_smallest_that_holds():
    for a in (448.0, 448.0000001, 447.9, 224.0, 1.0, 1.75, 1.7500001, 3e-20, 2.0 ** 71, 0.0):
        e = K.block_exponent([a, -a / 2, np.nan, np.inf])
        assert e == 63 or a <= 448.0 * 2.0 ** e
        assert e == -64 or a > 448.0 * 2.0 ** (e - 1)


def test_store_rescales_earlier_rows_without_a_second_rounding():
    rng = np.random.default_rng(1)
    codes = np.full((3, 64, 576), 0x7F, dtype=np.uint8)
    exps = np.zeros(3, dtype=np.int8)
    table = [[2, 0]]
    first = rng.standard_normal((60, 576))
    codes, exps = K.store(codes, exps, first, [0] * 60, list(range(60)), table)
    before = e4m3_decode(codes[2, :60]) * 2.0 ** float(exps[2])
    more = rng.standard_normal((10, 576)) * 8
    codes, exps = K.store(codes, exps, more, [0] * 10, list(range(60, 70)), table)
    after = e4m3_decode(codes[2, :60]) * 2.0 ** float(exps[2])
    small = np.abs(before) < 2.0 ** (int(exps[2]) - 6 + 4)       # may be subnormal now
    assert np.array_equal(before[~small], after[~small])
    assert np.max(np.abs(before - after)) <= 2.0 ** (int(exps[2]) - 10)
    assert np.all(np.isnan(e4m3_decode(codes[0, 6:])))           # behind the last row: untouched
    amax = np.abs(more[4:]).max()
    assert 448 * 2.0 ** (int(exps[0]) - 1) < amax <= 448 * 2.0 ** int(exps[0])


def test_attend_matches_torch_softmax():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(5, 576, generator=g, dtype=torch.float64)
    x = torch.randn(33, 576, generator=g, dtype=torch.float64)
    z = q @ x.T * 0.05
    out, lse, p = K.attend(q.numpy(), x.numpy(), 0.05)
    ref = torch.softmax(z, dim=1)
    np.testing.assert_allclose(p, ref.numpy(), rtol=1e-12)
    np.testing.assert_allclose(out, (ref @ x[:, :512]).numpy(), rtol=1e-10)
    np.testing.assert_allclose(lse, torch.logsumexp(z, 1).numpy(), rtol=1e-13)
    out, lse, _ = K.attend(q.numpy(), x.numpy()[:0], 0.05)
    assert not out.any() and np.all(np.isneginf(lse))


def test_keep_rules():
    acc = [5.0, 0.0, 3.0, 3.0, np.nan, -0.0, 1.0, 3.0, 9.0, 0.0]
    assert K.keep(acc, 4, 4, 1, 1) == [0, 1, 2, 3]
    assert K.keep(acc, 10, 5, 1, 1) == [0, 2, 3, 8, 9][:1] + [2, 3, 8] + [9]
    assert K.keep(acc, 10, 4, 0, 0) == [0, 2, 3, 8]              # ties to the lower position
    assert K.keep(acc, 10, 8, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8]  # zeros before the NaN, low first
    assert K.keep(acc, 10, 3, 1, 2) == [0, 8, 9]


def test_move_takes_the_largest_exponent():
    codes = np.zeros((4, 64, 576), dtype=np.uint8)
    exps = np.array([0, 3, 0, 0], dtype=np.int8)
    codes[0, 5], codes[1, 7] = 0x40, 0x41                        # 2.0, 2.25
    out, eo = K.move(codes, exps, [5, 64 + 7], [3])
    assert eo[3] == 3
    assert np.all(e4m3_decode(out[3, 0]) * 8 == 2.0) and np.all(out[3, 1] == 0x41)
