"""Host-side refusals of the 8-bit latent cache's calls: every malformed call
returns its status before anything is launched. Fake device addresses, so only
on a host without a CUDA device, as in test_abi_checks."""
import ctypes

import pytest
import torch

from test_abi_checks import FAKE, _expect, _mut, _p, _paged

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device pointers: host-only checks")
P = FAKE + 0x400000


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_tcgen05_b200 import _build
    _build.build()
    from sparse_attention_long_tcgen05_b200 import dsa
    return dsa


def _lay(dsa, n_seq=64):
    return _mut(_paged(dsa), n_seq=n_seq)


def _attn(dsa, heads=128, n_q=64, kv=None):
    return dsa.AttnIn(dsa.DSA_BF16, n_q, 0, heads, 576, 512, 576 ** -0.5, FAKE + 0x60000,
                      heads * 576, FAKE + 0x70000, 576, None, 0, kv if kv is not None else _lay(dsa))


def _cache(dsa, kv=None, n_keys=0):
    return dsa.Kv8Cache(FAKE + 0x10000, 576, FAKE + 0x20001, n_keys,
                        kv if kv is not None else _lay(dsa))


def _contig(dsa):
    return dsa.KvLayout(dsa.DSA_KV_CONTIGUOUS, 0, None, 0, 0, 0, None)


def test_struct_layout(dsa, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "l.c").write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void) {'
        'printf("%zu %zu %zu %zu %zu %d %d", sizeof(dsa_kv8_cache), offsetof(dsa_kv8_cache, ld),'
        'offsetof(dsa_kv8_cache, exps), offsetof(dsa_kv8_cache, n_keys), offsetof(dsa_kv8_cache, kv),'
        'DSA_OP_KV8_MQA, DSA_OP_KV8_ACCUMULATE); return 0; }')
    exe = str(tmp_path / "l")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    C = dsa.Kv8Cache
    assert [int(x) for x in got] == [ctypes.sizeof(C), C.ld.offset, C.exps.offset, C.n_keys.offset,
                                     C.kv.offset, dsa.DSA_OP_KV8_MQA, dsa.DSA_OP_KV8_ACCUMULATE]


def test_store_refusals(dsa):
    INV, UNS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED

    def store(c=None, dt=dsa.DSA_BF16, rows=P, ld=576, cu=P + 0x1000, n=100):
        c = c if c is not None else _cache(dsa)
        return dsa.LIB.dsa_kv8_store(ctypes.byref(c), dt, _p(rows), ld, _p(cu), n, None)
    _expect(dsa, dsa.DSA_ERR_CUDA, lambda: store())
    _expect(dsa, dsa.DSA_ERR_CUDA, lambda: store(cu=None, n=64))
    _expect(dsa, INV, lambda: store(cu=None, n=65))               # one row a sequence
    _expect(dsa, INV, lambda: dsa.LIB.dsa_kv8_store(None, 2, _p(P), 576, None, 1, None))
    for st, kw in ((INV, dict(rows=None)), (INV, dict(n=0)), (INV, dict(ld=575)), (INV, dict(ld=577)),
                   (INV, dict(rows=P + 8)), (UNS, dict(dt=dsa.DSA_E4M3)), (UNS, dict(dt=7))):
        _expect(dsa, st, lambda: store(**kw))
    for st, kw in ((INV, dict(codes=None)), (INV, dict(exps=None)), (INV, dict(ld=560)), (INV, dict(ld=584)),
                   (INV, dict(codes=FAKE + 8)), (INV, dict(kv=_lay(dsa, 0))),
                   (UNS, dict(kv=_mut(_lay(dsa), page_size=32))), (INV, dict(kv=_mut(_lay(dsa), ctx_lens=None)))):
        _expect(dsa, st, lambda: store(_mut(_cache(dsa), **kw)))
    c = _cache(dsa, _contig(dsa), 200)
    _expect(dsa, dsa.DSA_ERR_CUDA, lambda: store(c, cu=None))
    _expect(dsa, INV, lambda: store(c))                           # no runs in a contiguous cache
    _expect(dsa, INV, lambda: store(c, cu=None, n=201))
    _expect(dsa, INV, lambda: store(_cache(dsa, _contig(dsa), 0), cu=None))


def test_attention_and_accumulate_refusals(dsa):
    INV, UNS, WS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE_TOO_SMALL

    def fwd(a=None, e=P, idx=P + 0x1000, ld=2048, k=2048, out=P + 0x2000, ws=P + 0x100000, nb=1 << 34):
        a = a if a is not None else _attn(dsa)
        return dsa.LIB.dsa_kv8_mqa_fwd(ctypes.byref(a), _p(e), _p(idx), ld, k, _p(out), None, _p(ws), nb, None)

    def acc(a=None, e=P, idx=P + 0x1000, ld=2048, k=2048, lse=P + 0x2000, decay=1.0, ac=P + 0x3000,
            ld_acc=2048 * 64, ws=P + 0x100000, nb=1 << 34):
        a = a if a is not None else _attn(dsa)
        return dsa.LIB.dsa_kv8_accumulate(ctypes.byref(a), _p(e), _p(idx), ld, k, _p(lse), decay, _p(ac),
                                          ld_acc, _p(ws), nb, None)
    for f in (fwd, acc):
        _expect(dsa, dsa.DSA_ERR_CUDA, lambda: f())
        _expect(dsa, dsa.DSA_ERR_CUDA, lambda: f(idx=None, k=0, ld=0))
        _expect(dsa, dsa.DSA_ERR_CUDA, lambda: f(_attn(dsa, 1)))
        for st, kw in ((INV, dict(e=None)), (INV, dict(k=0)), (INV, dict(k=2049)), (INV, dict(ld=2047))):
            _expect(dsa, st, lambda: f(**kw))
        for st, kw in ((INV, dict(q=None)), (INV, dict(kv=None)), (INV, dict(scale=0.0)),
                       (INV, dict(scale=float("nan"))), (UNS, dict(dtype=dsa.DSA_F32)), (UNS, dict(d_qk=512)),
                       (UNS, dict(d_v=256)), (UNS, dict(v=P)), (INV, dict(heads=0)),
                       (UNS, dict(heads=129, ld_q=129 * 576)), (INV, dict(ld_q=576)), (INV, dict(ld_kv=570)),
                       (INV, dict(ld_kv=584)), (INV, dict(ld_q=128 * 576 + 4)), (INV, dict(q=FAKE + 4)),
                       (INV, dict(kv=FAKE + 8)), (INV, dict(n_q=0)), (INV, dict(n_q=65))):
            _expect(dsa, st, lambda: f(_mut(_attn(dsa), **kw)))
        need = dsa.dsa_workspace_size(dsa.DSA_OP_KV8_MQA if f is fwd else dsa.DSA_OP_KV8_ACCUMULATE, None,
                                      dsa._Keep(_attn(dsa), []), 0, 0, 2048)
        if need:
            _expect(dsa, dsa.DSA_ERR_CUDA, lambda: f(nb=need))
            for kw in (dict(ws=None), dict(ws=P + 0x100080), dict(nb=need - 1)):
                _expect(dsa, WS, lambda: f(**kw))
    _expect(dsa, INV, lambda: fwd(out=None))
    _expect(dsa, INV, lambda: fwd(out=P + 8))
    for kw in (dict(lse=None), dict(ac=None), dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")),
               dict(ld_acc=2048 * 64 - 1)):
        _expect(dsa, INV, lambda: acc(**kw))
    out = ctypes.c_size_t(0)
    for op in (dsa.DSA_OP_KV8_MQA, dsa.DSA_OP_KV8_ACCUMULATE):
        a = _attn(dsa)
        for k in (-1, 2049):
            assert dsa.LIB.dsa_workspace_size(op, None, ctypes.byref(a), 0, 0, k, ctypes.byref(out)) == INV
        assert dsa.LIB.dsa_workspace_size(op, None, None, 0, 0, 64, ctypes.byref(out)) == INV


def test_evict_refusals(dsa):
    INV, UNS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED

    def ev(c=None, ik=None, ld_ik=0, iks=None, acc=P, ld_acc=2048 * 64, budget=1000, sink=4, recent=100,
           dst=P + 0x1000, ld_dst=16, lens=P + 0x2000, kept=P + 0x3000, ld_kept=1000, ao=P + 0x4000, ld_ao=1024):
        c = c if c is not None else _cache(dsa)
        return dsa.LIB.dsa_kv8_evict(ctypes.byref(c), _p(ik), ld_ik, _p(iks), _p(acc), ld_acc, budget, sink, recent,
                                     _p(dst), ld_dst, _p(lens), _p(kept), ld_kept, _p(ao), ld_ao, None)
    keys = dict(ik=P + 0x5000, ld_ik=128, iks=P + 0x6000)
    _expect(dsa, dsa.DSA_ERR_CUDA, lambda: ev())
    _expect(dsa, dsa.DSA_ERR_CUDA, lambda: ev(**keys))
    _expect(dsa, UNS, lambda: ev(_cache(dsa, _contig(dsa), 100)))
    for kw in (dict(acc=None), dict(dst=None), dict(lens=None), dict(kept=None), dict(ao=None), dict(budget=0),
               dict(sink=-1), dict(recent=-1), dict(sink=950), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1),
               dict(ld_acc=100), dict(ld_dst=15), dict(ld_kept=999), dict(ld_ao=999), dict(ik=P), dict(iks=P),
               dict(keys, ld_ik=120), dict(keys, ld_ik=136), dict(keys, ik=P + 8)):
        _expect(dsa, INV, lambda: ev(**kw))
    _expect(dsa, INV, lambda: ev(_mut(_cache(dsa), codes=None)))


def test_binding_refuses_other_element_types(dsa):
    codes, exps = torch.zeros(2, 64, 576, dtype=torch.uint8), torch.zeros(2, dtype=torch.int8)
    with pytest.raises(dsa.DsaError):
        dsa.kv8_cache(codes, exps.int())
    with pytest.raises(dsa.DsaError):
        dsa.kv8_cache(codes.float(), exps)
    cache = dsa.kv8_cache(codes[0], exps)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_kv8_store(cache, torch.zeros(1, 576, dtype=torch.float16))
