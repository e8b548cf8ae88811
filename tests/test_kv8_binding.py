"""The binding's refusals for the 8-bit latent cache, on the CPU: tensors that the C
side would misread or write past are refused before any address is taken. A call
that is right but for its tensors lying on the CPU gets as far as the check of the
device."""
import pytest
import torch

N_SEQ, PAGES, H, K_SEL, BUDGET = 3, 20, 4, 32, 100


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_tcgen05_b200 import _build
    _build.build()
    from sparse_attention_long_tcgen05_b200 import dsa
    return dsa


def _tensors():
    i32 = dict(dtype=torch.int32)
    return {"table": torch.zeros(N_SEQ, 4, **i32), "ctx": torch.ones(N_SEQ, **i32),
            "codes": torch.zeros(PAGES, 64, 576, dtype=torch.uint8), "exps": torch.zeros(PAGES, dtype=torch.int8),
            "rows": torch.zeros(N_SEQ, 576, dtype=torch.bfloat16), "cu": torch.arange(N_SEQ + 1, **i32),
            "q": torch.zeros(N_SEQ, H, 576, dtype=torch.bfloat16), "idx": torch.zeros(N_SEQ, K_SEL, **i32),
            "out": torch.zeros(N_SEQ, H, 512, dtype=torch.bfloat16), "lse": torch.zeros(N_SEQ, H),
            "ws": torch.zeros(1 << 20, dtype=torch.uint8), "acc": torch.zeros(N_SEQ, 256),
            "dst": torch.zeros(N_SEQ, 2, **i32), "lens": torch.zeros(N_SEQ, **i32),
            "kept": torch.zeros(N_SEQ, BUDGET, **i32), "acc_out": torch.zeros(N_SEQ, BUDGET),
            "ik": torch.zeros(PAGES, 64, 128, dtype=torch.uint8), "iks": torch.zeros(PAGES, 64)}


def _calls(dsa):
    def lay(t):
        return dsa.paged_layout(t["table"], t["ctx"], PAGES)

    def att(t):
        return dsa.attn_in(t["q"], t["codes"], 0.1, 512, kv_layout=lay(t))
    return {
        "store": lambda t: dsa.dsa_kv8_store(dsa.kv8_cache(t["codes"], t["exps"], lay(t)), t["rows"], t["cu"]),
        "attend": lambda t: dsa.dsa_kv8_mqa_fwd(att(t), t["exps"], t["idx"], K_SEL, t["out"], t["lse"], t["ws"]),
        "weigh": lambda t: dsa.dsa_kv8_accumulate(att(t), t["exps"], t["idx"], K_SEL, t["lse"], 1.0, t["acc"], t["ws"]),
        "evict": lambda t: dsa.dsa_kv8_evict(dsa.kv8_cache(t["codes"], t["exps"], lay(t)), t["acc"], BUDGET, 1, 2,
                                             t["dst"], t["lens"], t["kept"], t["acc_out"], t["ik"], t["iks"])}


def _refused(dsa, call, message, **changed):
    with pytest.raises(dsa.DsaError, match=message) as e:
        _calls(dsa)[call]({**_tensors(), **changed})
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["store", "attend", "weigh", "evict"])
def test_tensors_elsewhere(dsa, call):
    _refused(dsa, call, "current device")


@pytest.mark.parametrize("call,names", [
    ("store", ["codes", "exps", "table", "ctx", "cu"]),
    ("attend", ["codes", "exps", "table", "ctx", "idx", "out", "lse"]),
    ("weigh", ["codes", "exps", "table", "ctx", "idx", "lse", "acc"]),
    ("evict", ["codes", "exps", "table", "ctx", "acc", "dst", "lens", "kept", "acc_out", "ik", "iks"])])
def test_element_types(dsa, call, names):
    other = {torch.int32: torch.int64, torch.float32: torch.float16, torch.bfloat16: torch.float16,
             torch.uint8: torch.int8, torch.int8: torch.uint8}
    for name in names:
        t = _tensors()[name]
        if name == "codes" and call in ("attend", "weigh"):
            t = t.to(torch.int8)                          # attn_in takes other types for other calls
            _refused(dsa, call, "must be torch", codes=t)
        else:
            _refused(dsa, call, "must be torch", **{name: t.to(other[t.dtype])})


@pytest.mark.parametrize("call", ["store", "attend", "weigh", "evict"])
def test_pages_of_a_pool_of_layers(dsa, call):
    """One layer of [pages, layers, 64, 576]: its pages do not follow one another."""
    pool = torch.zeros(PAGES, 3, 64, 576, dtype=torch.uint8)
    _refused(dsa, call, "follow one another", codes=pool[:, 1])
    _refused(dsa, call, "follow one another", codes=torch.zeros(2 * PAGES, 32, 576, dtype=torch.uint8))
    _refused(dsa, call, "rows of 576", codes=torch.zeros(PAGES, 64, 592, dtype=torch.uint8))
    _refused(dsa, call, "rows of 576", codes=torch.zeros(PAGES - 1, 64, 576, dtype=torch.uint8))
    _refused(dsa, call, "contiguous elements", exps=torch.zeros(PAGES - 1, dtype=torch.int8))
    wide = torch.zeros(PAGES, 64, 592, dtype=torch.uint8)
    _refused(dsa, call, "current device", codes=wide[:, :, :576])          # rows may be further apart
    _refused(dsa, call, "current device", codes=wide.view(-1, 592)[:, :576])


@pytest.mark.parametrize("call,name,bad", [
    ("store", "rows", lambda t: t[:, :512]), ("store", "rows", lambda t: t.t().contiguous().t()),
    ("store", "cu", lambda t: t[:-1]), ("store", "cu", lambda t: t.repeat_interleave(2)[::2]),
    ("store", "table", lambda t: t[:-1]), ("store", "table", lambda t: t.t().contiguous().t()),
    ("attend", "ctx", lambda t: t.repeat_interleave(2)[::2]),
    ("attend", "q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)),
    ("attend", "idx", lambda t: t[:-1]), ("attend", "idx", lambda t: t[:, :-1]),
    ("attend", "idx", lambda t: t.t().contiguous().t()), ("attend", "out", lambda t: t[:-1]),
    ("attend", "out", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)), ("attend", "lse", lambda t: t[:-1]),
    ("attend", "ws", lambda t: t[::2]), ("weigh", "acc", lambda t: t[:-1]), ("weigh", "acc", lambda t: t[:, :-1]),
    ("weigh", "lse", lambda t: t.t().contiguous().t()), ("evict", "acc", lambda t: t[:, :-1]),
    ("evict", "dst", lambda t: t[:, :-1]), ("evict", "lens", lambda t: t[:-1]), ("evict", "kept", lambda t: t[:, :-1]),
    ("evict", "acc_out", lambda t: t[:-1]), ("evict", "ik", lambda t: t[:-1]),
    ("evict", "ik", lambda t: t.repeat(1, 2, 1)[:, :64]), ("evict", "iks", lambda t: t[:-1])])
def test_shapes_and_strides(dsa, call, name, bad):
    _refused(dsa, call, "must", **{name: bad(_tensors()[name])})


def test_contiguous_caches(dsa):
    codes, exps = torch.zeros(200, 576, dtype=torch.uint8), torch.zeros(4, dtype=torch.int8)
    dsa.kv8_cache(codes, exps)
    dsa.kv8_cache(codes.view(2, 100, 576), exps, None, 200)
    q = torch.zeros(1, 4, 576, dtype=torch.bfloat16)
    dsa.attn_in(q, codes, 0.1, 512)
    for build in (lambda: dsa.kv8_cache(codes.view(2, 100, 576), exps),          # 2 keys?
                  lambda: dsa.attn_in(q, codes.view(2, 100, 576), 0.1, 512)):
        with pytest.raises(dsa.DsaError, match="must be .n_keys, 576."):
            build()
    with pytest.raises(dsa.DsaError, match="200|201"):
        dsa.kv8_cache(codes, exps, None, 201)
    with pytest.raises(dsa.DsaError, match="4 contiguous"):
        dsa.kv8_cache(codes, exps[:3])
    with pytest.raises(dsa.DsaError, match="follow one another"):
        dsa.kv8_cache(codes.view(2, 100, 576)[:, :90], exps, None, 180)
