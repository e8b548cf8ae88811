"""Workloads of the 8-bit latent-cache operators, in their plain form and as calls of the library.

The latent KV cache holds e4m3 codes of 576-wide rows (512 latent + 64 rope columns) with one power-of-two
scale 2^e for every page of 64 tokens (the cache has a single head, shared by all query heads). Four
operators work on it:

  store       quantise new rows into their pages; a page that already holds rows takes the larger of its
              exponent and the one the new rows need, and its earlier codes are rewritten to it
  attn        softmax(scale q.k) v over the listed keys of each query ("sparse") or over every preceding
              key ("dense"), with all query heads on the same rows, keys all 576 and values the first 512
              columns; also the log-sum-exp of each head
  accumulate  each cached token's running attention weight, the mean over the heads added to decay * acc
  evict       keep `budget` tokens of each sequence (the first `sink`, the last `recent`, and in between
              those of the largest weight, ties to the lower index) and move them, in order, into new pages

run() is one pass; with own False in elementary torch operations in 32 bits, else through the library.
"""
import math

import torch

own = False

D, DV, PAGE, D_IDX = 576, 512, 64, 128
SCALE = 1.0 / math.sqrt(D)
MAX_CODE = 448.0
E_MIN, E_MAX = -64, 63


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token for each of 64 decoding sequences: the smallest call, all latency
        {"name": "store_decode_64", "op": "store", "n_seq": 64, "rows_lo": 1, "rows_hi": 1, "old_lo": 1023,
         "old_hi": 32767, "dtype": "bf16", "paged": True},
        # a step of chunked prefill: a few prompts of odd lengths behind what their pages already hold
        {"name": "store_prefill_ragged", "op": "store", "n_seq": 7, "rows_lo": 1500, "rows_hi": 16384, "old_lo": 0,
         "old_hi": 8191, "dtype": "bf16", "paged": True},
        # fp32 rows of one long prompt in a contiguous cache
        {"name": "store_contig_f32", "op": "store", "n_seq": 1, "rows_lo": 32741, "rows_hi": 32741, "old_lo": 37,
         "old_hi": 37, "dtype": "f32", "paged": False},
        # the decode workload: 64 sequences, 2048 selected keys each, all 128 heads
        {"name": "attn_sparse_decode_64", "op": "attn", "mode": "sparse", "n_seq": 64, "q_per_seq": 1, "heads": 128,
         "k": 2048, "ctx_lo": 8192, "ctx_hi": 131072, "paged": True},
        # one sequence on a GPU that holds 16 of the heads: latency
        {"name": "attn_sparse_one_h16", "op": "attn", "mode": "sparse", "n_seq": 1, "q_per_seq": 1, "heads": 16,
         "k": 2048, "ctx_lo": 30001, "ctx_hi": 30001, "paged": True},
        # a chunk of a 32K prefill over its selection
        {"name": "attn_sparse_chunk", "op": "attn", "mode": "sparse", "n_seq": 1, "q_per_seq": 1021, "heads": 128,
         "k": 2048, "ctx_lo": 32768, "ctx_hi": 32768, "paged": False},
        # dense attention of ragged long sequences (no selection), all heads: bound by the tensor cores
        {"name": "attn_dense_decode_h128", "op": "attn", "mode": "dense", "n_seq": 12, "q_per_seq": 1, "heads": 128,
         "k": 0, "ctx_lo": 8192, "ctx_hi": 131072, "paged": True},
        # the same with 16 heads a GPU: bound by the cache's bytes
        {"name": "attn_dense_decode_h16", "op": "attn", "mode": "dense", "n_seq": 8, "q_per_seq": 1, "heads": 16,
         "k": 0, "ctx_lo": 65536, "ctx_hi": 131072, "paged": True},
        # weights of the decode workload's step, and of a dense step with two new tokens a sequence
        {"name": "accumulate_sparse_64", "op": "accumulate", "mode": "sparse", "n_seq": 64, "q_per_seq": 1,
         "heads": 128, "k": 2048, "ctx_lo": 8192, "ctx_hi": 131072, "paged": True, "decay": 1.0},
        {"name": "accumulate_dense_h32", "op": "accumulate", "mode": "dense", "n_seq": 6, "q_per_seq": 2,
         "heads": 32, "k": 0, "ctx_lo": 8192, "ctx_hi": 65536, "paged": True, "decay": 0.98},
        # a few short sequences, and a batch of long ones brought down to 8192 tokens each
        {"name": "evict_small", "op": "evict", "n_seq": 3, "ctx_lo": 700, "ctx_hi": 3001, "budget": 641, "sink": 4,
         "recent": 129, "idx_keys": False},
        {"name": "evict_batch", "op": "evict", "n_seq": 24, "ctx_lo": 16384, "ctx_hi": 65536, "budget": 8192,
         "sink": 64, "recent": 1024, "idx_keys": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "accumulate", "evict"])
    if op == "store":
        paged = rng.random() < 0.7
        n = _log(rng, 1, 96) if paged else 1
        hi = _log(rng, 1, max(1, 50000 // n))
        old = _log(rng, 1, 16384) if rng.random() < 0.8 else 0
        return {"op": "store", "n_seq": n, "rows_lo": 0 if n > 1 and rng.random() < 0.3 else max(1, hi // 3),
                "rows_hi": hi, "old_lo": old // 2 if paged else old, "old_hi": old,
                "dtype": rng.choice(["bf16", "f32"]), "paged": paged}
    if op == "evict":
        n = _log(rng, 1, 32)
        hi = _log(rng, 64, min(65536, 1200000 // n))
        budget = _log(rng, 8, min(16384, max(9, hi)))
        recent = rng.randint(0, budget // 2)
        return {"op": "evict", "n_seq": n, "ctx_lo": max(1, hi // 4), "ctx_hi": hi, "budget": budget,
                "sink": rng.randint(0, budget // 4), "recent": recent, "idx_keys": rng.random() < 0.6}
    dense = rng.random() < 0.45
    paged = dense or rng.random() < 0.7
    heads = rng.choice([1, 8, 16, 24, 32, 48, 64, 100, 128])
    n = _log(rng, 1, 10 if dense else 64) if paged else 1
    per = rng.randint(1, 4) if paged else _log(rng, 1, 900)
    hi = _log(rng, max(1, per), (min(131072, 600000 // (n * per)) if dense else 131072 if paged else 32768))
    k = 0 if dense else _log(rng, 1, 2048)
    if not dense and paged and n * per > 64:
        per = 1
    c = {"op": op, "mode": "dense" if dense else "sparse", "n_seq": n, "q_per_seq": per, "heads": heads, "k": k,
         "ctx_lo": max(per, hi // 4) if paged else max(per, hi), "ctx_hi": max(per, hi), "paged": paged}
    if op == "accumulate":
        c["decay"] = rng.choice([1.0, 0.98])
    return c


# ------------------------------------------------------------------------------------------ inputs

def _seeded(seed):
    return torch.Generator(device="cuda").manual_seed(seed), torch.Generator().manual_seed(seed)


def _table(lens, extra, cg, g):
    """A shuffled block table over all pages of the sequences, -1 past each; the number of pages."""
    pages = [-(-max(n, 1) // PAGE) for n in lens]
    total = sum(pages) + extra
    perm = torch.randperm(total, generator=cg).to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    off = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[off:off + n]
        off += n
    return table.cuda(), perm[off:].cuda(), total


def _rows(n, g, dtype=torch.bfloat16):
    """Latent rows: normal draws with a gain of each token's own and a wider rope part, made in pieces."""
    out = torch.empty(n, D, dtype=dtype, device="cuda")
    for r in range(0, n, 1 << 18):
        m = min(n, r + (1 << 18)) - r
        x = torch.randn(m, D, generator=g, device="cuda")
        x *= torch.exp2(0.5 * torch.randn(m, 1, generator=g, device="cuda"))
        x[:, DV:] *= 1.5
        out[r:r + m] = x
    return out


def _pool(num_pages, g):
    """A filled cache: codes [num_pages, 64, 576] and exponents [num_pages]."""
    codes = torch.empty(num_pages, PAGE, D, dtype=torch.uint8, device="cuda")
    exps = torch.empty(num_pages, dtype=torch.int8, device="cuda")
    step = 4096
    for p in range(0, num_pages, step):
        n = min(num_pages, p + step) - p
        x = _rows(n * PAGE, g, torch.float32).view(n, PAGE, D)
        e = _need(x.abs().amax(dim=(1, 2)))
        codes[p:p + n] = _encode(x, e[:, None, None])
        exps[p:p + n] = e
    return codes, exps


def _need(amax):
    """The smallest exponent e with amax <= 448 * 2^e, in [-64, 63]: int8."""
    m, x = torch.frexp(amax.float())
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX).to(torch.int8)


def _encode(x, e):
    y = torch.ldexp(x.float(), -e.to(torch.int32)).clamp(-MAX_CODE, MAX_CODE)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _lens(case, lo="ctx_lo", hi="ctx_hi"):
    """Ragged lengths: they belong to the case, so that outputs of all seeds have the same shapes."""
    g = torch.Generator().manual_seed(31 * case[hi] + case["n_seq"])
    return torch.randint(case[lo], case[hi] + 1, (case["n_seq"],), generator=g).tolist()


def prepare(case, seed):
    g, cg = _seeded(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "store":
        n_new = _lens(case, "rows_lo", "rows_hi")
        if sum(n_new) == 0:
            n_new[-1] = 1
        old = _lens(case, "old_lo", "old_hi")
        lens = [a + b for a, b in zip(n_new, old)]
        s["rows"] = _rows(sum(n_new), g, torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["cu"] = torch.tensor([0] + n_new).cumsum(0).to(torch.int32).cuda()
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["paged"]:
            s["table"], _, s["num_pages"] = _table(lens, 3, cg, g)
        else:
            n = -(-lens[0] // PAGE)
            s["table"], s["num_pages"] = torch.arange(n, dtype=torch.int32, device="cuda")[None], n
        s["n_keys"] = lens[0]
        s["codes"], s["exps"] = _pool(s["num_pages"], g)
        return s
    if case["op"] == "evict":
        lens = _lens(case)
        kept = [min(n, case["budget"]) for n in lens]
        need = [-(-n // PAGE) for n in kept]
        s["table"], free, s["num_pages"] = _table(lens, sum(need), cg, g)
        dst = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
        off = 0
        for b, n in enumerate(need):
            dst[b, :n] = free[off:off + n]
            off += n
        s["dst"] = dst
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["codes"], s["exps"] = _pool(s["num_pages"], g)
        n = s["table"].shape[1] * PAGE
        # accumulated weights fall off steeply; many tokens have never been chosen and stand at zero
        acc = torch.rand(len(lens), n, generator=g, device="cuda") ** 6
        s["acc"] = torch.where(torch.rand(len(lens), n, generator=g, device="cuda") < 0.3, torch.zeros_like(acc), acc)
        s["kept"] = torch.empty(len(lens), case["budget"], dtype=torch.int32, device="cuda")
        s["lens"] = torch.empty(len(lens), dtype=torch.int32, device="cuda")
        s["acc_out"] = torch.zeros(len(lens), dst.shape[1] * PAGE, device="cuda")
        if case["idx_keys"]:
            s["ik"] = torch.randint(0, 255, (s["num_pages"], PAGE, D_IDX), generator=g, device="cuda").to(torch.uint8)
            s["ik"] &= 0x77
            s["iks"] = torch.rand(s["num_pages"], PAGE, generator=g, device="cuda") + 0.5
        return s
    # attention and its weights
    n_seq, per, H, k = case["n_seq"], case["q_per_seq"], case["heads"], case["k"]
    lens = _lens(case)
    n_q = n_seq * per
    s["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["paged"]:
        s["table"], _, s["num_pages"] = _table(lens, 0, cg, g)
    else:
        n = -(-lens[0] // PAGE)
        s["table"], s["num_pages"] = torch.arange(n, dtype=torch.int32, device="cuda")[None], n
    s["n_keys"] = lens[0]
    s["codes"], s["exps"] = _pool(s["num_pages"], g)
    s["q"] = torch.randn(n_q, H, D, generator=g, device="cuda").to(torch.bfloat16)
    s["seq"] = torch.arange(n_q, device="cuda") // per
    # the newest `per` tokens of each sequence are the queries
    s["pos"] = s["ctx"].long()[s["seq"]] - per + torch.arange(n_q, device="cuda") % per
    if case["mode"] == "sparse":
        # one key from each of k strata of the prefix; every preceding key where there are no more than k
        j = torch.arange(k, device="cuda", dtype=torch.float64)
        p1 = s["pos"].double()[:, None] + 1
        lo, hi = torch.floor(j * p1 / k), torch.floor((j + 1) * p1 / k)
        pick = lo + torch.floor(torch.rand(n_q, k, generator=g, device="cuda", dtype=torch.float64) * (hi - lo))
        s["idx"] = torch.where(p1 > k, pick, torch.where(j < p1, j, torch.full_like(pick, -1))).to(torch.int32)
    s["q_seq"], s["q_pos"] = s["seq"].to(torch.int32), s["pos"].to(torch.int32)
    s["out"] = torch.empty(n_q, H, DV, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(n_q, H, device="cuda")
    if case["op"] == "accumulate":
        s["lse"] = _attend(s)[1]
        s["acc"] = 1e-3 * torch.rand(n_seq, s["table"].shape[1] * PAGE, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _keys(s):
    """Positions [n, keys] of each query's keys and which of them count. Dense: one row a sequence."""
    if s["case"]["mode"] == "sparse":
        return s["idx"].long().clamp(min=0), s["idx"] >= 0
    n = int(s["table"].shape[1]) * PAGE
    p = torch.arange(n, device="cuda")[None]
    return p.expand(s["case"]["n_seq"], n), p <= s["pos"][:, None]


def _gather(s, seq, p):
    """The cache's rows at positions p [n, keys] of the sequences seq [n], as the values they stand for."""
    page = s["table"].long()[seq[:, None], p // PAGE].clamp(min=0)
    codes = s["codes"].view(-1, D)[page * PAGE + p % PAGE]
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), s["exps"].to(torch.int32)[page][..., None])


def _logits(s):
    p, ok = _keys(s)
    n_q, H = s["q"].shape[:2]
    n = p.shape[0]
    x = _gather(s, s["seq"] if s["case"]["mode"] == "sparse" else torch.arange(n, device="cuda"), p)
    z = torch.matmul(s["q"].float().view(n, -1, D), x.transpose(1, 2)).view(n_q, H, -1) * SCALE
    return x, torch.where(ok[:, None], z, torch.full_like(z, -math.inf)), p, ok


def _attend(s):
    x, z, _, _ = _logits(s)
    n_q, H = s["q"].shape[:2]
    m = z.amax(dim=2, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(z - m)
    l = p.sum(dim=2, keepdim=True)
    o = torch.matmul(p.view(x.shape[0], -1, x.shape[1]), x[..., :DV]).view(n_q, H, DV)
    return torch.where(l > 0, o / l, torch.zeros_like(o)).to(torch.bfloat16), (m + torch.log(l))[..., 0]


def _accumulate(s):
    _, z, p, ok = _logits(s)
    w = torch.exp(z - s["lse"][..., None]).mean(dim=1)
    n_seq, width = s["acc"].shape
    live = torch.arange(width, device="cuda")[None] < s["ctx"][:, None]
    s["acc"] = torch.where(live, s["acc"] * s["case"]["decay"], s["acc"])
    if s["case"]["mode"] == "dense":
        s["acc"] += w.view(n_seq, -1, width).sum(dim=1)
    else:
        s["acc"].view(-1).index_add_(0, (s["seq"][:, None] * width + p).reshape(-1),
                                     torch.where(ok, w, torch.zeros_like(w)).reshape(-1))
    return s["acc"]


def _store(s):
    rows, cu, ctx = s["rows"], s["cu"].long(), s["ctx"].long()
    i = torch.arange(rows.shape[0], device="cuda")
    seq = torch.searchsorted(cu, i, right=True) - 1
    pos = ctx[seq] - (cu[seq + 1] - cu[seq]) + i - cu[seq]
    page = s["table"].long()[seq, pos // PAGE]
    amax = torch.zeros(s["num_pages"], device="cuda").scatter_reduce(0, page, rows.abs().amax(dim=1).float(), "amax")
    first = torch.full((s["num_pages"],), PAGE, device="cuda").scatter_reduce(0, page, pos % PAGE, "amin")
    touched = first < PAGE
    need = _need(amax)
    kept = touched & (first > 0)
    e = torch.where(kept, torch.maximum(need, s["exps"]), torch.where(touched, need, s["exps"]))
    # at most the first page of each sequence's run holds earlier rows: rewrite them to the new exponent
    at = page[cu[:-1].clamp(max=rows.shape[0] - 1)]
    before = torch.arange(PAGE, device="cuda")[None] < torch.where(kept[at], first[at], torch.zeros_like(first[at]))[:, None]
    held = s["codes"][at]
    again = torch.ldexp(held.view(torch.float8_e4m3fn).float(), (s["exps"][at].int() - e[at].int())[:, None, None])
    s["codes"][at] = torch.where(before[..., None], _encode(again, torch.zeros_like(e[at])[:, None, None]), held)
    s["codes"].view(-1, D)[page * PAGE + pos % PAGE] = _encode(rows, e[page][:, None])
    s["exps"].copy_(e)
    return s["codes"].view(torch.float8_e4m3fn), s["exps"]


def _evict(s):
    case, acc, ctx = s["case"], s["acc"], s["ctx"].long()
    n_seq, width = acc.shape
    budget = case["budget"]
    p = torch.arange(width, device="cuda")[None]
    always = (p < case["sink"]) | (p >= ctx[:, None] - case["recent"])
    key = torch.where(p >= ctx[:, None], torch.full_like(acc, -math.inf),
                      torch.where(always, torch.full_like(acc, math.inf), acc))
    kept = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
    kept = torch.sort(torch.cat([kept, kept.new_full((n_seq, budget - kept.shape[1]), width)], dim=1)).values
    ok = kept < ctx[:, None]
    src = torch.where(ok, kept, torch.zeros_like(kept))
    page = s["table"].long()[torch.arange(n_seq, device="cuda")[:, None], src // PAGE]
    j = torch.arange(budget, device="cuda")
    to = s["dst"].long()[:, torch.clamp(j // PAGE, max=s["dst"].shape[1] - 1)]
    e_src = torch.where(ok, s["exps"][page].int(), torch.full_like(src, E_MIN, dtype=torch.int32))
    e = torch.full((s["num_pages"],), E_MIN, dtype=torch.int32, device="cuda")
    e = e.scatter_reduce(0, to[ok], e_src[ok], "amax")
    to_row = (to * PAGE + j % PAGE)[ok]
    from_row = (page * PAGE + src % PAGE)[ok]
    x = s["codes"].view(-1, D)[from_row].view(torch.float8_e4m3fn).float()
    y = torch.ldexp(x, (e_src - e[to.clamp(min=0)])[ok][:, None])
    s["codes"].view(-1, D)[to_row] = _encode(y, torch.zeros_like(to_row)[:, None])
    s["exps"][to[ok]] = e[to[ok]].to(torch.int8)
    s["kept"] = torch.where(ok, kept, torch.full_like(kept, -1)).to(torch.int32)
    s["lens"] = torch.clamp(ctx, max=budget).to(torch.int32)
    cols = min(budget, s["acc_out"].shape[1])
    s["acc_out"][:, :cols] = torch.where(ok, torch.gather(acc, 1, src), torch.zeros((), device="cuda"))[:, :cols]
    got = [s["kept"], s["lens"], s["acc_out"], s["codes"].view(torch.float8_e4m3fn), s["exps"]]
    if case["idx_keys"]:
        s["ik"].view(-1, D_IDX)[to_row] = s["ik"].view(-1, D_IDX)[from_row]
        s["iks"].view(-1)[to_row] = s["iks"].view(-1)[from_row]
        got += [s["ik"].view(torch.float8_e4m3fn), s["iks"]]
    return got


# ------------------------------------------------------------------------------------------ the library's calls

def _layout(dsa, s, queries=True):
    case = s["case"]
    if not case.get("paged", True):
        return None
    several = queries and case["q_per_seq"] > 1
    return dsa.paged_layout(s["table"], s["ctx"], s["num_pages"], s["q_seq"] if several else None,
                            s["q_pos"] if several else None)


def _own(s):
    from sparse_attention_long_tcgen05_b200 import dsa
    case = s["case"]
    if case["op"] == "store":
        cache = dsa.kv8_cache(s["codes"], s["exps"], _layout(dsa, s, False), s["n_keys"])
        dsa.dsa_kv8_store(cache, s["rows"], s["cu"] if case["paged"] else None)
        return s["codes"].view(torch.float8_e4m3fn), s["exps"]
    if case["op"] == "evict":
        cache = dsa.kv8_cache(s["codes"], s["exps"], _layout(dsa, s, False))
        # the new tables span the budget; those of sequences that are all well below it are shorter
        dst, acc_out, more = s["dst"], s["acc_out"], -(-case["budget"] // PAGE) - s["dst"].shape[1]
        if more > 0:
            dst = torch.nn.functional.pad(dst, (0, more), value=-1)
            acc_out = torch.nn.functional.pad(acc_out, (0, more * PAGE))
        dsa.dsa_kv8_evict(cache, s["acc"], case["budget"], case["sink"], case["recent"], dst, s["lens"],
                          s["kept"], acc_out, s.get("ik"), s.get("iks"))
        if more > 0:
            s["acc_out"].copy_(acc_out[:, :s["acc_out"].shape[1]])
        got = [s["kept"], s["lens"], s["acc_out"], s["codes"].view(torch.float8_e4m3fn), s["exps"]]
        if case["idx_keys"]:
            got += [s["ik"].view(torch.float8_e4m3fn), s["iks"]]
        return got
    codes = s["codes"] if case["paged"] else s["codes"].view(-1, D)[:s["n_keys"]]
    att = dsa.attn_in(s["q"], codes, SCALE, DV, kv_layout=_layout(dsa, s))
    idx, k = s.get("idx"), case["k"]
    if case["op"] == "attn":
        ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_MQA, None, att, 0, 0, k))
        dsa.dsa_kv8_mqa_fwd(att, s["exps"], idx, k, s["out"], s["lse"], ws)
        return s["out"], s["lse"]
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_KV8_ACCUMULATE, None, att, 0, 0, k))
    dsa.dsa_kv8_accumulate(att, s["exps"], idx, k, s["lse"], case["decay"], s["acc"], ws)
    return s["acc"]


def run(s):
    if own:
        return _own(s)
    return {"store": _store, "attn": _attend, "accumulate": _accumulate, "evict": _evict}[s["op"]](s)


# ------------------------------------------------------------------------------------------ work and exact values

def work(case):
    n = case["n_seq"]
    mean = lambda lo, hi: (case[lo] + case[hi]) / 2  # noqa: E731
    if case["op"] == "store":
        r = n * max(1.0, mean("rows_lo", "rows_hi"))
        return {"bytes": r * D * (1 + (2 if case["dtype"] == "bf16" else 4)), "flops": r * D}
    if case["op"] == "evict":
        ctx = mean("ctx_lo", "ctx_hi")
        r = n * min(case["budget"], ctx)
        row = D + 8 + (D_IDX + 4 if case["idx_keys"] else 0)
        return {"bytes": n * ctx * 4 + 2 * r * row, "flops": n * ctx}
    ctx, H, per, k = mean("ctx_lo", "ctx_hi"), case["heads"], case["q_per_seq"], case["k"]
    pairs = n * per * (min(k, ctx) if case["mode"] == "sparse" else ctx)
    rows = min(n * ctx, pairs)
    q = n * per * H * (2 * D + 4)
    if case["op"] == "attn":
        return {"bytes": rows * D + q + n * per * H * 2 * DV + (4 * pairs if k else 0), "flops": 2.0 * H * (D + DV) * pairs}
    moved = 8 * (rows if k and case["decay"] == 1.0 else n * ctx)
    return {"bytes": rows * D + q + moved + (4 * pairs if k else 0), "flops": 2.0 * H * D * pairs}


def _round64(v):
    """v rounded to e4m3, to the nearest and ties to even, in 64 bits: within +-448, quantum 2^(x - 3), x >= -6."""
    v = v.clamp(-448.0, 448.0)
    x = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    x = torch.where(torch.exp2(x) > v.abs(), x - 1, x).clamp(min=-6)
    step = torch.exp2(x - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _value64(codes):
    c = codes.long()
    mant, ex = c & 7, (c >> 3) & 15
    v = torch.where(ex > 0, (8 + mant).double() * torch.exp2((ex - 10).double()), mant.double() * 2.0 ** -9)
    return torch.where(c >= 128, -v, v)


def _least64(a):
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
    return torch.where(a > 0, e, torch.full_like(e, -64.0)).clamp(-64, 63)


def exact(case, seed):
    s = prepare(case, seed)
    table, ctx = s["table"].tolist(), s["ctx"].tolist()
    if case["op"] == "store":
        vals, cu = _value64(s["codes"]), s["cu"].tolist()
        exps = s["exps"].double()
        if case["n_seq"] > 200 or sum(cu[b + 1] - cu[b] for b in range(case["n_seq"])) > 70000:
            return None
        for b in range(case["n_seq"]):
            i = cu[b]
            while i < cu[b + 1]:
                p = ctx[b] - cu[b + 1] + i
                pg, slot = table[b][p // 64], p % 64
                m = min(cu[b + 1] - i, 64 - slot)
                new = s["rows"][i:i + m].double()
                e = _least64(new.abs().max())
                if slot:
                    e = torch.maximum(e, exps[pg])
                    vals[pg, :slot] = _round64(vals[pg, :slot] * torch.exp2(exps[pg] - e))
                vals[pg, slot:slot + m] = _round64(new * torch.exp2(-e))
                exps[pg] = e
                i += m
        return vals, None
    if case["op"] == "evict":
        vals, exps = _value64(s["codes"]), s["exps"].double()
        old, olde, acc_out = vals.clone(), exps.clone(), s["acc_out"].double()
        ik = _value64(s["ik"]) if case["idx_keys"] else None
        iks = s["iks"].double() if case["idx_keys"] else None
        for b, n in enumerate(ctx):
            lo, hi = min(case["sink"], n), max(min(case["sink"], n), n - case["recent"])
            if n > case["budget"]:
                w = s["acc"][b, lo:hi].double()
                i = torch.arange(hi - lo, device="cuda")
                mid = sorted(zip((-w).tolist(), i.tolist()))[:case["budget"] - lo - (n - hi)]
                keep = list(range(lo)) + sorted(lo + i for _, i in mid) + list(range(hi, n))
            else:
                keep = list(range(n))
            src = torch.tensor(keep, device="cuda")
            acc_out[b, :len(keep)] = s["acc"][b].double()[src]
            pg = s["table"][b].long()[src // 64]
            for d in range(-(-len(keep) // 64)):
                a, to = slice(64 * d, min(64 * d + 64, len(keep))), int(s["dst"][b, d])
                m = a.stop - a.start
                e = olde[pg[a]].max()
                vals[to, :m] = _round64(old[pg[a], src[a] % 64] * torch.exp2(olde[pg[a]] - e)[:, None])
                if ik is not None:
                    ik[to, :m], iks[to, :m] = ik[pg[a], src[a] % 64], iks[pg[a], src[a] % 64]
        return [None, None, acc_out, vals, None] + ([ik, iks] if ik is not None else [])
    n_q, H = s["q"].shape[:2]
    if n_q * H * max(ctx) * (case["mode"] == "dense") > 4e9:
        return None
    out, lse = torch.zeros(n_q, H, DV, dtype=torch.float64, device="cuda"), torch.empty(n_q, H, dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if case["op"] == "accumulate" else None
    if acc is not None:
        for b, n in enumerate(ctx):
            acc[b, :n] *= case["decay"]
    for i in range(n_q):
        b, pos = int(s["seq"][i]), int(s["pos"][i])
        p = torch.arange(pos + 1, device="cuda") if case["mode"] == "dense" else s["idx"][i][s["idx"][i] >= 0].long()
        pg = s["table"][b].long()[p // 64]
        x = _value64(s["codes"].view(-1, D)[pg * 64 + p % 64]) * torch.exp2(s["exps"][pg].double())[:, None]
        z = s["q"][i].double() @ x.T / math.sqrt(576.0)
        if acc is not None:
            acc[b].index_add_(0, p, torch.exp(z - s["lse"][i].double()[:, None]).mean(dim=0))
        else:
            lse[i] = torch.logsumexp(z, dim=1)
            out[i] = torch.exp(z - lse[i][:, None]) @ x[:, :512]
    return acc if acc is not None else (out, lse)
