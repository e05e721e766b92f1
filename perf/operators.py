"""Cases of the 4-bit paged cache and of cache eviction, with their plain forms.

Four operators, each with what a serving program holds when it calls them:

  store    write new K/V rows into a 4-bit pool (pa_reshape_and_cache, "int4") and read rows back as values
           (pa_gather_cache), as a prompt chunk is cached and later handed to a dense kernel
  attend   attention over a 4-bit pool: one query token per sequence (pa_decode) or several causal ones (pa_attention)
  observe  a decode step that also adds every key's softmax weight, summed over its group's heads, to a pool of
           accumulated weights (pa_decode_weights)
  evict    bring sequences down to a budget of tokens per KV head: sinks, the most attended and the most recent
           stay (pa_evict), in place or into other blocks

Layouts: 16- and 32-bit pools [num_blocks, block_size, num_kv_heads, head_dim]; a 4-bit pool is uint8
[num_blocks, block_size, num_kv_heads, head_dim / 2 + 4] whose blocks hold codes [num_kv_heads, block_size, head_dim / 2]
(dimension 2b in the low nibble of byte b), then float16 (step, low) [num_kv_heads, block_size, 2]: value = low + step * code.
Accumulated weights are float32 [num_blocks, num_kv_heads, block_size].
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
WIDTH = {"f16": 2.0, "bf16": 2.0, "f32": 4.0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the tokens of one decode step of a 64-sequence batch on a 7B-like layer: launch latency counts
        dict(name="store_step_f16", op="store", tokens=64, kv_heads=4, head_dim=128, block=16, dtype="f16"),
        # a long prompt of a 32/8-head layer
        dict(name="store_prompt_bf16", op="store", tokens=65536, kv_heads=8, head_dim=128, block=32, dtype="bf16"),
        # an odd count of float32 rows of the narrow head, small blocks
        dict(name="store_odd_f32_d64", op="store", tokens=5003, kv_heads=2, head_dim=64, block=8, dtype="f32"),
        # four short sequences on a small model: latency
        dict(name="attend_tiny_f16", op="attend", batch=4, lo=5, hi=40, q_heads=4, kv_heads=2, head_dim=64, block=16,
             queries=1, dtype="f16"),
        # a 7B-like layer, 64 sequences of 100 to 8192 tokens
        dict(name="attend_7b_f16", op="attend", batch=64, lo=100, hi=8192, q_heads=28, kv_heads=4, head_dim=128,
             block=16, queries=1, dtype="f16"),
        # a serving mix of many short sequences
        dict(name="attend_mix_bf16", op="attend", batch=1024, lo=20, hi=2048, q_heads=32, kv_heads=8, head_dim=128,
             block=16, queries=1, dtype="bf16"),
        # few long contexts
        dict(name="attend_long_bf16", op="attend", batch=8, lo=32768, hi=131072, q_heads=32, kv_heads=8, head_dim=128,
             block=32, queries=1, dtype="bf16"),
        # a speculative step: one to four causal query tokens per sequence
        dict(name="attend_spec_f16", op="attend", batch=64, lo=100, hi=8192, q_heads=28, kv_heads=4, head_dim=128,
             block=16, queries=4, dtype="f16"),
        # a decode step that keeps the weights that eviction reads, 7B-like layer, 16-bit cache
        dict(name="observe_7b_f16", op="observe", batch=64, lo=100, hi=8192, q_heads=28, kv_heads=4, head_dim=128,
             block=16, cache="f16", dtype="f16"),
        # the same on few long contexts held in 4 bits
        dict(name="observe_long_int4", op="observe", batch=8, lo=32768, hi=131072, q_heads=32, kv_heads=8,
             head_dim=128, block=32, cache="int4", dtype="bf16"),
        # steady serving: every sequence is one block over its budget and gives that block back
        dict(name="evict_block_f16", op="evict", batch=64, lo=2064, hi=2064, kv_heads=4, head_dim=128, block=16,
             budget=2048, sink=4, recent=256, in_place=True, dtype="f16"),
        # long prompts cut to a fixed budget, into other blocks (their own are shared)
        dict(name="evict_prompt_bf16", op="evict", batch=8, lo=32768, hi=131072, kv_heads=8, head_dim=128, block=32,
             budget=4096, sink=4, recent=512, in_place=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "observe", "evict"])
    head_dim = rng.choice([64, 128, 128])
    block = rng.choice([8, 16, 32, 64])
    kv_heads = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["f16", "bf16"])
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 65536), kv_heads=kv_heads, head_dim=head_dim, block=block,
                    dtype=rng.choice(["f16", "bf16", "f32"]))
    # lengths up to 131072 and up to half a million tokens times heads in all
    hi = _log_int(rng, 40, 131072)
    lo = max(1, int(hi * rng.uniform(0.02, 1.0)))
    most = max(1, min(512, 4000000 // (hi * kv_heads)))
    batch = _log_int(rng, 1, most)
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "attend":
        queries = rng.choice([1, 1, 2, 3, 5, 8])
        return dict(op=op, batch=batch, lo=lo, hi=hi, q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim,
                    block=block, queries=queries, dtype=dtype)
    if op == "observe":
        return dict(op=op, batch=batch, lo=lo, hi=hi, q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim,
                    block=block, cache=rng.choice([dtype, "int4"]), dtype=dtype)
    budget = max(2, int(hi * rng.uniform(0.05, 0.95)))
    recent = rng.randint(0, budget // 2)
    sink = rng.randint(0, min(8, budget - recent))
    return dict(op=op, batch=batch, lo=lo, hi=hi, kv_heads=kv_heads, head_dim=head_dim, block=block, budget=budget,
                sink=sink, recent=recent, in_place=rng.random() < 0.5, dtype=dtype)


def _lens(case):
    """Sequence lengths: the case's alone, the longest among them; a batch of over 100 has mostly short ones."""
    r = random.Random(case["batch"] * 1000003 + case["hi"])
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    if n > 100 and hi > 8 * lo:
        lens = [r.randint(lo, 2 * lo) if r.random() < 0.7 else int(math.exp(r.uniform(math.log(lo), math.log(hi))))
                for _ in range(n)]
    else:
        lens = [r.randint(lo, hi) for _ in range(n)]
    lens[r.randrange(n)] = hi
    return lens


def _query_counts(case):
    r = random.Random(case["batch"] * 7919 + case["queries"])
    c = [r.randint(1, case["queries"]) for _ in range(case["batch"])]
    c[0] = case["queries"]
    return c


def work(case):
    D, Hkv = case["head_dim"], case["kv_heads"]
    row4 = Hkv * (D // 2 + 4)                       # bytes of one token's 4-bit K (or V) row
    if case["op"] == "store":
        T, e = case["tokens"], WIDTH[case["dtype"]]
        # the values in, the codes out, the codes in, the values out; K and V; a slot each time
        return {"bytes": T * (2 * (2 * Hkv * D * e + 2 * row4) + 16.0), "flops": T * 2.0 * Hkv * D * 6}
    lens = _lens(case)
    if case["op"] == "evict":
        n, e, bud, rec, snk = float(sum(lens)), WIDTH[case["dtype"]], case["budget"], case["recent"], case["sink"]
        moved = 0.0
        for L in lens:
            if L <= bud:
                moved += 0 if case["in_place"] else L
            elif case["in_place"]:
                # the recent rows move down; a selected row moves if it lies past the kept region (any is as likely)
                moved += rec + (bud - snk - rec) * (L - bud) / max(1.0, L - rec - snk)
            else:
                moved += bud
        kept = sum(min(L, bud) for L in lens)
        return {"bytes": 4.0 * Hkv * n + moved * Hkv * (4 * D * e + 8) + 4.0 * Hkv * kept, "flops": n * Hkv}
    Hq, n = case["q_heads"], float(sum(lens))
    if case["op"] == "attend":
        counts = _query_counts(case)
        keys = float(sum(L * c for L, c in zip(lens, counts)))
        return {"bytes": 2 * n * row4 + sum(counts) * Hq * D * 2 * 2.0, "flops": 4.0 * keys * Hq * D}
    kv = row4 if case["cache"] == "int4" else Hkv * D * 2
    return {"bytes": 2 * n * kv + 8.0 * n * Hkv + len(lens) * Hq * D * 2 * 2.0, "flops": 4.0 * n * Hq * D}


# ---------------------------------------------------------------------------
# what a program holds before the call
# ---------------------------------------------------------------------------
def _tables(lens, block, order, first=0):
    """Block tables over consecutive entries of `order`, -1 behind each sequence's last block."""
    n = [-(-L // block) for L in lens]
    t = torch.full((len(lens), max(n)), -1, dtype=torch.int32)
    for i, k in enumerate(n):
        t[i, :k] = order[first:first + k].to(torch.int32)
        first += k
    return t, first


def _pack4(x, block):
    """A 4-bit pool of the rows x [num_blocks, block, kv_heads, head_dim]."""
    x = x.float().transpose(1, 2)
    low = x.amin(-1, keepdim=True).half()
    step = ((x.amax(-1, keepdim=True) - low.float()) / 15).half()
    c = ((x - low.float()) / step.float().clamp_min(1e-7)).round_().clamp_(0, 15).to(torch.uint8)
    NB, Hkv, bs, D = c.shape
    codes = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(NB, -1)
    par = torch.cat([step, low], -1).contiguous().view(torch.uint8).reshape(NB, -1)
    return torch.cat([codes, par], 1).view(NB, bs, Hkv, D // 2 + 4)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    D, Hkv, bs, dt = case["head_dim"], case["kv_heads"], case["block"], DTYPES[case["dtype"]]
    s = dict(case=case, err=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "store":
        T = case["tokens"]
        NB = -(-T // bs) + 3
        s["key"] = (rnd(T, Hkv, D) + rnd(Hkv, D)).to(dt)      # keys keep a mean per channel
        s["value"] = rnd(T, Hkv, D).to(dt)
        s["slots"] = torch.randperm(NB * bs, generator=g, device=dev)[:T]
        s["k"] = torch.zeros(NB, bs, Hkv, D // 2 + 4, dtype=torch.uint8, device=dev)
        s["v"] = torch.zeros_like(s["k"])
        s["key_out"], s["value_out"] = torch.empty_like(s["key"]), torch.empty_like(s["value"])
        return s
    lens = _lens(case)
    used = sum(-(-L // bs) for L in lens)
    new = sum(-(-min(L, case["budget"]) // bs) for L in lens) if case["op"] == "evict" else 0
    NB = used + new + 1
    order = torch.randperm(NB - 1, generator=g, device=dev).cpu()              # the last block is nobody's
    bt, first = _tables(lens, bs, order)
    s["tables"], s["lens"] = bt.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    cache = case.get("cache", "int4" if case["op"] == "attend" else case["dtype"])
    for name in ("k", "v"):
        x = rnd(NB, bs, Hkv, D)
        if name == "k":
            x += rnd(Hkv, D) * 0.5
        s[name] = _pack4(x, bs) if cache == "int4" else x.to(DTYPES[cache])
        del x
    if case["op"] != "attend":
        # what earlier steps added up: few tokens hold most of it, some nothing at all
        w = torch.exp(2 * rnd(NB, Hkv, bs)) * 0.1
        s["weights"] = torch.where(torch.rand(NB, Hkv, bs, generator=g, device=dev) < 0.05, 0.0, w)
    if case["op"] == "evict":
        s["new_tables"] = s["tables"]
        if not case["in_place"]:
            s["new_tables"] = _tables([min(L, case["budget"]) for L in lens], bs, order, first)[0].to(dev)
        s["stored"] = s["weights"].clone()
        s["new_lens"] = torch.empty_like(s["lens"])
        s["kept"] = torch.empty(len(lens), Hkv, case["budget"], dtype=torch.int32, device=dev)
        return s
    counts = _query_counts(case) if case["op"] == "attend" else [1] * len(lens)
    q = rnd(sum(counts), case["q_heads"], D)
    s["q"] = q.to(dt)
    s["out"] = torch.empty_like(s["q"])
    start = [0]
    for c in counts:
        start.append(start[-1] + c)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device=dev)
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"store": _store, "attend": _attend, "observe": _observe, "evict": _evict}[s["case"]["op"]](s)


def _run_own(s):
    import paged_kv_cache_69_gb300 as pa
    c = s["case"]
    if c["op"] == "store":
        pa.pa_reshape_and_cache(s["k"], s["v"], s["key"], s["value"], s["slots"], "int4", err_flag=s["err"])
        pa.pa_gather_cache(s["key_out"], s["value_out"], s["k"], s["v"], s["slots"], "int4", err_flag=s["err"])
        return {"key": s["key_out"], "value": s["value_out"]}
    bt, MB = s["tables"], s["tables"].shape[1]
    if c["op"] == "evict":
        s["weights"].copy_(s["stored"])
        if "ws" not in s:
            s["ws"] = torch.empty(pa.pa_evict_workspace_size(c["batch"], c["kv_heads"], MB * c["block"], c["budget"]),
                                  dtype=torch.uint8, device=bt.device)
        pa.pa_evict(s["k"], s["v"], s["weights"], bt, s["lens"], s["new_lens"], c["budget"], num_sink=c["sink"],
                    num_recent=c["recent"], new_block_tables=s["new_tables"], kept=s["kept"], workspace=s["ws"],
                    err_flag=s["err"])
        return {"k": s["k"], "v": s["v"], "weights": s["weights"], "lens": s["new_lens"], "kept": s["kept"]}
    if c["op"] == "attend" and c["queries"] > 1:
        if "ws" not in s:
            s["ws"] = torch.empty(pa.pa_attention_workspace_size(c["batch"], c["queries"], c["q_heads"],
                                                                 MB * c["block"], c["head_dim"], 0),
                                  dtype=torch.uint8, device=bt.device)
        pa.pa_attention(s["out"], s["q"], s["k"], s["v"], bt, s["lens"], s["q_start"], s["scale"], c["queries"],
                        "int4", workspace=s["ws"], err_flag=s["err"])
        return {"out": s["out"]}
    if c["op"] == "attend":
        if "ws" not in s:
            s["ws"] = pa.alloc_workspace(c["batch"], c["q_heads"], MB * c["block"], c["head_dim"], device=bt.device)
        pa.pa_decode(s["out"], s["q"], s["k"], s["v"], bt, s["lens"], s["scale"], "int4", workspace=s["ws"],
                     err_flag=s["err"])
        return {"out": s["out"]}
    if "ws" not in s:
        s["ws"] = torch.empty(pa.pa_decode_weights_workspace_size(c["batch"], c["q_heads"], MB * c["block"],
                                                                  c["head_dim"]), dtype=torch.uint8, device=bt.device)
    pa.pa_decode_weights(s["out"], s["weights"], s["q"], s["k"], s["v"], bt, s["lens"], s["scale"], c["cache"],
                         workspace=s["ws"], err_flag=s["err"])
    return {"out": s["out"], "weights": s["weights"]}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _to_half64(x):
    """x (float64) rounded once to a float16 value, kept in float64."""
    _, e = torch.frexp(x)
    unit = ((torch.clamp_min(e - 11, -24).long() + 1023) << 52).view(torch.float64)   # a power of two, exactly
    return torch.round(x / unit) * unit


def _quantise(x):
    """(codes, step, low) of the rows of x, in 64 bits: a code sits next to a border where 32 would move it."""
    x = x.double().clamp(-65504.0, 65504.0)
    low = _to_half64(x.amin(-1, keepdim=True))
    step = _to_half64((x.amax(-1, keepdim=True) - low) / 15).clamp_min(0.0)
    code = torch.where(step > 0, (x - low) / step, torch.zeros_like(x)).round().clamp(0, 15)
    return code, step, low


def _split4(pool):
    """(codes [num_blocks, kv_heads, block, head_dim / 2], (step, low) float16 [num_blocks, kv_heads, block, 2])."""
    NB, bs, Hkv, R = pool.shape
    flat, n = pool.view(NB, -1), Hkv * bs * (R - 4)
    return flat[:, :n].unflatten(1, (Hkv, bs, R - 4)), flat[:, n:].contiguous().view(torch.float16).view(NB, Hkv, bs, 2)


def _values4(codes, par):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return c * par[..., :1].float() + par[..., 1:].float()


def _store(s):
    out = {}
    for name, pool, x in (("key", s["k"], s["key"]), ("value", s["v"], s["value"])):
        NB, bs, Hkv, R = pool.shape
        code, step, low = _quantise(x)
        code = code.to(torch.uint8)
        blk, off = s["slots"] // bs, s["slots"] % bs
        n = Hkv * bs * (R - 4)
        flat = pool.view(NB, -1)
        codes, par = flat[:, :n].unflatten(1, (Hkv, bs, R - 4)), flat[:, n:].unflatten(1, (Hkv, bs, 4))
        codes[blk, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
        par[blk, :, off] = torch.cat([step, low], -1).half().view(torch.uint8)
        codes, par = _split4(pool)
        out[name] = _values4(codes[blk, :, off], par[blk, :, off]).to(x.dtype)
    return out


def _rows(s, name):
    """The rows of every sequence in float32, [batch, kv_heads, max tokens, head_dim]."""
    bt, pool = s["tables"].long().clamp_min(0), s[name]
    if s["case"].get("cache", "int4") == "int4":
        codes, par = _split4(pool)
        x = _values4(codes[bt], par[bt])
    else:
        x = pool[bt].transpose(2, 3).float()
    return x.transpose(1, 2).flatten(2, 3)


def _softmax_rows(s, q, last):
    """Softmax weights [batch, kv_heads, rows, max tokens] of the rows q [batch, kv_heads, rows, head_dim], a row
    attending the keys up to last [batch, 1, rows, 1]."""
    x = torch.matmul(q, _rows(s, "k").transpose(2, 3)) * s["scale"]
    pos = torch.arange(x.shape[-1], device=x.device)
    x = x.masked_fill(pos > last, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e30))
    return x / x.sum(-1, keepdim=True).clamp_min(1e-38)


def _attend(s):
    c = s["case"]
    B, Hkv, G, D, n = c["batch"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"], c["queries"]
    start = s["q_start"].long()
    count = start[1:] - start[:-1]
    j = torch.arange(n, device=start.device)
    row = torch.minimum(start[:-1, None] + j, start[1:, None] - 1)             # padded with each one's last token
    q = s["q"][row].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    last = s["lens"].long()[:, None] - count[:, None] + torch.minimum(j, count[:, None] - 1)
    p = _softmax_rows(s, q, last.repeat_interleave(G, 1).view(B, 1, n * G, 1))
    o = torch.matmul(p, _rows(s, "v")).view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B * n, Hkv * G, D)
    out = torch.empty_like(s["q"])
    out[row.flatten()] = o.to(out.dtype)
    return {"out": out}


def _observe(s):
    c = s["case"]
    B, Hkv, G, D, bs = c["batch"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"], c["block"]
    lens = s["lens"].long()
    p = _softmax_rows(s, s["q"].float().view(B, Hkv, G, D), (lens - 1).view(B, 1, 1, 1))
    out = torch.matmul(p, _rows(s, "v")).view(B, Hkv * G, D).to(s["q"].dtype)
    # every key gains its weight; the newest token's, just written, starts from it
    w = p.sum(2).view(B, Hkv, -1, bs).transpose(1, 2)
    pos = torch.arange(w.shape[1] * bs, device=w.device).view(-1, bs)
    at = torch.where(s["tables"] >= 0, s["tables"].long(), s["weights"].shape[0] - 1)   # nobody's block gains zeros
    newest = (pos[None] == lens.view(B, 1, 1) - 1)[:, :, None]
    old = s["weights"][at]
    s["weights"].index_put_((at,), torch.where(newest, w, old + w))
    return {"out": out, "weights": s["weights"]}


def _evict(s):
    c = s["case"]
    s["weights"].copy_(s["stored"])
    B, Hkv, bs, bud, rec, snk = c["batch"], c["kv_heads"], c["block"], c["budget"], c["recent"], c["sink"]
    bt = s["tables"].long().clamp_min(0)
    nbt = s["new_tables"].long().clamp_min(0)
    L = s["lens"].long().view(B, 1, 1)
    w = s["weights"][bt].transpose(1, 2).flatten(2, 3)                          # [batch, kv_heads, max tokens]
    pos = torch.arange(w.shape[2], device=w.device)
    heavy, over = bud - rec, L > bud
    cand = (pos >= snk) & (pos < L - rec)
    order = torch.argsort(torch.where(cand, w, -math.inf), dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(2, order, pos.expand_as(order))
    keep = (pos < snk) | (cand & (rank < heavy - snk))
    # the i-th free place below `heavy` takes the i-th kept row from behind it
    j = torch.arange(bud, device=w.device)
    fill = torch.argsort(torch.where(keep & (pos >= heavy), pos, pos + w.shape[2]), dim=-1)
    low = torch.zeros(B, Hkv, bud, dtype=torch.bool, device=w.device)
    n = min(heavy, w.shape[2])
    low[..., :n] = ~keep[..., :n]
    nth = (low.cumsum(-1) - 1).clamp(0, w.shape[2] - 1)
    src = torch.where(low, fill.gather(2, nth), j)
    src = torch.where(j >= heavy, L - bud + j, src)
    src = torch.where(over, src, j.expand_as(src))
    new = torch.clamp(L, max=bud)
    kept = torch.where(j < new, src, -1).to(torch.int32)
    # rows past the new length repeat the first one's move
    first = src[..., :1].expand_as(src)
    src, dst = torch.where(j < new, src, first), torch.where(j < new, j.expand_as(src), 0)
    b, h = torch.arange(B, device=w.device).view(B, 1, 1), torch.arange(Hkv, device=w.device).view(1, Hkv, 1)
    sb, so, db, do = bt[b, src // bs], src % bs, nbt[b, dst // bs], dst % bs
    for name in ("k", "v"):
        s[name][db, do, h] = s[name][sb, so, h]
    s["weights"][db, h, do] = s["weights"][sb, h, so]
    return {"k": s["k"], "v": s["v"], "weights": s["weights"], "lens": new.view(B).to(torch.int32), "kept": kept}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _row64(s, name, i, n):
    """The first n rows of sequence i in float64, [n, kv_heads, head_dim]."""
    c, pool = s["case"], s[name]
    pos = torch.arange(n, device=pool.device)
    blk, off = s["tables"][i].long()[pos // c["block"]], pos % c["block"]
    if c["op"] != "attend" and c.get("cache") != "int4":
        return pool[blk, off].double()
    NB, bs, Hkv, R = pool.shape
    by = pool.reshape(NB, bs * Hkv * R)[blk]
    out = torch.empty(n, Hkv, 2 * (R - 4), dtype=torch.float64, device=pool.device)
    for h in range(Hkv):
        at = (h * bs + off) * (R - 4)
        code = by.gather(1, at[:, None] + torch.arange(R - 4, device=by.device))
        at = Hkv * bs * (R - 4) + (h * bs + off) * 4
        par = by.gather(1, at[:, None] + torch.arange(4, device=by.device)).contiguous().view(torch.float16).double()
        out[:, h, 0::2] = par[:, 1:] + par[:, :1] * (code % 16).double()
        out[:, h, 1::2] = par[:, 1:] + par[:, :1] * torch.div(code, 16, rounding_mode="floor").double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "store":
        def back(x):
            x = x.double()
            low = _nearest_half(x.min(-1).values)
            step = _nearest_half((x.max(-1).values - low) / 15)
            t = (x - low[..., None]) / torch.where(step == 0, 1.0, step)[..., None]
            f = torch.floor(t)
            up = (t - f > 0.5) | ((t - f == 0.5) & (f % 2 == 1))              # ties to even
            code = torch.minimum(torch.maximum(f + up, torch.zeros_like(f)), torch.full_like(f, 15.0))
            code = torch.where((step == 0)[..., None], 0.0, code)
            return low[..., None] + step[..., None] * code
        return {"key": back(s["key"]), "value": back(s["value"])}
    lens = _lens(c)
    if c["op"] == "evict":
        return _exact_evict(s, lens)
    G = c["q_heads"] // c["kv_heads"]
    counts = _query_counts(c) if c["op"] == "attend" else [1] * len(lens)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    weights = s["weights"].double() if c["op"] == "observe" else None
    r = 0
    for i, (L, n) in enumerate(zip(lens, counts)):
        k, v = _row64(s, "k", i, L), _row64(s, "v", i, L)
        for h in range(c["kv_heads"]):
            q = s["q"][r:r + n, h * G:(h + 1) * G].double()
            x = torch.einsum("jgd,td->jgt", q, k[:, h]) * s["scale"]
            seen = torch.arange(L, device=x.device)[None, :] <= (L - n + torch.arange(n, device=x.device))[:, None]
            x = torch.where(seen[:, None, :], x, -math.inf)
            e = torch.exp(x - x.max(-1, keepdim=True).values.clamp(min=-1e300))
            p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
            out[r:r + n, h * G:(h + 1) * G] = torch.einsum("jgt,td->jgd", p, v[:, h])
            if weights is not None:
                pos = torch.arange(L, device=x.device)
                blk, off = s["tables"][i].long()[pos // c["block"]], pos % c["block"]
                gain = p[0].sum(0)
                weights[blk[:-1], h, off[:-1]] += gain[:-1]
                weights[blk[-1], h, off[-1]] = gain[-1]
        r += n
    return {"out": out} if weights is None else {"out": out, "weights": weights}


def _nearest_half(x):
    """The float16 value nearest to x (float64), ties to the even one, by trying the neighbours of a first guess."""
    guess = x.float().half()
    bits = guess.view(torch.int16).int()
    ordinal = torch.where(bits < 0, -(bits & 0x7FFF), bits)
    best, err, even = guess.double(), (guess.double() - x).abs(), bits % 2 == 0
    for d in (-1, 1):
        o = (ordinal + d).clamp(-0x7BFF, 0x7BFF)
        b = torch.where(o < 0, (-o) | 0x8000, o)
        v = torch.where(b >= 0x8000, b - 0x10000, b).to(torch.int16).view(torch.float16).double()
        e = (v - x).abs()
        better = (e < err) | ((e == err) & ~even & (b % 2 == 0))
        best, even, err = torch.where(better, v, best), torch.where(better, b % 2 == 0, even), torch.minimum(err, e)
    return best


def _exact_evict(s, lens):
    c = s["case"]
    bs, bud, rec, snk = c["block"], c["budget"], c["recent"], c["sink"]
    dev = s["k"].device
    k, v, w = s["k"].double(), s["v"].double(), s["weights"].double()
    new = torch.empty(len(lens), dtype=torch.int32, device=dev)
    kept = torch.full((len(lens), c["kv_heads"], bud), -1, dtype=torch.int32, device=dev)
    for i, L in enumerate(lens):
        n = min(L, bud)
        new[i] = n
        bt, nbt = s["tables"][i].long(), s["new_tables"][i].long()
        pos = torch.arange(L, device=dev)
        for h in range(c["kv_heads"]):
            src = torch.arange(n, device=dev)
            if L > bud:
                score = s["weights"][bt[pos // bs], h, pos % bs][snk:L - rec].double()
                best = torch.sort(score, descending=True, stable=True).indices[:bud - rec - snk] + snk
                chosen = torch.zeros(L, dtype=torch.bool, device=dev)
                chosen[:snk] = True
                chosen[best] = True
                front = chosen[:bud - rec]
                src[:bud - rec][~front] = torch.nonzero(chosen[bud - rec:L - rec]).flatten() + bud - rec
                src[bud - rec:] = torch.arange(L - rec, L, device=dev)
            kept[i, h, :n] = src.to(torch.int32)
            d = torch.arange(n, device=dev)
            sb, so, db, do = bt[src // bs], src % bs, nbt[d // bs], d % bs
            k[db, do, h] = s["k"][sb, so, h].double()
            v[db, do, h] = s["v"][sb, so, h].double()
            w[db, h, do] = s["weights"][sb, h, so].double()
    return {"k": k, "v": v, "weights": w, "lens": new, "kept": kept}
