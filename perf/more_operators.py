"""Cases of rotated cache writes, prompt attention and shared-prefix decode, with their plain forms.

Four calls, each with what a serving program holds when it makes them:

  rope     rotate the queries and keys of new tokens by their positions and write K/V into the pool
           (pa_rope_and_cache); one axis of positions, or several (time, height, width)
  prefill  causal attention of whole prompts packed one behind the other, K/V as the projection left them (pa_prefill)
  cached   the same with K/V in the paged pool, where a sequence's earlier tokens are already (pa_prefill_cached):
           a chunk of a prompt, or a prompt whose first blocks were found in the prefix cache
  shared   one decode token per sequence; the sequences of a group share the blocks of a prefix, which is attended
           once for all of them (pa_decode_shared)

Layouts: pools [num_blocks, block_size, num_kv_heads, head_dim]; q and out [tokens, num_q_heads, head_dim]; key and
value [tokens, num_kv_heads, head_dim]; cos_sin float32 [positions, rotated dims]: cosines, then sines, of half of them.
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
        dict(name="rope_step_f16", op="rope", tokens=64, prompt=False, q_heads=28, kv_heads=4, head_dim=128, rot=128,
             axes=1, interleaved=False, block=16, dtype="f16"),
        # long prompts of a 32/8-head layer
        dict(name="rope_prompt_bf16", op="rope", tokens=65536, prompt=True, q_heads=32, kv_heads=8, head_dim=128,
             rot=128, axes=1, interleaved=False, block=32, dtype="bf16"),
        # an odd count of image tokens, three axes, half of a narrow head rotated, float32
        dict(name="rope_image_f32_d64", op="rope", tokens=5003, prompt=True, q_heads=4, kv_heads=2, head_dim=64,
             rot=48, axes=3, interleaved=True, block=8, dtype="f32"),
        # four short prompts on a small model: latency
        dict(name="prefill_tiny_f16", op="prefill", batch=4, lo=5, hi=40, q_heads=4, kv_heads=2, head_dim=64,
             dtype="f16"),
        # prompts of 100 to 8192 tokens on a 7B-like layer
        dict(name="prefill_7b_f16", op="prefill", batch=16, lo=100, hi=8192, q_heads=28, kv_heads=4, head_dim=128,
             dtype="f16"),
        # a serving mix of many short prompts
        dict(name="prefill_mix_bf16", op="prefill", batch=256, lo=20, hi=2048, q_heads=32, kv_heads=8, head_dim=128,
             dtype="bf16"),
        # one long document
        dict(name="prefill_long_bf16", op="prefill", batch=1, lo=32768, hi=32768, q_heads=32, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # what is left of eight prompts behind their cached first blocks, 7B-like layer
        dict(name="cached_7b_f16", op="cached", batch=8, lo=100, hi=8192, queries=512, q_heads=28, kv_heads=4,
             head_dim=128, block=16, dtype="f16"),
        # the last chunks of two long prompts
        dict(name="cached_long_bf16", op="cached", batch=2, lo=32768, hi=65536, queries=2048, q_heads=32, kv_heads=8,
             head_dim=128, block=32, dtype="bf16"),
        # two samples of a short prompt on a small model: latency
        dict(name="shared_tiny_f16", op="shared", groups=2, members=3, prefix=48, ragged=False, own_lo=1, own_hi=20,
             q_heads=4, kv_heads=2, head_dim=64, block=16, dtype="f16"),
        # parallel sampling: 32 prompts of 2048 tokens, four branches each, 7B-like layer
        dict(name="shared_branches_f16", op="shared", groups=32, members=4, prefix=2048, ragged=False, own_lo=1,
             own_hi=256, q_heads=28, kv_heads=4, head_dim=128, block=16, dtype="f16"),
        # 128 conversations about one long document
        dict(name="shared_document_bf16", op="shared", groups=1, members=128, prefix=32768, ragged=False, own_lo=20,
             own_hi=2048, q_heads=32, kv_heads=8, head_dim=128, block=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefill", "cached", "shared"])
    head_dim = rng.choice([64, 128, 128])
    block = rng.choice([8, 16, 32, 64])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    dtype = rng.choice(["f16", "bf16"])
    base = dict(op=op, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype)
    if op == "rope":
        return dict(base, tokens=_log_int(rng, 1, 65536 * 16 // max(32, q_heads)), prompt=rng.random() < 0.5,
                    rot=rng.choice([head_dim, head_dim, head_dim // 2, head_dim - 16]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.5, block=block, dtype=rng.choice(["f16", "bf16", "f32"]))
    # no more arithmetic than the longest listed prompt has, nor more tokens times heads than the widest listed batch
    most = 2.0 * 32768 ** 2 * 32 * 128 / (4.0 * q_heads * head_dim)             # (query token, key) pairs
    if op == "prefill":
        hi = _log_int(rng, 1, min(32768, int(math.sqrt(2 * most))))
        lo = max(1, int(hi * rng.uniform(0.02, 1.0)))
        most_batch = int(max(1, min(256, 1500000 // (hi * q_heads), most / (hi * hi / 2))))
        return dict(base, batch=_log_int(rng, 1, most_batch), lo=lo, hi=hi)
    if op == "cached":
        hi = _log_int(rng, 2, 65536)
        lo = max(1, int(hi * rng.uniform(0.02, 1.0)))
        queries = _log_int(rng, 1, min(hi, 4096, int(most / hi)))
        most_batch = int(max(1, min(256, 1048576 // (hi * kv_heads), most / (hi * queries))))
        return dict(base, batch=_log_int(rng, 1, most_batch), lo=lo, hi=hi, queries=queries, block=block)
    prefix = _log_int(rng, 1, 65536)
    groups = _log_int(rng, 1, max(1, min(64, 1048576 // (prefix * kv_heads))))
    own_hi = _log_int(rng, 1, 4096)
    members = _log_int(rng, 1, max(1, min(256 // groups, 2097152 // (groups * own_hi * kv_heads))))
    return dict(base, groups=groups, members=members, prefix=prefix, ragged=rng.random() < 0.7, block=block,
                own_lo=max(1, int(own_hi * rng.uniform(0.01, 1.0))), own_hi=own_hi)


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


def _query_counts(case, lens):
    """Query tokens per sequence: all of them, or the last 1 to `queries`."""
    if case["op"] == "prefill":
        return lens
    r = random.Random(case["batch"] * 7919 + case["queries"])
    return [min(L, r.randint(1, case["queries"]) if i else case["queries"]) for i, L in enumerate(lens)]


def _groups(case):
    """(members of each group, prefix of each group, own tokens of each sequence); prefixes in whole blocks. Of a
    ragged case's groups the first is the largest."""
    r = random.Random(case["groups"] * 104729 + case["members"] * 31 + case["prefix"])
    m, bs, size = case["members"], case["block"], [(case["members"], case["prefix"])] * case["groups"]
    if case["ragged"]:
        size[1:] = [(r.randint(max(1, m // 2), m), r.randint(case["prefix"] // 2, case["prefix"])) for _ in size[1:]]
    n, prefix = [a for a, _ in size], [b // bs * bs for _, b in size]
    own_lens = [r.randint(case["own_lo"], case["own_hi"]) for _ in range(sum(n))]
    return n, prefix, own_lens


def work(case):
    D, Hq, Hkv, e = case["head_dim"], case["q_heads"], case["kv_heads"], WIDTH[case["dtype"]]
    if case["op"] == "rope":
        T = case["tokens"]
        # queries, keys and values in and out, a row of the table, positions and a slot
        return {"bytes": T * (2 * e * (Hq + 2 * Hkv) * D + 4 * case["rot"] + 8 * case["axes"] + 8.0),
                "flops": T * 3.0 * (Hq + Hkv) * case["rot"]}
    if case["op"] == "shared":
        n, prefix, own_lens = _groups(case)
        rows = float(sum(prefix) + sum(own_lens))
        pairs = float(sum(a * b for a, b in zip(n, prefix)) + sum(own_lens))
        return {"bytes": 2 * rows * Hkv * D * e + 2.0 * sum(n) * Hq * D * e, "flops": 4.0 * pairs * Hq * D}
    lens = _lens(case)
    counts = _query_counts(case, lens)
    pairs = float(sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, counts)))
    return {"bytes": 2.0 * sum(lens) * Hkv * D * e + 2.0 * sum(counts) * Hq * D * e, "flops": 4.0 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# what a program holds before the call
# ---------------------------------------------------------------------------
def _sections(case):
    """Rotated pairs of each axis: equal shares, the first axis takes what is left over."""
    half, a = case["rot"] // 2, case["axes"]
    return [half - (a - 1) * (half // a)] + [half // a] * (a - 1)


def _table(positions, rot, device):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    D, Hq, Hkv, dt = case["head_dim"], case["q_heads"], case["kv_heads"], DTYPES[case["dtype"]]
    s = dict(case=case, err=torch.zeros(1, dtype=torch.int32, device=dev), scale=1.0 / math.sqrt(D))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    def starts(counts):
        t = [0]
        for c in counts:
            t.append(t[-1] + c)
        return ints(t)

    def pool(NB, bs):
        return (rnd(NB, bs, Hkv, D) + rnd(Hkv, D) * 0.5).to(dt), rnd(NB, bs, Hkv, D).to(dt)

    if case["op"] == "rope":
        T, bs = case["tokens"], case["block"]
        NB = -(-T // bs) + 3
        s["table"] = _table(65536, case["rot"], dev)
        if case["prompt"]:
            t = torch.arange(T, device=dev) % 16384
            grid = [t // 1024, t % 1024 // 32, t % 32]                    # pictures of 32 x 32 tokens
        else:
            grid = [torch.randint(0, 65536, (T,), generator=g, device=dev) for _ in range(3)]
            t = grid[0]
        s["positions"] = t if case["axes"] == 1 else torch.stack(grid[:case["axes"]])
        s["sections"] = None if case["axes"] == 1 else _sections(case)
        s["q"], s["key"] = rnd(T, Hq, D).to(dt), (rnd(T, Hkv, D) + rnd(Hkv, D)).to(dt)   # keys keep a mean per channel
        s["value"] = rnd(T, Hkv, D).to(dt)
        blocks = torch.randperm(NB, generator=g, device=dev)
        at = torch.arange(T, device=dev)
        s["slots"] = blocks[at // bs] * bs + at % bs
        s["k"] = torch.zeros(NB, bs, Hkv, D, dtype=dt, device=dev)
        s["v"], s["q_out"] = torch.zeros_like(s["k"]), torch.empty_like(s["q"])
        return s
    if case["op"] == "shared":
        n, prefix, own_lens = _groups(case)
        bs = case["block"]
        used = sum(p // bs for p in prefix) + sum(-(-x // bs) for x in own_lens)
        order = torch.randperm(used + 1, generator=g, device=dev).cpu().tolist()
        rows, lens, at, j = [], [], 0, 0
        for m, p in zip(n, prefix):
            common = order[at:at + p // bs]
            at += p // bs
            for _ in range(m):
                k = -(-own_lens[j] // bs)
                rows.append(common + order[at:at + k])
                lens.append(p + own_lens[j])
                at += k
                j += 1
        MB = max(len(r) for r in rows)
        s["tables"] = ints([r + [-1] * (MB - len(r)) for r in rows])
        s["lens"], s["group_start"], s["prefix_lens"] = ints(lens), starts(n), ints(prefix)
        s["k"], s["v"] = pool(used + 1, bs)
        s["q"] = rnd(len(lens), Hq, D).to(dt)
        s["out"] = torch.empty_like(s["q"])
        return s
    lens = _lens(case)
    counts = _query_counts(case, lens)
    s["q_start"] = starts(counts)
    s["q"] = rnd(sum(counts), Hq, D).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if case["op"] == "prefill":
        s["key"], s["value"] = (rnd(sum(lens), Hkv, D) + rnd(Hkv, D) * 0.5).to(dt), rnd(sum(lens), Hkv, D).to(dt)
        return s
    bs = case["block"]
    need = [-(-L // bs) for L in lens]
    order = torch.randperm(sum(need) + 1, generator=g, device=dev).to(torch.int32)
    s["tables"] = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, k in enumerate(need):
        s["tables"][i, :k] = order[at:at + k]
        at += k
    s["lens"] = ints(lens)
    s["k"], s["v"] = pool(sum(need) + 1, bs)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope, "prefill": _prompt, "cached": _prompt, "shared": _shared}[s["case"]["op"]](s)


def _run_own(s):
    import paged_kv_cache_69_gb300 as pa
    c = s["case"]
    if c["op"] == "rope":
        pa.pa_rope_and_cache(s["k"], s["v"], s["q_out"], s["q"], s["key"], s["value"], s["positions"], s["table"],
                             s["slots"], sections=s["sections"], interleaved=c["interleaved"], err_flag=s["err"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "shared":
        MB = s["tables"].shape[1]
        if "ws" not in s:
            s["ws"] = torch.empty(pa.pa_decode_shared_workspace_size(s["lens"].numel(), s["prefix_lens"].numel(), Hq,
                                                                     Hkv, MB * c["block"], D),
                                  dtype=torch.uint8, device=s["q"].device)
        pa.pa_decode_shared(s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["group_start"],
                            s["prefix_lens"], s["scale"], workspace=s["ws"], err_flag=s["err"])
        return {"out": s["out"]}
    if "ws" not in s:
        s["ws"] = torch.empty(pa.pa_prefill_workspace_size(c["batch"], s["q"].shape[0], Hq, Hkv, D), dtype=torch.uint8,
                              device=s["q"].device)
    if c["op"] == "prefill":
        pa.pa_prefill(s["out"], s["q"], s["key"], s["value"], s["q_start"], s["scale"], workspace=s["ws"],
                      err_flag=s["err"])
    else:
        pa.pa_prefill_cached(s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["q_start"], s["scale"],
                             workspace=s["ws"], err_flag=s["err"])
    return {"out": s["out"]}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _angles(s):
    """(cos, sin) float32 [tokens, 1, pairs]: pair i by the position on its axis."""
    half = s["case"]["rot"] // 2
    if s["sections"] is None:
        row = s["table"][s["positions"]]
    else:
        axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=s["table"].device),
                                       torch.tensor(s["sections"], device=s["table"].device))
        at = s["positions"][axis].t()                                      # [tokens, pairs]
        pair = torch.arange(half, device=at.device)
        row = torch.cat([s["table"][at, pair], s["table"][at, half + pair]], 1)
    return row[:, None, :half], row[:, None, half:]


def _rope(s):
    c = s["case"]
    rot = c["rot"]
    cos, sin = _angles(s)

    def turn(x):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([z, y[..., rot:]], -1).to(x.dtype)

    s["q_out"].copy_(turn(s["q"]))
    row = s["k"].shape[2:]
    s["k"].view(-1, *row)[s["slots"]] = turn(s["key"])
    s["v"].view(-1, *row)[s["slots"]] = s["value"]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _prompt(s):
    c = s["case"]
    Hkv, D = c["kv_heads"], c["head_dim"]
    G = c["q_heads"] // Hkv
    lens = _lens(c)
    at, first = 0, 0
    for i, (L, n) in enumerate(zip(lens, _query_counts(c, lens))):
        if c["op"] == "prefill":
            k, v = s["key"][first:first + L], s["value"][first:first + L]
        else:
            blocks = s["tables"][i, :-(-L // c["block"])].long()
            k, v = (x[blocks].flatten(0, 1)[:L] for x in (s["k"], s["v"]))
        k, v = k.float().transpose(0, 1), v.float().transpose(0, 1)         # [kv_heads, L, head_dim]
        pos = torch.arange(L, device=k.device)
        step = max(1, (1 << 29) // (L * c["q_heads"]))                      # query tokens of 2 GB of scores
        for a in range(0, n, step):
            m = min(step, n - a)
            end = L - n + a + m                                             # keys that any of these tokens attends
            q = s["q"][at + a:at + a + m].float().view(m, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            x = torch.matmul(q, k[:, :end].transpose(1, 2)) * s["scale"]
            last = (torch.arange(m, device=x.device) + L - n + a).repeat_interleave(G)
            x.masked_fill_(pos[:end] > last[:, None], -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(x, v[:, :end]) / x.sum(-1, keepdim=True)
            o = o.view(Hkv, m, G, D).permute(1, 0, 2, 3).reshape(m, Hkv * G, D)
            s["out"][at + a:at + a + m] = o.to(s["out"].dtype)
        at += n
        first += L
    return {"out": s["out"]}


def _shared(s):
    c = s["case"]
    Hkv, D, bs = c["kv_heads"], c["head_dim"], c["block"]
    G = c["q_heads"] // Hkv
    n, prefix, own_lens = _groups(c)
    at = 0
    for m, P in zip(n, prefix):
        lens = own_lens[at:at + m]
        common = s["tables"][at, :P // bs].long()
        tail = s["tables"][at:at + m, P // bs:P // bs + -(-max(lens) // bs)].long().clamp_min(0)
        q = s["q"][at:at + m].float().view(m, Hkv, G, D)
        k, v = (x[common].flatten(0, 1).float().transpose(0, 1) for x in (s["k"], s["v"]))      # [kv_heads, P, D]
        kt, vt = (x[tail].flatten(1, 2).float().transpose(1, 2) for x in (s["k"], s["v"]))      # [m, kv_heads, own, D]
        x = torch.matmul(q.transpose(0, 1).reshape(Hkv, m * G, D), k.transpose(1, 2)).view(Hkv, m, G, P).transpose(0, 1)
        y = torch.matmul(q, kt.transpose(2, 3))
        seen = torch.arange(y.shape[-1], device=y.device) < torch.tensor(lens, device=y.device)[:, None]
        z = torch.cat([x, y.masked_fill(~seen[:, None, None], -math.inf)], -1) * s["scale"]
        z = torch.exp(z - z.amax(-1, keepdim=True))
        o = torch.matmul(z[..., :P].transpose(0, 1).reshape(Hkv, m * G, P), v).view(Hkv, m, G, D).transpose(0, 1)
        o = (o + torch.matmul(z[..., P:], vt)) / z.sum(-1, keepdim=True)
        s["out"][at:at + m] = o.reshape(m, Hkv * G, D).to(s["out"].dtype)
        at += m
    return {"out": s["out"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _exact_rope(s)
    G = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    row = 0
    if c["op"] == "shared":
        lens, counts = s["lens"].tolist(), [1] * s["lens"].numel()
    else:
        lens = _lens(c)
        counts = _query_counts(c, lens)
    first = 0
    for i, (L, n) in enumerate(zip(lens, counts)):
        pos = torch.arange(L, device=out.device)
        if c["op"] == "prefill":
            k, v = s["key"][first:first + L].double(), s["value"][first:first + L].double()
        else:
            blk, off = s["tables"][i].long()[pos // c["block"]], pos % c["block"]
            k, v = s["k"][blk, off].double(), s["v"][blk, off].double()
        for h in range(c["kv_heads"]):
            for a in range(0, n, 1024):
                b = min(n, a + 1024)
                end = L - n + b
                q = s["q"][row + a:row + b, h * G:(h + 1) * G].double()
                x = torch.einsum("jgd,td->jgt", q, k[:end, h]) * s["scale"]
                ahead = pos[None, :end] > torch.arange(L - n + a, L - n + b, device=out.device)[:, None]
                x = torch.where(ahead[:, None, :], -math.inf, x)
                p = torch.exp(x - x.max(-1, keepdim=True).values)
                out[row + a:row + b, h * G:(h + 1) * G] = (torch.einsum("jgt,td->jgd", p, v[:end, h]) /
                                                           p.sum(-1, keepdim=True))
        row += n
        first += L
    return {"out": out}


def _exact_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    pos = s["positions"].view(c["axes"], -1)
    table = s["table"].double()
    axis = [0] * half if s["sections"] is None else [a for a, m in enumerate(s["sections"]) for _ in range(m)]

    def turn(x):
        y = x.double().clone()
        for i in range(half):
            i0, i1 = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            co, si = (table[pos[axis[i]], j][:, None] for j in (i, half + i))
            u, w = x[..., i0].double(), x[..., i1].double()
            y[..., i0] = u * co - w * si
            y[..., i1] = u * si + w * co
        return y

    k, v = s["k"].double(), s["v"].double()
    blk, off = s["slots"] // c["block"], s["slots"] % c["block"]
    k[blk, off] = turn(s["key"])
    v[blk, off] = s["value"].double()
    return {"q": turn(s["q"]), "k": k, "v": v}
