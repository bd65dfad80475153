"""What the cache's newer operators are measured on: attention behind a sliding window, rotary positions with the
append, and copying, forking and compacting blocks.

Every case is a dict of plain values.  `prepare` makes what a serving program holds before the call (inputs, the
pool, block tables, the pass's plan); `run` is one call, either the library's (`own`) or its plain form in elementary
torch operations; `exact` is the operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per block
F16, E4M3 = 0, 1


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    window = dict(op="window", kv_dtype=F16, append=False, lens=1)
    rope = dict(op="rope", layout="half", base=10000.0, scaling="none", factor=1.0, original=8192, packed=False)
    return [
        # one user's decode step with the append fused into it: latency alone
        dict(window, name="window_one", q_heads=12, kv_heads=2, head_dim=128, decode=1, ctx_lo=700, ctx_hi=700, chunks="",
             window=256, sinks=4, append=True),
        # a full decode batch, contexts from a few tokens to 8k, the pages behind the window given back
        dict(window, name="window_decode", q_heads=12, kv_heads=2, head_dim=128, decode=256, ctx_lo=1, ctx_hi=8192,
             chunks="", window=1024, sinks=4),
        # long conversations on the 8-bit cache with wide heads
        dict(window, name="window_decode_8bit", q_heads=16, kv_heads=4, head_dim=256, decode=48, ctx_lo=2000,
             ctx_hi=60000, chunks="", window=4096, sinks=64, kv_dtype=E4M3),
        # a mixed pass: decode rows and two prompt chunks, one of them far into its prompt
        dict(window, name="window_chunks", q_heads=12, kv_heads=2, head_dim=128, decode=83, ctx_lo=64, ctx_hi=1100,
             chunks="2048:0,1024:5000", window=1024, sinks=4),
        # one token of one row: latency alone
        dict(rope, name="rope_one", q_heads=12, kv_heads=2, head_dim=128, rot_dim=128, tokens=1, reach=4000),
        # a pass of prompt chunks out of one packed projection, half of each head rotated, scaled for long contexts
        dict(rope, name="rope_chunks", q_heads=12, kv_heads=2, head_dim=128, rot_dim=64, tokens=8192, reach=200000,
             layout="interleaved", base=500000.0, scaling="bands", factor=8.0, packed=True),
        # copy on write of a few blocks
        dict(op="copy", name="copy_few", layers=28, kv_heads=2, head_dim=128, blocks=64, pairs=3, kv_dtype=F16),
        # a batch of requests' blocks duplicated at once
        dict(op="copy", name="copy_many", layers=16, kv_heads=4, head_dim=256, blocks=2500, pairs=1024, kv_dtype=F16),
        # one prompt, four samples
        dict(op="fork", name="fork_one", layers=28, kv_heads=2, head_dim=128, parents=1, children=4, ctx_lo=777,
             ctx_hi=777, kv_dtype=F16, lens=2),
        # a beam step of a batch on the 8-bit cache
        dict(op="fork", name="fork_many", layers=28, kv_heads=2, head_dim=128, parents=96, children=3, ctx_lo=16,
             ctx_hi=1500, kv_dtype=E4M3, lens=3),
        # a small pool, nearly empty
        dict(op="compact", name="compact_small", layers=28, kv_heads=2, head_dim=128, blocks=200, rows=3, ctx_lo=50,
             ctx_hi=400, shared=0, kv_dtype=F16, lens=4),
        # a large pool after many requests have left, rows with a common prefix
        dict(op="compact", name="compact_large", layers=28, kv_heads=2, head_dim=128, blocks=5000, rows=64, ctx_lo=100,
             ctx_hi=1000, shared=16, kv_dtype=F16, lens=5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["window", "window", "rope", "copy", "fork", "compact"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 6, 8])
    layers = rng.choice([1, 2, 5, 16, 28])
    lens = rng.randrange(1 << 20)
    if op == "window":
        case = dict(op=op, q_heads=hq, kv_heads=hkv, head_dim=d, window=_log(rng, 1, 4096), sinks=rng.choice([0, 0, 1, 4, 16, 100]),
                    kv_dtype=rng.choice([F16, F16, E4M3]), decode=0, ctx_lo=1, ctx_hi=1, chunks="", append=False, lens=lens)
        if rng.random() < 0.6:
            case.update(decode=_log(rng, 1, 256), ctx_hi=_log(rng, 1, 20000), append=case["kv_dtype"] == F16 and rng.random() < 0.5)
        else:
            case.update(decode=_log(rng, 1, 40), ctx_hi=_log(rng, 1, 2000),
                        chunks=",".join("%d:%d" % (_log(rng, 2, 1500), rng.choice([0, _log(rng, 1, 4000)])) for _ in range(rng.randint(1, 3))))
        while case["decode"] > 1 and work(case)["bytes"] > 4e8:
            case["decode"] //= 2
        while case["window"] > 16 and (work(case)["flops"] > 1.6e10 or _gathered(case) > 1e9):
            case["window"] //= 2
        return case
    if op == "rope":
        tokens = _log(rng, 1, 8192)
        while tokens > 1 and tokens * (hq + 2 * hkv) * d > 8192 * 16 * 128:
            tokens //= 2
        return dict(op=op, q_heads=hq, kv_heads=hkv, head_dim=d, rot_dim=rng.choice([d, d, d // 2, d // 4]), tokens=tokens,
                    reach=_log(rng, 10, 1000000), layout=rng.choice(["half", "interleaved"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "linear", "bands", "ramp"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]), original=rng.choice([2048, 4096, 8192]), packed=rng.random() < 0.5)
    kv_dtype = rng.choice([F16, E4M3])
    block = layers * 2 * hkv * BS * d * 2  # bytes of a block in fp16
    if op == "copy":
        pairs = _log(rng, 1, min(1024, max(1, (1 << 30) // block)))
        return dict(op=op, layers=layers, kv_heads=hkv, head_dim=d, blocks=2 * pairs + rng.randint(1, 200), pairs=pairs, kv_dtype=kv_dtype)
    if op == "fork":
        parents, children = _log(rng, 1, 96), rng.randint(1, 4)
        ctx_hi = _log(rng, 1, 1500)
        while parents > 1 and parents * (ctx_hi / BS + children + 1) * block > 2 << 30:
            parents //= 2
        return dict(op=op, layers=layers, kv_heads=hkv, head_dim=d, parents=parents, children=children, ctx_lo=1, ctx_hi=ctx_hi,
                    kv_dtype=kv_dtype, lens=lens)
    rows = _log(rng, 1, 200)
    ctx_hi = _log(rng, 16, 2000)
    while rows > 1 and rows * (ctx_hi / BS) * block > 1 << 30:
        rows //= 2
    case = dict(op=op, layers=layers, kv_heads=hkv, head_dim=d, blocks=0, rows=rows, ctx_lo=1, ctx_hi=ctx_hi,
                shared=rng.choice([0, 0, 1, 10]), kv_dtype=kv_dtype, lens=lens)
    case["blocks"] = math.ceil(_live_blocks(case) * rng.uniform(1.0, 3.0)) + rng.randint(0, 9)
    return case


def _row_lens(case, count):
    rng = random.Random(case["lens"])
    return [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(count)]


def _window_rows(case):
    """(new tokens, context with them) of every row."""
    rows = [(1, c) for c in _row_lens(case, case["decode"])]
    for c in case["chunks"].split(","):
        if c:
            new, cached = (int(x) for x in c.split(":"))
            rows.append((new, new + cached))
    random.Random(case["lens"]).shuffle(rows)
    return rows


def _gathered(case):
    """Values that the plain form reads of K: every token's keys, as many as the one that sees most."""
    tokens = sum(new for new, _ in _window_rows(case))
    return tokens * (case["window"] + case["sinks"]) * case["kv_heads"] * case["head_dim"]


def _live_blocks(case):
    shared = case["shared"]
    return shared + sum(max(1, -(-c // BS)) for c in _row_lens(case, case["rows"]))


def _token_bytes(case):
    """Bytes of one cached token of one layer, K and V."""
    return 2 * case["kv_heads"] * (case["head_dim"] + 1 if case["kv_dtype"] == E4M3 else 2 * case["head_dim"])


def work(case):
    if case["op"] == "window":
        w, s, d = case["window"], case["sinks"], case["head_dim"]
        keys = pairs = tokens = 0
        for new, ctx in _window_rows(case):
            lo = max(0, ctx - new - w + 1)
            keys += ctx - lo + min(s, lo)
            tokens += new
            for p in range(ctx - new, ctx):
                first = max(0, p - w + 1)
                pairs += p + 1 - first + min(s, first)
        io = tokens * case["q_heads"] * d * 4 + 4 * keys / BS
        if case["append"]:
            io += tokens * case["kv_heads"] * d * 4 + tokens * 8
        return {"bytes": keys * _token_bytes(case) + io, "flops": 4 * pairs * case["q_heads"] * d}
    if case["op"] == "rope":
        t, d = case["tokens"], case["head_dim"]
        return {"bytes": t * (4 * case["q_heads"] * d + 8 * case["kv_heads"] * d + 12),
                "flops": 3 * t * (case["q_heads"] + case["kv_heads"]) * case["rot_dim"]}
    token = case["layers"] * _token_bytes(case)
    if case["op"] == "copy":
        return {"bytes": case["pairs"] * (2 * BS * token + 8), "flops": 0}
    if case["op"] == "fork":
        ctx = _row_lens(case, case["parents"])
        return {"bytes": case["children"] * sum((c % BS) * 2 * token + 8 * -(-c // BS) for c in ctx), "flops": 0}
    n, entries = _live_blocks(case), case["rows"] * case["shared"] + _live_blocks(case)
    return {"bytes": n * (1 - n / case["blocks"]) * 2 * BS * token + 8 * entries + 4 * case["blocks"], "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float16)


def _cache(case, g, blocks, layers=1):
    """The cache's memory, filled: every block holds some request's values.  Returns the state's entries."""
    hkv, d = case["kv_heads"], case["head_dim"]
    values = _normal(g, layers, 2, blocks, hkv, BS, d)
    state = {}
    if case.get("kv_dtype", F16) == E4M3:
        top = values.abs().amax(-1).float()
        m, e = torch.frexp(top / 448)  # the smallest power of two that covers top / 448
        e = torch.where(m == 0.5, e - 1, e)
        codes = torch.ldexp(values.float(), -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales = (e + 127).to(torch.uint8).permute(0, 2, 3, 1, 4).contiguous()  # [layer][block][head][K, V][slot]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pool = pkv.Pool(layers, case.get("q_heads", hkv), hkv, d, blocks, kv_dtype=case.get("kv_dtype", F16))
        state["pool"] = pool
        if case.get("kv_dtype", F16) == E4M3:
            state["cache"], state["scales"] = pool.cache_view().copy_(codes), pool.scales_view().copy_(scales)
        else:
            state["cache"] = pool.cache_view().copy_(values)
    elif case.get("kv_dtype", F16) == E4M3:
        state["cache"], state["scales"] = codes, scales
    else:
        state["cache"] = values
    return state


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def prepare(case, seed):
    g, rng = _rng(seed), random.Random(seed)
    return {"window": _prepare_window, "rope": _prepare_rope, "copy": _prepare_copy, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, g, rng)


def _prepare_window(case, g, rng):
    rows = _window_rows(case)
    w, s = case["window"], case["sinks"]
    width = max(-(-ctx // BS) for _, ctx in rows)
    held = []  # the blocks of each row that some new token sees: the others have been given back
    for new, ctx in rows:
        lo = max(0, ctx - new - w + 1)
        held.append([j for j in range(-(-ctx // BS)) if j * BS < s or j * BS + BS > lo])
    need = sum(map(len, held))
    blocks = need + need // 8 + 2
    ids = rng.sample(range(blocks), need)
    tables = [[-1] * width for _ in rows]
    for row, js in zip(tables, held):
        for j in js:
            row[j] = ids.pop()
    state = {"case": case, **_cache(case, g, blocks)}
    starts = [0]
    for new, _ in rows:
        starts.append(starts[-1] + new)
    tokens = starts[-1]
    pos = [p for new, ctx in rows for p in range(ctx - new, ctx)]
    row_of = [b for b, (new, _) in enumerate(rows) for _ in range(new)]
    hkv, d = case["kv_heads"], case["head_dim"]
    state.update(tables=_ints(tables), ctx=_ints([c for _, c in rows]), starts=_ints(starts), tokens=tokens, rows=len(rows),
                 width=width, pos=_ints(pos, torch.int64), row_of=_ints(row_of, torch.int64), q=_normal(g, tokens, case["q_heads"], d),
                 seen=max(min(p + 1, w + min(s, max(0, p + 1 - w))) for p in pos),
                 slots=_ints([tables[b][p // BS] * BS + p % BS for b, p in zip(row_of, pos)], torch.int64))
    if case["append"]:
        state["k"], state["v"] = _normal(g, tokens, hkv, d), _normal(g, tokens, hkv, d)
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        h = state["pool"].handle
        n = pkv.pkv_attention_window_workspace_bytes(h, len(rows), tokens, width, w, s)
        state["ws"], state["ws_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
        state["out"] = torch.empty_like(state["q"])
        pkv.pkv_attention_window_plan(h, state["ctx"], state["starts"], len(rows), tokens, width, w, s, state["ws"], n)
    return state


def _prepare_rope(case, g, rng):
    t, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    blocks = -(-t // BS) * 5 // 4 + 2
    state = {"case": case, **_cache(case, g, blocks)}
    if case["packed"]:  # q, k and v side by side in one row of the projection's output
        row = _normal(g, t, (hq + 2 * hkv), d)
        state["q"], state["k"], state["v"] = row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:]
    else:
        state["q"], state["k"], state["v"] = _normal(g, t, hq, d), _normal(g, t, hkv, d), _normal(g, t, hkv, d)
    pos, left = [], t
    while left:  # runs of consecutive positions, as chunks and single tokens have them
        n = min(left, _log(rng, 1, 4096))
        at = rng.randrange(max(1, case["reach"]))
        pos += range(at, at + n)
        left -= n
    ids = rng.sample(range(blocks), -(-t // BS))
    state.update(pos=_ints(pos), slots=_ints([ids[i // BS] * BS + i % BS for i in range(t)], torch.int64))
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        state["rope"] = pkv.Rope(case["head_dim"], case["rot_dim"], interleaved=case["layout"] == "interleaved", base=case["base"],
                                 scaling=case["scaling"], factor=case["factor"], original_context=case["original"])
        state["q_out"] = torch.empty(t, hq, d, dtype=torch.float16, device="cuda")
    return state


def _prepare_copy(case, g, rng):
    ids = rng.sample(range(case["blocks"]), 2 * case["pairs"])
    pairs = [(ids[2 * i], ids[2 * i + 1]) for i in range(case["pairs"])]
    return {"case": case, **_cache(case, g, case["blocks"], case["layers"]), "pairs": _ints(pairs)}


def _prepare_fork(case, g, rng):
    ctx = _row_lens(case, case["parents"])
    p, c = case["parents"], case["children"]
    width = max(-(-x // BS) for x in ctx) + 1
    need = sum(-(-x // BS) for x in ctx) + p * c
    ids = rng.sample(range(need + 8), need)
    tables = [[ids.pop() for _ in range(-(-x // BS))] for x in ctx]
    tables = [r + [-1] * (width - len(r)) for r in tables] + [[-1] * width for _ in range(p * c)]
    forks = [(i, p + i * c + j, ids.pop()) for i in range(p) for j in range(c)]
    rng.shuffle(forks)
    return {"case": case, **_cache(case, g, need + 8, case["layers"]), "tables": _ints(tables), "ctx": _ints(ctx + [0] * (p * c)),
            "forks": _ints(forks), "rows": p * (1 + c), "width": width}


def _prepare_compact(case, g, rng):
    ctx = _row_lens(case, case["rows"])
    ids = rng.sample(range(case["blocks"]), _live_blocks(case))
    common = [ids.pop() for _ in range(case["shared"])]
    tables = [common + [ids.pop() for _ in range(max(1, -(-x // BS)))] for x in ctx]
    width = max(map(len, tables))
    tables = [r + [-1] * (width - len(r)) for r in tables]
    state = {"case": case, **_cache(case, g, case["blocks"], case["layers"]), "tables": _ints(tables), "rows": len(tables), "width": width}
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        n = pkv.pkv_compact_workspace_bytes(state["pool"].handle)
        state["ws"], state["ws_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
        state["new"], state["remap"] = torch.empty_like(state["tables"]), torch.empty(case["blocks"], dtype=torch.int32, device="cuda")
        state["live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return state


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    return {"window": _run_window, "rope": _run_rope, "copy": _run_copy, "fork": _run_fork, "compact": _run_compact}[state["case"]["op"]](state)


def _contents(state):
    """The whole cache as the values it stands for (8-bit: the codes' values and the scale bytes beside them)."""
    if "scales" in state:
        return state["cache"].view(torch.float8_e4m3fn), state["scales"]
    return (state["cache"],)


def _run_window(st):
    case = st["case"]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        h, rest = st["pool"].handle, (st["tables"], st["width"], st["ctx"], st["starts"], st["rows"], st["tokens"], st["out"],
                                      st["ws"], st["ws_bytes"])
        if case["append"]:
            pkv.pkv_attention_append(h, 0, st["q"], st["k"], st["v"], st["slots"], *rest)
            return (st["out"], *_contents(st))
        pkv.pkv_attention(h, 0, st["q"], *rest)
        return st["out"]
    cache, pos, t, hkv, d = st["cache"][0], st["pos"], st["tokens"], case["kv_heads"], case["head_dim"]
    if case["append"]:
        cache[0][st["slots"] // BS, :, st["slots"] % BS] = st["k"]
        cache[1][st["slots"] // BS, :, st["slots"] % BS] = st["v"]
    # the positions that each token sees, side by side: the first tokens outside its window, then the window
    first = (pos + 1 - case["window"]).clamp(min=0)
    head = first.clamp(max=case["sinks"])
    j = torch.arange(st["seen"], device="cuda")
    key = torch.where(j < head[:, None], j, first[:, None] + j - head[:, None])
    there = key <= pos[:, None]
    key = torch.where(there, key, pos[:, None])
    block = st["tables"][st["row_of"][:, None], key // BS].long()
    k, v = cache[0][block, :, key % BS], cache[1][block, :, key % BS]  # [token, key, head, dim]
    if case["kv_dtype"] == E4M3:
        s = st["scales"][0][block, :, :, key % BS].int() - 127  # [token, key, head, K or V]
        k = torch.ldexp(k.view(torch.float8_e4m3fn).float(), s[..., 0, None])
        v = torch.ldexp(v.view(torch.float8_e4m3fn).float(), s[..., 1, None])
    q = st["q"].float().view(t, hkv, -1, d)
    x = torch.einsum("tghd,tkgd->tghk", q, k.float()) / math.sqrt(d)
    x = x.masked_fill(~there[:, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    out = torch.einsum("tghk,tkgd->tghd", e / e.sum(-1, keepdim=True), v.float()).reshape(t, -1, d).half()
    return (out, *_contents(st)) if case["append"] else out


def _frequencies(case):
    """Radians a token of each rotated pair, in 64 bits."""
    r = case["rot_dim"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    f = case["base"] ** (-2 * i / r)
    if case["scaling"] == "linear":
        f = f / case["factor"]
    elif case["scaling"] == "bands":  # pairs that turn often over the original context keep their pace
        keep = ((case["original"] * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / case["factor"]
    elif case["scaling"] == "ramp":  # the same between two pairs, linear in the pair's number
        lo, hi = (r * math.log(case["original"] / (n * 2 * math.pi)) / (2 * math.log(case["base"])) for n in (32, 1))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / case["factor"]
    return f


def _rotated(x, cos, sin, case):
    r = case["rot_dim"]
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1).half()


def _run_rope(st):
    case = st["case"]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pkv.pkv_rope_append(st["pool"].handle, 0, st["rope"].handle, st["q"], st["q"].stride(0), st["k"], st["k"].stride(0), st["v"],
                            st["v"].stride(0), st["pos"], st["slots"], case["tokens"], st["q_out"])
        return st["q_out"], st["cache"]
    angle = st["pos"].double()[:, None, None] * _frequencies(case)
    cos, sin = angle.cos().float(), angle.sin().float()
    cache = st["cache"][0]
    cache[0][st["slots"] // BS, :, st["slots"] % BS] = _rotated(st["k"], cos, sin, case)
    cache[1][st["slots"] // BS, :, st["slots"] % BS] = st["v"]
    return _rotated(st["q"], cos, sin, case), st["cache"]


def _run_copy(st):
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pkv.pkv_copy_blocks(st["pool"].handle, st["pairs"], st["case"]["pairs"])
        return _contents(st)
    src, dst = st["pairs"].long().unbind(1)
    st["cache"][:, :, dst] = st["cache"][:, :, src]
    if "scales" in st:
        st["scales"][:, dst] = st["scales"][:, src]
    return _contents(st)


def _run_fork(st):
    case = st["case"]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pkv.pkv_fork_rows(st["pool"].handle, st["tables"], st["width"], st["ctx"], st["rows"], st["forks"],
                          case["parents"] * case["children"])
        return (*_contents(st), st["tables"], st["ctx"])
    parent, child, new = st["forks"].long().unbind(1)
    ctx, table = st["ctx"][parent], st["tables"][parent]
    full, tail = (ctx // BS)[:, None], (ctx % BS)[:, None]
    at = torch.arange(st["width"], device="cuda")
    st["tables"][child] = torch.where(at < full, table, torch.where((at == full) & (tail > 0), new[:, None].int(), -1))
    st["ctx"][child] = ctx
    last = table.gather(1, full.long())[:, 0]
    last = torch.where(last >= 0, last, 0).long()
    copied = torch.arange(BS, device="cuda") < tail  # [fork, slot]
    st["cache"][:, :, new] = torch.where(copied[:, None, :, None], st["cache"][:, :, last], st["cache"][:, :, new])
    if "scales" in st:
        st["scales"][:, new] = torch.where(copied[:, None, None], st["scales"][:, last], st["scales"][:, new])
    return (*_contents(st), st["tables"], st["ctx"])


def _run_compact(st):
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pkv.pkv_compact(st["pool"].handle, st["tables"], st["width"], st["rows"], st["new"], st["remap"], st["live"], st["ws"], st["ws_bytes"])
        return (*_contents(st), st["new"], st["remap"], st["live"])
    n = st["case"]["blocks"]
    held = torch.zeros(n + 1, dtype=torch.bool, device="cuda")
    held[(st["tables"] + 1).long()] = True
    held = held[1:]
    live = held.sum()
    at = torch.arange(n, device="cuda")
    src, dst = (held & (at >= live)).nonzero()[:, 0], (~held & (at < live)).nonzero()[:, 0]
    st["cache"][:, :, dst] = st["cache"][:, :, src]
    if "scales" in st:
        st["scales"][:, dst] = st["scales"][:, src]
    remap = torch.where(held, at, -1)
    remap[src] = dst
    tables = torch.where(st["tables"] >= 0, remap[st["tables"].clamp(min=0).long()], -1)
    return (*_contents(st), tables.int(), remap.int(), live.int()[None])


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"window": _exact_window, "rope": _exact_rope, "copy": _exact_copy, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](case, st)


def _exact_window(case, st):
    cache = st["cache"][0].clone()
    tables, slots = st["tables"].tolist(), st["slots"].tolist()
    if case["append"]:
        for t, slot in enumerate(slots):
            cache[0, slot // BS, :, slot % BS] = st["k"][t]
            cache[1, slot // BS, :, slot % BS] = st["v"][t]
    group = case["q_heads"] // case["kv_heads"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (new, ctx) in enumerate(_window_rows(case)):
        held = [j for j in range(-(-ctx // BS)) if tables[b][j] >= 0]
        ids = _ints([tables[b][j] for j in held], torch.int64)
        key = (_ints(held, torch.int64)[:, None] * BS + torch.arange(BS, device="cuda")).flatten()
        kv = cache[:, ids]  # [K or V, block, head, slot, dim]
        if case["kv_dtype"] == E4M3:
            e = st["scales"][0, ids].permute(2, 0, 1, 3).double() - 127
            kv = kv.view(torch.float8_e4m3fn).double() * torch.exp2(e)[..., None]
        kv = kv.double().transpose(1, 2).flatten(2, 3).repeat_interleave(group, 1)  # [K or V, query head, key, dim]
        p = torch.arange(ctx - new, ctx, device="cuda")[:, None]
        sees = (key <= p) & ((key > p - case["window"]) | (key < case["sinks"]))
        x = st["q"][at:at + new].double().transpose(0, 1) @ kv[0].transpose(1, 2) / math.sqrt(case["head_dim"])
        prob = torch.softmax(x.masked_fill(~sees, -math.inf), -1)
        kv[1][:, ~sees.any(0)] = 0
        out[at:at + new] = (prob @ kv[1]).transpose(0, 1)
        at += new
    return (out, cache[None]) if case["append"] else out


def _exact_rope(case, st):
    r, out = case["rot_dim"], []
    pair = range(r // 2)
    turn = []
    for i in pair:  # each pair's radians a token, from the definition
        f = case["base"] ** (-2.0 * i / r)
        slow = f / case["factor"]
        if case["scaling"] == "linear":
            f = slow
        elif case["scaling"] == "bands":
            turns = case["original"] * f / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - 1) / 3))
            f = slow + share * (f - slow)
        elif case["scaling"] == "ramp":
            lo, hi = (r * math.log(case["original"] / (2 * math.pi * n)) / (2 * math.log(case["base"])) for n in (32, 1))
            lo, hi = max(0, math.floor(lo)), min(r - 1, math.ceil(hi))
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f + share * (slow - f)
        turn.append(f)
    angle = st["pos"].double()[:, None] * torch.tensor(turn, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.ones_like(angle), angle)[:, None]  # a rotation is a complex product
    first = list(pair) if case["layout"] == "half" else [2 * i for i in pair]
    second = [i + r // 2 for i in pair] if case["layout"] == "half" else [2 * i + 1 for i in pair]
    for x in (st["q"], st["k"]):
        x = x.double().clone()
        y = torch.complex(x[..., first], x[..., second]) * z
        x[..., first], x[..., second] = y.real, y.imag
        out.append(x)
    cache = st["cache"].double()
    for t, slot in enumerate(st["slots"].tolist()):
        cache[0, 0, slot // BS, :, slot % BS], cache[0, 1, slot // BS, :, slot % BS] = out[1][t], st["v"][t].double()
    return out[0], cache


def _exact_copy(case, st):
    got = [x.clone() for x in _contents_raw(st)]
    for src, dst in st["pairs"].tolist():
        for x in got:
            x[:, dst] = x[:, src]
    return _as_contents(st, got)


def _exact_fork(case, st):
    got = [x.clone() for x in _contents_raw(st)]
    tables, ctx = st["tables"].tolist(), st["ctx"].tolist()
    for parent, child, new in st["forks"].tolist():
        n, rest = divmod(ctx[parent], BS)
        tables[child] = tables[parent][:n] + ([new] if rest else [])
        tables[child] += [-1] * (st["width"] - len(tables[child]))
        ctx[child] = ctx[parent]
        if rest:
            last = tables[parent][n]
            values = got[0]  # [layer, block, K or V, head, slot, dim]
            values[:, new, :, :, :rest] = values[:, last, :, :, :rest]
            if len(got) > 1:
                got[1][:, new, :, :, :rest] = got[1][:, last, :, :, :rest]
    return (*_as_contents(st, got), _ints(tables), _ints(ctx))


def _exact_compact(case, st):
    got = [x.clone() for x in _contents_raw(st)]
    tables = st["tables"].tolist()
    held = sorted({x for row in tables for x in row if x >= 0})
    n = len(held)
    there = set(held)
    remap = [x if x in there else -1 for x in range(case["blocks"])]
    holes = [x for x in range(n) if x not in there]
    for src, dst in zip([x for x in held if x >= n], holes):
        for x in got:
            x[:, dst] = x[:, src]
        remap[src] = dst
    tables = [[remap[x] if x >= 0 else -1 for x in row] for row in tables]
    return (*_as_contents(st, got), _ints(tables), _ints(remap), _ints([n]))


def _contents_raw(st):
    """The cache with the block as its second dimension, and the scales (which have it there)."""
    return [st["cache"].transpose(1, 2).contiguous()] + ([st["scales"]] if "scales" in st else [])


def _as_contents(st, got):
    cache = got[0].transpose(1, 2).contiguous()
    return (cache.view(torch.float8_e4m3fn), got[1]) if "scales" in st else (cache,)
