"""What the 4-bit cache and the normalising append are measured on: attention over a cache held in 4 bits, storing into it
and reading back, and norms of queries and keys with the position rotation on the way into the cache.

Every case is a dict of plain values.  `prepare` makes what a serving program holds before the call (inputs, the
pool, block tables, the pass's plan); `run` is one call, either the library's (`own`) or its plain form in elementary
torch operations; `exact` is the operator's definition in 64 bits.

The 4-bit cache: 32 consecutive values of a cached row (one token, one KV head, K or V) share a scale s, the smallest
fp16 number of at most 8 significant bits that is no less than a seventh of their largest magnitude; each is held as the
integer nearest to x / s (ties to even), -7 .. 7, plus 8.  A (block, KV head) is a record of 18 * head_dim bytes:
K's codes [head_dim / 32][16 tokens][16 bytes] (the lower half of a byte first), V's, then the scales
[16 tokens][K, V][head_dim / 32] in fp16.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per block
GROUP = 32  # values that share a scale


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    attend = dict(op="attend", window=0, sinks=0, chunks="", lens=11)
    norm = dict(op="norm", layout="half", base=10000.0, scaling="none", factor=1.0, original=8192, packed=False, eps=1e-6,
                offset=0.0)
    return [
        # one user's decode step: latency alone
        dict(attend, name="attend_one", q_heads=12, kv_heads=2, head_dim=128, decode=1, ctx_lo=700, ctx_hi=700),
        # a full decode batch, contexts from a few tokens to 8k
        dict(attend, name="attend_decode", q_heads=12, kv_heads=2, head_dim=128, decode=256, ctx_lo=1, ctx_hi=8192),
        # a few very long contexts with wide heads
        dict(attend, name="attend_long", q_heads=16, kv_heads=4, head_dim=256, decode=4, ctx_lo=262144, ctx_hi=262144),
        # long conversations behind a sliding window, small heads, the pages behind the window given back
        dict(attend, name="attend_window", q_heads=8, kv_heads=2, head_dim=64, decode=200, ctx_lo=1, ctx_hi=20000,
             window=2048, sinks=4),
        # a mixed pass: decode rows and two prompt chunks, one of them far into its prompt
        dict(attend, name="attend_chunks", q_heads=12, kv_heads=2, head_dim=128, decode=83, ctx_lo=64, ctx_hi=1100,
             chunks="2048:0,1000:5000"),
        # one token of one row: latency alone
        dict(norm, name="norm_one", q_heads=12, kv_heads=2, head_dim=128, rot_dim=128, tokens=1, reach=4000),
        # a pass of prompt chunks out of one packed projection
        dict(norm, name="norm_chunks", q_heads=12, kv_heads=2, head_dim=128, rot_dim=128, tokens=8192, reach=200000,
             base=1000000.0, packed=True),
        # wide heads, a quarter of each rotated, weights kept as their distance from one
        dict(norm, name="norm_wide", q_heads=16, kv_heads=4, head_dim=256, rot_dim=64, tokens=1501, reach=60000,
             layout="interleaved", scaling="ramp", factor=4.0, eps=1e-5, offset=1.0),
        # the new tokens of a few rows
        dict(op="store", name="store_few", kv_heads=2, head_dim=128, tokens=5),
        # a pass of prompt chunks
        dict(op="store", name="store_many", kv_heads=2, head_dim=128, tokens=8192),
        # a pass with wide heads, an odd number of tokens
        dict(op="store", name="store_wide", kv_heads=4, head_dim=256, tokens=3001),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "norm", "store"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 6, 8])
    if op == "attend":
        windowed = rng.random() < 0.4
        case = dict(op=op, q_heads=hq, kv_heads=hkv, head_dim=d, window=_log(rng, 1, 4096) if windowed else 0,
                    sinks=rng.choice([0, 1, 4, 16, 100]) if windowed else 0, decode=0, ctx_lo=1, ctx_hi=1, chunks="",
                    lens=rng.randrange(1 << 20))
        if rng.random() < 0.6:
            case.update(decode=_log(rng, 1, 256), ctx_hi=_log(rng, 1, 60000))
        else:
            case.update(decode=_log(rng, 1, 40), ctx_hi=_log(rng, 1, 2000),
                        chunks=",".join("%d:%d" % (_log(rng, 2, 1500), rng.choice([0, _log(rng, 1, 5000)])) for _ in range(rng.randint(1, 3))))
        # no more than the largest listed ones, nor more keys side by side than the plain form has room for
        while case["ctx_hi"] > 1 and (work(case)["bytes"] > 3e8 or work(case)["flops"] > 2e10 or
                                      case["decode"] * case["ctx_hi"] * hkv * d > 2e9):
            case["ctx_hi"] //= 2
        while case["chunks"] and work(case)["flops"] > 2e10:
            case["chunks"] = ",".join("%d:%d" % (max(2, int(c.split(":")[0]) // 2), int(c.split(":")[1]) // 2) for c in case["chunks"].split(","))
        return case
    if op == "norm":
        tokens = _log(rng, 1, 8192)
        while tokens > 1 and tokens * (hq + 2 * hkv) * d > 8192 * 16 * 128:
            tokens //= 2
        return dict(op=op, q_heads=hq, kv_heads=hkv, head_dim=d, rot_dim=rng.choice([d, d, d // 2, d // 4]), tokens=tokens,
                    reach=_log(rng, 10, 1000000), layout=rng.choice(["half", "interleaved"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "linear", "bands", "ramp"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]), original=rng.choice([2048, 4096, 8192]), packed=rng.random() < 0.5,
                    eps=rng.choice([1e-5, 1e-6]), offset=rng.choice([0.0, 1.0]))
    tokens = _log(rng, 1, 8192)
    while tokens > 1 and tokens * hkv * d > 3001 * 4 * 256:
        tokens //= 2
    return dict(op=op, kv_heads=hkv, head_dim=d, tokens=tokens)


def _rows(case):
    """(new tokens, context with them) of every row."""
    rng = random.Random(case["lens"])
    rows = [(1, rng.randint(case["ctx_lo"], case["ctx_hi"])) for _ in range(case["decode"])]
    for c in case["chunks"].split(","):
        if c:
            new, cached = (int(x) for x in c.split(":"))
            rows.append((new, new + cached))
    rng.shuffle(rows)
    return rows


def _token_bytes(case):
    """Bytes of one token's K and V in the 4-bit cache: half a byte a value and an fp16 scale for 32 of them."""
    return 2 * case["kv_heads"] * (case["head_dim"] // 2 + 2 * case["head_dim"] // GROUP)


def work(case):
    d = case["head_dim"]
    if case["op"] == "attend":
        w, s = case["window"] or 1 << 30, case["sinks"]
        keys = pairs = tokens = 0
        for new, ctx in _rows(case):
            lo = max(0, ctx - new - w + 1)
            keys += ctx - lo + min(s, lo)
            tokens += new
            if ctx <= w:
                pairs += new * (2 * ctx - new + 1) // 2
            else:
                for p in range(ctx - new, ctx):
                    first = max(0, p - w + 1)
                    pairs += p + 1 - first + min(s, first)
        return {"bytes": keys * _token_bytes(case) + tokens * case["q_heads"] * d * 4 + 4 * keys // BS,
                "flops": 4 * pairs * case["q_heads"] * d}
    t = case["tokens"]
    if case["op"] == "norm":
        heads = case["q_heads"] + case["kv_heads"]
        return {"bytes": t * (4 * case["q_heads"] * d + 8 * case["kv_heads"] * d + 12) + 4 * d,
                "flops": t * heads * (4 * d + 3 * case["rot_dim"])}
    # the new rows read and stored, then every slot read back
    slots = _store_blocks(case) * BS
    return {"bytes": t * (4 * case["kv_heads"] * d + _token_bytes(case) + 8) + slots * (_token_bytes(case) + 4 * case["kv_heads"] * d + 8),
            "flops": 4 * t * case["kv_heads"] * d + 2 * slots * case["kv_heads"] * d}


def _store_blocks(case):
    return -(-case["tokens"] // BS) * 9 // 8 + 1


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float16)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _quantized(x):
    """fp16 [.., d] as codes (uint8 [.., d / 2], two to a byte) and scales (fp16 [.., d / 32])."""
    x = x.float().unflatten(-1, (-1, GROUP))
    v = x.abs().amax(-1).double() / 7
    m, _ = torch.frexp(v)  # in [0.5, 1)
    s = torch.ceil(m * 256) * torch.where(v > 0, v / m, 0.0) / 256  # 8 significant bits, upwards
    s = (torch.ceil(s * 2.0 ** 24) * 2.0 ** -24).float()  # a multiple of fp16's smallest number
    q = torch.where(s[..., None] > 0, x / s[..., None], 0.0)
    code = (torch.round(q) + 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, s.half()


def _parts(records, d):
    """Views of the records [.., 18 d]: codes [.., K or V, group, token, 16] and scales [.., token, K or V, group]."""
    lead = records.shape[:-1]
    codes = records[..., :16 * d].unflatten(-1, (2, d // GROUP, BS, 16))
    scales = records[..., 16 * d:].view(torch.float16).view(*lead, BS, 2, d // GROUP)
    return codes, scales


def _values(records, d):
    """The values that records [.., 18 d] stand for, in 32 bits: [.., K or V, token, d]."""
    codes, scales = _parts(records, d)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)  # [.., K or V, group, token, 32]
    s = scales.float().movedim(-3, -1)  # [.., K or V, group, token]
    return ((c.float() - 8) * s[..., None]).movedim(-3, -2).flatten(-2)


def _filled(g, blocks, hkv, d):
    """Records of `blocks` blocks, every one holding some request's values."""
    records = torch.empty(blocks, hkv, 18 * d, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * BS * d))
    for b in range(0, blocks, step):
        part = records[b:b + step]
        codes, scales = _parts(part, d)
        for kv in range(2):
            c, s = _quantized(_normal(g, len(part), hkv, BS, d))
            codes[:, :, kv] = c.unflatten(-1, (-1, 16)).transpose(2, 3)
            scales[:, :, :, kv] = s
    return records


def _cache(case, records, q_heads):
    """The state's 4-bit cache: the records themselves, or a pool that holds them."""
    if not own:
        return {"records": records}
    from continuous_batching_paged_ragged_gb300 import pkv
    pool = pkv.Pool(1, q_heads, case["kv_heads"], case["head_dim"], len(records), kv_dtype=pkv.PKV_KV_INT4)
    pool.cache_view()[0].copy_(records)
    return {"pool": pool}


def prepare(case, seed):
    return {"attend": _prepare_attend, "norm": _prepare_norm, "store": _prepare_store}[case["op"]](case, _rng(seed), random.Random(seed))


def _prepare_attend(case, g, rng):
    rows, w, s = _rows(case), case["window"] or 1 << 30, case["sinks"]
    width = max(-(-ctx // BS) for _, ctx in rows)
    held = []  # the blocks of each row that some new token sees: the others have been given back
    for new, ctx in rows:
        lo = max(0, ctx - new - w + 1)
        held.append([j for j in range(-(-ctx // BS)) if j * BS < s or j * BS + BS > lo])
    need = sum(map(len, held))
    blocks = need + need // 8 + 2
    ids = rng.sample(range(blocks), need)
    tables = torch.full((len(rows), width), -1, dtype=torch.int32)
    at = 0
    for b, js in enumerate(held):
        tables[b, js] = torch.tensor(ids[at:at + len(js)], dtype=torch.int32)
        at += len(js)
    starts = [0]
    for new, _ in rows:
        starts.append(starts[-1] + new)
    tokens, hkv, d = starts[-1], case["kv_heads"], case["head_dim"]
    state = {"case": case, **_cache(case, _filled(g, blocks, hkv, d), case["q_heads"])}
    state.update(tables=tables.cuda(), ctx=_ints([c for _, c in rows]), starts=_ints(starts), tokens=tokens, rows=len(rows),
                 width=width, q=_normal(g, tokens, case["q_heads"], d))
    # rows with as many new tokens as one another go through the plain form together
    state["alike"] = {new: _ints([b for b, (n, _) in enumerate(rows) if n == new], torch.int64) for new in {n for n, _ in rows}}
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        h = state["pool"].handle
        state["out"] = torch.empty_like(state["q"])
        if case["window"]:
            n = pkv.pkv_attention_window_workspace_bytes(h, len(rows), tokens, width, w, s)
            state["ws"], state["ws_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
            pkv.pkv_attention_window_plan(h, state["ctx"], state["starts"], len(rows), tokens, width, w, s, state["ws"], n)
        else:
            n = pkv.pkv_attention_workspace_bytes(h, len(rows), tokens, width)
            state["ws"], state["ws_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
            pkv.pkv_attention_plan(h, state["ctx"], state["starts"], len(rows), tokens, width, state["ws"], n)
    return state


def _prepare_norm(case, g, rng):
    t, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    blocks = -(-t // BS) * 5 // 4 + 2
    state = {"case": case}
    values = _normal(g, 1, 2, blocks, hkv, BS, d)
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        state["pool"] = pkv.Pool(1, hq, hkv, d, blocks)
        state["cache"] = state["pool"].cache_view().copy_(values)
        state["rope"] = pkv.Rope(d, case["rot_dim"], interleaved=case["layout"] == "interleaved", base=case["base"],
                                 scaling=case["scaling"], factor=case["factor"], original_context=case["original"])
        state["q_out"] = torch.empty(t, hq, d, dtype=torch.float16, device="cuda")
    else:
        state["cache"] = values
    # heads of a projection's output differ in size, by a factor of e either way
    size = torch.exp(2 * torch.rand(hq + 2 * hkv, 1, generator=g, device="cuda") - 1).half()
    row = _normal(g, t, hq + 2 * hkv, d) * size
    if case["packed"]:  # q, k and v side by side in one row of the projection's output
        state["q"], state["k"], state["v"] = row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:]
    else:
        state["q"], state["k"], state["v"] = (x.contiguous() for x in row.split([hq, hkv, hkv], 1))
    for name in ("q_weight", "k_weight"):
        state[name] = (1 - case["offset"] + 0.2 * _normal(g, d)).half()
    pos, left = [], t
    while left:  # runs of consecutive positions, as chunks and single tokens have them
        n = min(left, _log(rng, 1, 4096))
        at = rng.randrange(max(1, case["reach"]))
        pos += range(at, at + n)
        left -= n
    ids = rng.sample(range(blocks), -(-t // BS))
    state.update(pos=_ints(pos), slots=_ints([ids[i // BS] * BS + i % BS for i in range(t)], torch.int64))
    return state


def _prepare_store(case, g, rng):
    t, hkv, d, blocks = case["tokens"], case["kv_heads"], case["head_dim"], _store_blocks(case)
    state = {"case": case, **_cache(case, _filled(g, blocks, hkv, d), hkv)}
    ids = rng.sample(range(blocks), -(-t // BS))
    state.update(k=_normal(g, t, hkv, d), v=_normal(g, t, hkv, d), blocks=blocks,
                 slots=_ints([ids[i // BS] * BS + i % BS for i in range(t)], torch.int64),
                 all=torch.arange(blocks * BS, device="cuda"))
    if own:
        state["k_out"] = torch.empty(blocks * BS, hkv, d, dtype=torch.float16, device="cuda")
        state["v_out"] = torch.empty_like(state["k_out"])
    return state


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    return {"attend": _run_attend, "norm": _run_norm, "store": _run_store}[state["case"]["op"]](state)


def _run_attend(st):
    case = st["case"]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pkv.pkv_attention(st["pool"].handle, 0, st["q"], st["tables"], st["width"], st["ctx"], st["starts"], st["rows"], st["tokens"],
                          st["out"], st["ws"], st["ws_bytes"])
        return st["out"]
    out = torch.empty_like(st["q"])
    for new, rows in st["alike"].items():
        for part in [rows] if new == 1 else rows.split(1):
            token = st["starts"][part].long()[:, None] + torch.arange(new, device="cuda")
            out[token] = _attended(st, part, new, st["q"][token])
    return out


def _attended(st, rows, new, q):
    """Attention of `new` tokens of each of these rows: q [row, token, head, dim]."""
    case = st["case"]
    hkv, d, w, s = case["kv_heads"], case["head_dim"], case["window"], case["sinks"]
    ctx, table = st["ctx"][rows].long(), st["tables"][rows]
    p = ctx[:, None] - new + torch.arange(new, device="cuda")  # positions [row, token]
    j = torch.arange(st["width"], device="cuda").expand(len(rows), -1)
    if w:  # the sinks' blocks, then those from the first token's window on
        first = (p[:, :1] - w + 1).clamp(min=0) // BS
        head = -(-s // BS)
        n = min(st["width"], (w + new - 2) // BS + 2)
        j = torch.cat([torch.arange(head, device="cuda").expand(len(rows), -1), first + torch.arange(n, device="cuda")], 1)
        twice = torch.cat([torch.arange(head, device="cuda") >= first, torch.zeros(len(rows), n, dtype=torch.bool, device="cuda")], 1)
    block = table.gather(1, j.clamp(max=st["width"] - 1)).clamp(min=0).long()
    kv = _values(st["records"][block], d)  # [row, block, head, K or V, slot, dim]
    k, v = (kv[:, :, :, i].transpose(1, 2).flatten(2, 3) for i in (0, 1))  # [row, head, key, dim]
    key = (j[..., None] * BS + torch.arange(BS, device="cuda")).flatten(1)[:, None]  # [row, 1, key]
    sees = key <= p[..., None]
    if w:
        sees &= ((key > p[..., None] - w) | (key < s)) & ~twice.repeat_interleave(BS, 1)[:, None]
    q = q.float().unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [row, head, of its group x token, dim]
    x = (q @ k.transpose(2, 3) / math.sqrt(d)).unflatten(2, (-1, new))
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = (e / e.sum(-1, keepdim=True)).flatten(2, 3) @ v
    return o.unflatten(2, (-1, new)).permute(0, 3, 1, 2, 4).flatten(2, 3).half()


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


def _normed_and_rotated(x, weight, cos, sin, case):
    r = case["rot_dim"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + case["eps"]) * (case["offset"] + weight.float())
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1).half()


def _run_norm(st):
    case = st["case"]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        pkv.pkv_norm_rope_append(st["pool"].handle, 0, st["rope"].handle, st["q_weight"], st["k_weight"], case["eps"], case["offset"],
                                 st["q"], st["q"].stride(0), st["k"], st["k"].stride(0), st["v"], st["v"].stride(0), st["pos"],
                                 st["slots"], case["tokens"], st["q_out"])
        return st["q_out"], st["cache"]
    angle = st["pos"].double()[:, None, None] * _frequencies(case)
    cos, sin = angle.cos().float(), angle.sin().float()
    cache = st["cache"][0]
    cache[0][st["slots"] // BS, :, st["slots"] % BS] = _normed_and_rotated(st["k"], st["k_weight"], cos, sin, case)
    cache[1][st["slots"] // BS, :, st["slots"] % BS] = st["v"]
    return _normed_and_rotated(st["q"], st["q_weight"], cos, sin, case), st["cache"]


def _run_store(st):
    d = st["case"]["head_dim"]
    if own:
        from continuous_batching_paged_ragged_gb300 import pkv
        h = st["pool"].handle
        pkv.pkv_append(h, 0, st["k"], st["v"], st["slots"], st["case"]["tokens"])
        pkv.pkv_gather(h, 0, st["all"], st["blocks"] * BS, st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    codes, scales = _parts(st["records"], d)  # views
    block, slot = st["slots"] // BS, st["slots"] % BS
    for kv, x in enumerate((st["k"], st["v"])):
        c, s = _quantized(x)  # [token, head, ..]
        codes[block, :, kv, :, slot] = c.unflatten(-1, (-1, 16))
        scales[block, :, slot, kv] = s
    block, slot = st["all"] // BS, st["all"] % BS
    kv = _values(st["records"], d)[block, :, :, slot]  # [token, head, K or V, dim]
    return kv[:, :, 0].half().contiguous(), kv[:, :, 1].half().contiguous()


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
    return {"attend": _exact_attend, "norm": _exact_norm, "store": _exact_store}[case["op"]](case, st)


def _exact_rows(records, block, slot, d):
    """What tokens at (block, slot) hold, value by value: [token, head, K or V, d]."""
    hkv = records.shape[1]
    record = (block[:, None] * hkv + torch.arange(hkv, device="cuda"))[..., None, None] * (18 * d)
    kv = torch.arange(2, device="cuda")[:, None]
    i = torch.arange(d, device="cuda")
    slot = slot[:, None, None, None]
    byte = records.view(-1)[record + kv * (8 * d) + i // 32 * 256 + slot * 16 + i % 32 // 2].int()
    code = torch.where(i % 2 == 1, byte // 16, byte % 16) - 8
    at = (record + 16 * d) // 2 + (slot * 2 + kv) * (d // 32) + i // 32
    return code.double() * records.view(torch.float16).view(-1)[at].double()


def _exact_attend(case, st):
    group = case["q_heads"] // case["kv_heads"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (new, ctx) in enumerate(_rows(case)):
        p = torch.arange(ctx - new, ctx, device="cuda")[:, None]
        key = torch.arange(ctx, device="cuda")
        sees = key <= p
        if case["window"]:
            sees &= (key > p - case["window"]) | (key < case["sinks"])
        key = key[sees.any(0)]
        sees = sees[:, key]
        kv = _exact_rows(st["records"], st["tables"][b][key // BS].long(), key % BS, case["head_dim"])
        for h in range(case["kv_heads"]):
            q = st["q"][at:at + new, h * group:(h + 1) * group].double().transpose(0, 1)
            x = (q @ kv[:, h, 0].T / math.sqrt(case["head_dim"])).masked_fill(~sees, -math.inf)
            out[at:at + new, h * group:(h + 1) * group] = (torch.softmax(x, -1) @ kv[:, h, 1]).transpose(0, 1)
        at += new
    return out


def _exact_norm(case, st):
    r, out = case["rot_dim"], []
    turn = []
    for i in range(r // 2):  # each pair's radians a token, from the definition
        f = case["base"] ** (-2.0 * i / r)
        slow = f / case["factor"]
        if case["scaling"] == "linear":
            f = slow
        elif case["scaling"] == "bands":
            turns = case["original"] * f / (2 * math.pi)
            f = slow + min(1.0, max(0.0, (turns - 1) / 3)) * (f - slow)
        elif case["scaling"] == "ramp":
            lo, hi = (r * math.log(case["original"] / (2 * math.pi * n)) / (2 * math.log(case["base"])) for n in (32, 1))
            lo, hi = max(0, math.floor(lo)), min(r - 1, math.ceil(hi))
            f = f + min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) * (slow - f)
        turn.append(f)
    angle = st["pos"].double()[:, None] * torch.tensor(turn, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.ones_like(angle), angle)[:, None]  # a rotation is a complex product
    pair = list(range(r // 2))
    first = pair if case["layout"] == "half" else [2 * i for i in pair]
    second = [i + r // 2 for i in pair] if case["layout"] == "half" else [2 * i + 1 for i in pair]
    for x, weight in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        x = x.double()
        x = x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["head_dim"] + case["eps"]).sqrt()
        x = x * (weight.double() + case["offset"])
        y = torch.complex(x[..., first], x[..., second]) * z
        x[..., first], x[..., second] = y.real, y.imag
        out.append(x)
    cache = st["cache"].double()
    for t, slot in enumerate(st["slots"].tolist()):
        cache[0, 0, slot // BS, :, slot % BS], cache[0, 1, slot // BS, :, slot % BS] = out[1][t], st["v"][t].double()
    return out[0], cache


def _exact_store(case, st):
    d, n = case["head_dim"], st["blocks"] * BS
    at = torch.arange(n, device="cuda")
    got = _exact_rows(st["records"], at // BS, at % BS, d)
    # every scale that 8 significant bits can make, over fp16's range: the first that a seventh of the peak does not pass
    scales = sorted({m * 2.0 ** e for m in range(1, 256) for e in range(-24, 7)} | {0.0})
    scales = torch.tensor(scales, dtype=torch.float64, device="cuda")
    for kv, x in enumerate((st["k"], st["v"])):
        x = x.double().unflatten(-1, (d // 32, 32))
        s = scales[torch.searchsorted(scales * 7, x.abs().amax(-1))][..., None]
        low = torch.floor(x / s.clamp(min=2.0 ** -24))
        rest = x - low * s  # how far above the lower neighbour
        odd = torch.remainder(low, 2) == 1
        up = (2 * rest > s) | ((2 * rest == s) & odd)
        got[st["slots"], :, kv] = ((low + up) * s).flatten(-2)
    return got[:, :, 0], got[:, :, 1]
