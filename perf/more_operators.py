"""The operators of a decode step whose key/value cache holds 4 bits and is kept short, as they are
measured: appending rotated keys and values, attention over the cache, adding up the attention weight
that each cached position gets, and evicting the positions that got least.

`run` computes them in plain torch (own = False) or through the package's calls (own = True).

The cache holds, per page, key/value head and token, head dim / 2 bytes of 4-bit codes (an even dimension in
the low half of its byte) and an f16 scale d for each group of 32 values; a cached value is d * (code - 8).
A batch is S sequences; sequence s owns rows q_start[s] .. q_start[s + 1] - 1 of the call, and has
kv_len[s] cached tokens counting them.  Weights are f32, one per page, key/value head and token."""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32  # values of a head that share a scale


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    a = dict(op="attention", heads=32, kv_heads=8, dim=128, page=64, rows=1, window=0, lse=False)
    p = dict(op="append", heads=32, kv_heads=8, dim=128, page=64, rot=128, pairs="halves", shift=0)
    w = dict(op="weigh", heads=32, kv_heads=8, dim=128, page=64, rows=1, window=0)
    e = dict(op="evict", kv_heads=8, dim=128, page=64, sinks=4)
    return [
        # one request a few tokens in: nothing but latency
        dict(a, name="attend_1x19", seqs=1, len_min=19, len_max=19),
        # one request with a long document in its cache
        dict(a, name="attend_1x32768", seqs=1, len_min=32768, len_max=32768),
        # a served batch in full swing, its weights to be added up afterwards: the largest read of the cache
        dict(a, name="attend_40_ragged", seqs=40, len_min=1500, len_max=14011, lse=True),
        # checking five drafted tokens of each request at once (20 rows share a key/value head)
        dict(a, name="attend_verify_5_rows", seqs=8, len_min=650, len_max=3001, rows=5, page=32),
        # small heads, seven to a key/value head, a sliding window, pages of 16 tokens
        dict(a, name="attend_64_wide_window", seqs=20, len_min=1, len_max=7000, heads=28, kv_heads=4, dim=64, page=16,
             window=1900),
        # one new token for each of eight requests whose caches were thinned out: positions run ahead of slots
        dict(p, name="append_8x1", seqs=8, rows=1, len_min=3, len_max=4000, shift=9000),
        # prompts arriving beside requests that decode; adjacent pairs
        dict(p, name="append_prompts", seqs=6, rows=2777, len_min=0, len_max=900, pairs="adjacent"),
        # the weights of one decode step over caches that are held near 2048 tokens
        dict(w, name="weigh_24x2080", seqs=24, len_min=1990, len_max=2080),
        # the last 32 rows of a prompt judge all of it
        dict(w, name="weigh_prompt_end", seqs=1, len_min=16010, len_max=16010, rows=32),
        # a prompt thinned out once, before its first token is generated
        dict(e, name="evict_prompt", seqs=1, len_min=24000, len_max=24000, keep=2048, recent=32),
        # a served batch brought back to its budget after 64 more tokens each
        dict(e, name="evict_12_by_64", seqs=12, len_min=1000, len_max=1088, keep=1024, recent=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "weigh", "evict"])
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (16, 16), (64, 8), (9, 3), (8, 1)])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    case = dict(op=op, kv_heads=kv_heads, dim=dim, page=page)
    seqs = _log_int(rng, 1, 64)
    if op == "append":
        rows = _log_int(rng, 1, 2700)
        seqs = max(1, min(seqs, 15000 * 40 * 128 // (rows * (heads + 2 * kv_heads) * dim)))
        return dict(case, heads=heads, rows=rows, seqs=seqs, len_min=0, len_max=_log_int(rng, 1, 4000),
                    rot=rng.choice([dim, dim, dim // 2]), pairs=rng.choice(["halves", "adjacent"]),
                    shift=rng.choice([0, _log_int(rng, 1, 20000)]))
    if op == "evict":
        keep = _log_int(rng, 16, 4096)
        seqs = max(1, min(seqs, 16 * 1024 * 8 * 128 // (keep * kv_heads * dim)))
        len_max = _log_int(rng, keep // 2 + 1, max(keep // 2 + 1, min(32000, 40 * 7000 * 8 * 128 // (seqs * kv_heads * dim))))
        return dict(case, seqs=seqs, keep=keep, len_min=rng.randint(0, len_max), len_max=len_max,
                    sinks=rng.choice([0, 1, 4]), recent=rng.randint(0, keep - 4))
    # cached tokens x heads x dim at most those of the largest listed case, and not more products
    most = min(32768, 40 * 7000 * 8 * 128 // (seqs * kv_heads * dim), 40 * 7000 * 32 * 128 // (seqs * heads * dim))
    rows = rng.choice([1, 1, 1, 2, 3, 5, 8] if op == "attention" else [1, 1, 1, 4, 16, 32])
    len_max = _log_int(rng, rows, max(rows, most))
    if rows * heads * dim * len_max * seqs > 40 * 7000 * 32 * 128:
        rows = 1
    lse = rng.random() < 0.5
    case = dict(case, heads=heads, rows=rows, seqs=seqs, len_max=len_max, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]),
                len_min=rng.randint(rows if lse or op == "weigh" else 0, len_max))
    return dict(case, lse=lse) if op == "attention" else case


def _lengths(case):
    """(cached tokens counting the call's rows, rows) of each sequence: part of the case, not of the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lo, hi = case["len_min"], case["len_max"]
    out = []
    for s in range(case["seqs"]):
        ln = hi if s == 0 else rng.randint(lo, hi)
        if case["op"] == "append":
            n = case["rows"]
            n = n if s == 0 else rng.randint(max(1, n // 2), n)
            out.append((ln + n, n))
        elif case["op"] == "evict":
            out.append((ln, min(ln, case["keep"])))  # the rows are those that are left
        else:
            out.append((ln, case["rows"]))  # fewer tokens than rows leave rows without any
    return out


def work(case):
    H, D, lens = case["kv_heads"], case["dim"], _lengths(case)
    row = H * (D // 2 + D // 16)  # codes and scales of a token's keys, or of its values
    T = sum(n for _, n in lens)
    if case["op"] == "append":
        # q, k, v in; rotated q out; codes and scales in the cache; the table's rows; then the rows read back
        return {"bytes": T * (2 * case["heads"] * D * 4 + 2 * H * D * 4 + 2 * row + case["rot"] * 4) +
                T * (2 * row + 2 * H * D * 4), "flops": T * ((case["heads"] + H) * case["rot"] * 3 + 4 * H * D)}
    if case["op"] == "evict":
        # every weight; the rows that are left in and out; then read back
        over = [(ln, n) for ln, n in lens if ln > n]
        return {"bytes": sum(ln * H * 4 + n * (4 * row + 4 * H + 4 * H) for ln, n in over) + T * (2 * row + 2 * H * D * 4),
                "flops": sum(ln * H for ln, _ in over) + T * 2 * H * D}
    W, nbytes, pairs = case["window"], 0, 0
    token = 2 * row if case["op"] == "attention" else row + 8 * H  # keys and values, or keys and weights in and out
    for ln, n in lens:
        reach = [(max(0, e - W) if W else 0, max(0, e)) for e in range(ln - n + 1, ln + 1)]
        nbytes += (max(e for _, e in reach) - min(b for b, _ in reach)) * token
        pairs += sum(e - b for b, e in reach)
    if case["op"] == "weigh":
        return {"bytes": nbytes + T * case["heads"] * (D + 1) * 4, "flops": 2 * pairs * case["heads"] * D}
    return {"bytes": nbytes + T * case["heads"] * (2 * D + case["lse"]) * 4, "flops": 4 * pairs * case["heads"] * D}


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _quantise(x):
    """Codes (a byte holds two) and scales of rows of x [.., dim], a scale per group."""
    g = x.unflatten(-1, (-1, GROUP))
    size = g.abs()
    first = torch.where(size == size.amax(-1, keepdim=True), torch.arange(GROUP, device=DEV), GROUP).amin(-1, keepdim=True)
    d = (g.gather(-1, first)[..., 0] * -0.125).clamp(-65504, 65504).half()
    df = d.float()[..., None]
    inv = torch.where(df != 0, torch.ones_like(df) / df, torch.zeros_like(df))
    c = ((g * inv).round() + 8).clamp(0, 15).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | c[..., 1::2] << 4, d


def _values(codes, scale):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return ((c.float() - 8).unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


def _filled(pages, H, page, D, g):
    """Codes and scales of normally distributed values with outlying channels."""
    codes = torch.empty((pages, H, page, D // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((pages, H, page, D // GROUP), dtype=torch.float16, device=DEV)
    channel = 1 + 3 * (torch.rand(D, device=DEV, generator=g) < 0.04)
    step = max(1, (1 << 26) // (H * page * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        codes[a:a + n], scale[a:a + n] = _quantise(torch.randn((n, H, page, D), device=DEV, generator=g) * channel)
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(case)
    need = [max(1, -(-ln // page)) for ln, _ in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, device=DEV, generator=g, dtype=torch.int32).cpu()
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):  # the pages of a sequence lie anywhere in the pool
        table[s, :n] = order[at:at + n]
        at += n
    T = sum(n for _, n in lens)
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st["table"], st["kv_len"], st["q_start"] = table.to(DEV), i32([ln for ln, _ in lens]), i32(starts)
    st["max_q"], st["T"] = max(1, max(n for _, n in lens)), max(1, T)
    st["k_codes"], st["k_scale"] = _filled(pages, H, page, D, g)
    st["v_codes"], st["v_scale"] = _filled(pages, H, page, D, g)
    T = st["T"]
    if case["op"] == "append":
        Hq = case["heads"]
        # the three parts of one fused projection's output: rows of (Hq + 2 H) D values
        qkv = torch.randn((T, (Hq + 2 * H) * D), device=DEV, generator=g)
        st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        st["k"] = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        st["v"] = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
        half = case["rot"] // 2
        f = 500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        top = max(ln for ln, _ in lens) + case["shift"]
        angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * f
        st["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()  # [positions][cosines, sines]
        st["positions"] = None
        if case["shift"]:  # what was evicted from each sequence so far
            gone = random.Random(seed).choices(range(case["shift"] + 1), k=len(lens))
            st["positions"] = torch.cat([torch.arange(ln - n, ln) + x for (ln, n), x in zip(lens, gone)]).to(torch.int32).to(DEV)
        st["q_out"] = torch.empty((T, Hq, D), device=DEV)
    elif case["op"] == "evict":
        st["weight"] = torch.randn((pages, H, page), device=DEV, generator=g).mul(2).exp() * 0.05
        st["len_out"] = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
        st["kept"] = torch.zeros((len(lens), H, case["keep"]), dtype=torch.int32, device=DEV)
    else:
        st["q"] = torch.randn((T, case["heads"], D), device=DEV, generator=g) * 1.5
        st["out"] = torch.empty((T, case["heads"] * D), device=DEV)
        st["lse"] = torch.empty((T, case["heads"]), device=DEV) if case.get("lse") else None
    if case["op"] == "weigh":  # the rows' log-sum-exp, as attention has given it
        st["weight"] = torch.randn((pages, H, page), device=DEV, generator=g).mul(2).exp() * 0.05
        st["lse"] = torch.cat([torch.logsumexp(sc, -1).flatten(0, 1).T for _, _, sc in _scores64(st)]).float().contiguous()
    if case["op"] in ("append", "evict"):  # the rows read back
        st["k_out"] = torch.empty((T, H, D), device=DEV)
        st["v_out"] = torch.empty((T, H, D), device=DEV)
    if own:
        import quantised_decode_mat_gb300 as qmd
        st["cache"] = qmd.KV4Cache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
        st["batch"] = qmd.KVBatch(st["table"], st["kv_len"], st["q_start"], st["max_q"], T)
        if case["op"] == "evict":
            st["back"] = qmd.KVBatch(st["table"], st["len_out"], st["q_start"], st["max_q"], T)
        if case["op"] == "attention":
            st["workspace"] = qmd.kv_workspace()
    return st


# ---- the operators, plainly --------------------------------------------------------------------

def _rows(st):
    """Sequence and slot of each row."""
    q_start = st["q_start"].long()
    row = torch.arange(st["T"], device=DEV)
    s = torch.searchsorted(q_start[1:], row, right=True).clamp(max=len(q_start) - 2)
    return s, st["kv_len"].long()[s] - (q_start[s + 1] - row)


def _place(st, s, slot):
    page = st["case"]["page"]
    return st["table"].long()[s, (slot // page).clamp(0, st["table"].shape[1] - 1)], slot % page


def _rotate(x, rope, pos, rot, pairs):
    c, s = rope[pos, None, :rot // 2], rope[pos, None, rot // 2:]
    y = x.clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _read(st, s, slot):
    page, tok = _place(st, s, slot)
    return (_values(st["k_codes"][page, :, tok], st["k_scale"][page, :, tok]),
            _values(st["v_codes"][page, :, tok], st["v_scale"][page, :, tok]))


def _plain_append(st):
    case = st["case"]
    s, slot = _rows(st)
    pos = slot if st["positions"] is None else st["positions"].long()
    q = _rotate(st["q"], st["rope"], pos, case["rot"], case["pairs"])
    k = _rotate(st["k"], st["rope"], pos, case["rot"], case["pairs"])
    page, tok = _place(st, s, slot)
    for x, codes, scale in ((k, st["k_codes"], st["k_scale"]), (st["v"], st["v_codes"], st["v_scale"])):
        codes[page, :, tok], scale[page, :, tok] = _quantise(x)
    return (q,) + _read(st, s, slot)


def _scores(st):
    """Scores [seqs, kv heads, rows, heads to one, slots], what is seen of them, and the rows that they belong to."""
    case = st["case"]
    H, D, n = case["kv_heads"], case["dim"], st["max_q"]
    G = case["heads"] // H
    rows = (st["q_start"][1:] - st["q_start"][:-1]).long()
    i = torch.arange(n, device=DEV)
    at = (st["q_start"][:-1].long()[:, None] + i).clamp(max=st["T"] - 1)
    q = st["q"][at].unflatten(2, (H, G)).permute(0, 2, 1, 3, 4)
    table = st["table"].long()
    K = _values(st["k_codes"][table], st["k_scale"][table]).transpose(1, 2).flatten(2, 3)  # [seqs, kv heads, slots, dim]
    last = st["kv_len"].long()[:, None] - rows[:, None] + i  # the newest slot that a row sees
    j = torch.arange(K.shape[2], device=DEV)
    sees = j <= last[..., None]
    if case["window"]:
        sees &= j > last[..., None] - case["window"]
    sees = (sees & (i < rows[:, None])[..., None])[:, None, :, None]
    score = (q.flatten(2, 3) @ K.transpose(2, 3)).unflatten(2, (n, G)) * (1 / math.sqrt(D))
    return score, sees, at


def _plain_attention(st):
    score, sees, _ = _scores(st)
    S, H, n, G, _ = score.shape
    table = st["table"].long()
    V = _values(st["v_codes"][table], st["v_scale"][table]).transpose(1, 2).flatten(2, 3)
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = torch.where(sees, (score - top).exp(), 0.0)
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ V).unflatten(2, (n, G))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(S, n, -1)
    s, slot = _rows(st)
    i = torch.arange(st["T"], device=DEV) - st["q_start"].long()[s]
    if st["lse"] is None:
        return o[s, i]
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(S, n, -1)
    return o[s, i], lse[s, i]


def _plain_weigh(st):
    score, sees, at = _scores(st)
    S, H, n, G, L = score.shape
    lse = st["lse"][at].unflatten(2, (H, G)).permute(0, 2, 1, 3)
    add = torch.where(sees, (score - lse[..., None]).exp(), 0.0).sum((2, 3))  # [seqs, kv heads, slots]
    s = torch.arange(S, device=DEV)[:, None].expand(S, L)
    j = torch.arange(L, device=DEV).expand(S, L)
    held = j < st["kv_len"][:, None]
    new = j >= (st["kv_len"] - (st["q_start"][1:] - st["q_start"][:-1]))[:, None]  # the call's own rows begin at nothing
    page, tok = _place(st, s, j)
    w = torch.where(new[..., None], 0.0, st["weight"][page, :, tok]) + add.transpose(1, 2)
    st["weight"][page[held], :, tok[held]] = w[held]
    return st["weight"]


def _plain_evict(st):
    case = st["case"]
    H, keep = case["kv_heads"], case["keep"]
    S, ln = len(st["kv_len"]), st["kv_len"].long()[:, None]
    j = torch.arange(st["table"].shape[1] * case["page"], device=DEV).expand(S, -1)
    s = torch.arange(S, device=DEV)[:, None].expand_as(j)
    page, tok = _place(st, s, j)
    w = st["weight"][page, :, tok].transpose(1, 2)
    always = (j < case["sinks"]) | (j >= ln - case["recent"])
    w = torch.where(always[:, None], math.inf, w)
    w = torch.where((j < ln)[:, None], w, -math.inf)
    m = min(keep, w.shape[2])
    best = w.sort(dim=-1, descending=True, stable=True).indices[..., :m].sort(-1).values  # [seqs, kv heads, kept]
    i = torch.arange(keep, device=DEV).expand(S, H, keep)
    kept = i.clone()
    kept[..., :m] = torch.where(ln[..., None] > keep, best, kept[..., :m])
    kept = torch.where(i < ln[..., None], kept, -1)
    h = torch.arange(H, device=DEV)[:, None].expand(H, keep)
    live = kept >= 0
    sq = torch.arange(S, device=DEV)[:, None, None].expand_as(kept)[live]
    hd = h.expand_as(kept)[live]
    src, dst = kept[live], i[live]
    sp, stk = _place(st, sq, src)
    dp, dtk = _place(st, sq, dst)
    for t in ("k_codes", "k_scale", "v_codes", "v_scale", "weight"):
        st[t][dp, hd, dtk] = st[t][sp, hd, stk]
    new_len = st["kv_len"].clamp(max=keep)
    s, _ = _rows(st)
    slot = torch.arange(st["T"], device=DEV) - st["q_start"].long()[s]
    return (new_len, kept.int()) + _read(st, s, slot) + (st["weight"],)


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "weigh": _plain_weigh, "evict": _plain_evict}[op](st)
    import quantised_decode_mat_gb300 as qmd
    if op == "append":
        q = qmd.kv4_append(st["cache"], st["batch"], st["k"], st["v"], rope=st["rope"], q=st["q"], q_out=st["q_out"],
                           pairs=qmd.ROPE_HALVES if case["pairs"] == "halves" else qmd.ROPE_ADJACENT, positions=st["positions"])
        return (q,) + tuple(qmd.kv4_read(st["cache"], st["batch"], st["k_out"], st["v_out"]))
    if op == "attention":
        out = qmd.kv4_attention(st["cache"], st["batch"], st["q"], 1 / math.sqrt(case["dim"]), st["workspace"],
                                window=case["window"], out=st["out"], lse=st["lse"])
        return out if st["lse"] is None else (out, st["lse"])
    if op == "weigh":
        return qmd.kv4_weigh(st["cache"], st["batch"], st["q"], 1 / math.sqrt(case["dim"]), st["lse"], st["weight"],
                             window=case["window"])
    n = qmd.kv4_evict(st["cache"], st["batch"], st["weight"], case["keep"], sinks=case["sinks"], recent=case["recent"],
                      len_out=st["len_out"], kept=st["kept"])
    return (n, st["kept"]) + tuple(qmd.kv4_read(st["cache"], st["back"], st["k_out"], st["v_out"])) + (st["weight"],)


# ---- the definitions, in 64 bits ---------------------------------------------------------------

def _r32(x):
    """x rounded to 32 bits: the append is defined with every operation rounded so (the codes hang on it)."""
    return x.float().double()


def _held(codes, scale):
    """Codes and scales [.., bytes], [.., groups] as 64-bit values [.., dim]."""
    out = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=codes.device)
    out[..., 0::2] = (codes % 16).double() - 8
    out[..., 1::2] = (codes // 16).double() - 8
    return out * scale.double().repeat_interleave(GROUP, -1)


def _sequence(st, s, ln, codes, scale):
    """Slots 0 .. ln - 1 of sequence s in 64 bits: [slot][head][dim]."""
    page = st["case"]["page"]
    p = torch.arange(ln, device=DEV)
    at, tok = st["table"][s].long()[p // page], p % page
    return _held(st[codes][at, :, tok], st[scale][at, :, tok])


def _scores64(st):
    """Per sequence its first row, the slots, and the masked scores [kv heads, heads to one, rows, slots]."""
    case = st["case"]
    H, D = case["kv_heads"], case["dim"]
    for s, (ln, n) in enumerate(_lengths(case)):
        r0 = int(st["q_start"][s])
        K = _sequence(st, s, ln, "k_codes", "k_scale")
        q = st["q"][r0:r0 + n].double().unflatten(1, (H, -1))
        sc = torch.einsum("nhgd,lhd->hgnl", q, K) / math.sqrt(D)
        end = torch.arange(ln - n + 1, ln + 1, device=DEV)[:, None]
        j = torch.arange(ln, device=DEV)
        seen = j < end
        if case["window"]:
            seen &= j >= end - case["window"]
        yield r0, ln, sc.masked_fill(~seen, -math.inf)


def _exact_append(st):
    case = st["case"]
    s_all, k_all, v_all, q_all = 0, [], [], []
    for s, (ln, n) in enumerate(_lengths(case)):
        r0, half = s_all, case["rot"] // 2
        s_all += n
        at = torch.arange(ln - n, ln, device=DEV) if st["positions"] is None else st["positions"][r0:r0 + n].long()
        c, sn = st["rope"][at].double()[:, None].chunk(2, -1)
        turned = {}
        for name in ("q", "k"):
            x = st[name][r0:r0 + n].double()
            y = x.clone()
            halves = case["pairs"] == "halves"
            lo = torch.arange(half, device=DEV) * (1 if halves else 2)
            hi = lo + (half if halves else 1)
            y[:, :, lo] = _r32(_r32(x[:, :, lo] * c) - _r32(x[:, :, hi] * sn))
            y[:, :, hi] = _r32(_r32(x[:, :, hi] * c) + _r32(x[:, :, lo] * sn))
            turned[name] = y
        q_all.append(turned["q"])
        for x, out in ((turned["k"], k_all), (st["v"][r0:r0 + n].double(), v_all)):
            x = x.reshape(n, case["kv_heads"], -1, GROUP)
            hi, lo = x.amax(-1), x.amin(-1)
            top = torch.where(hi > -lo, hi, lo)  # the value of largest size
            tie = hi == -lo
            if tie.any():  # of two with opposite signs the first
                top = torch.where(tie & (x.argmax(-1) < x.argmin(-1)), hi, top)
            d = (top / -8).clamp(-65504, 65504).half().double()[..., None]
            inv = torch.where(d != 0, _r32(1 / d), 0.0)
            out.append((_r32(x * inv).round().clamp(-8, 7) * d).flatten(2))
    return torch.cat(q_all), torch.cat(k_all), torch.cat(v_all)


def _exact_evict(st):
    case = st["case"]
    H, D, page, keep = case["kv_heads"], case["dim"], case["page"], case["keep"]
    weight = st["weight"].double()
    new_len, kept, ks, vs = [], [], [], []
    for s, (ln, n) in enumerate(_lengths(case)):
        new_len.append(min(ln, keep))
        p = torch.arange(ln, device=DEV)
        at, tok = st["table"][s].long()[p // page], p % page
        w = st["weight"][at, :, tok].double().T.cpu()  # [head][slot]
        rows = []
        for h in range(H):
            stay = list(range(ln))
            if ln > keep:
                w_h = w[h].tolist()
                by_weight = sorted(stay[case["sinks"]:ln - case["recent"]], key=lambda j: (-w_h[j], j))
                stay = sorted(stay[:case["sinks"]] + stay[ln - case["recent"]:] +
                              by_weight[:keep - case["sinks"] - case["recent"]])
            rows.append(stay)
            i = torch.arange(len(rows[-1]), device=DEV)
            src = torch.tensor(rows[-1], device=DEV, dtype=torch.long)
            weight[at[i], h, tok[i]] = st["weight"][at[src], h, tok[src]].double()
        kept.append([r + [-1] * (keep - len(r)) for r in rows])
        if n:
            src = torch.tensor(rows, device=DEV).T  # [kept][head]
            for codes, scale, out in (("k_codes", "k_scale", ks), ("v_codes", "v_scale", vs)):
                x = _sequence(st, s, ln, codes, scale)
                out.append(x.gather(0, src[..., None].expand(-1, -1, D)))
    none = [torch.zeros((0, H, D), device=DEV, dtype=torch.float64)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return i32(new_len), i32(kept), torch.cat(ks or none), torch.cat(vs or none), weight


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "evict":
        return _exact_evict(st) if any(n for _, n in _lengths(case)) else None
    H, page = case["kv_heads"], case["page"]
    if case["op"] == "weigh":
        weight = st["weight"].double()
        for s, (r0, ln, sc) in enumerate(_scores64(st)):
            n = sc.shape[2]
            p = torch.arange(ln, device=DEV)
            at, tok = st["table"][s].long()[p // page], p % page
            lse = st["lse"][r0:r0 + n].double().T.unflatten(0, (H, -1))
            old = weight[at, :, tok]
            old[max(0, ln - n):] = 0
            weight[at, :, tok] = old + (sc - lse[..., None]).exp().sum((1, 2)).T
        return weight
    out, lse = [], []
    for s, (r0, ln, sc) in enumerate(_scores64(st)):
        V = _sequence(st, s, ln, "v_codes", "v_scale")
        p = torch.softmax(sc, -1).nan_to_num(0.0) if ln else sc  # rows that see nothing
        out.append(torch.einsum("hgnl,lhd->nhgd", p, V).flatten(1))
        lse.append(torch.logsumexp(sc, -1).flatten(0, 1).T if ln else None)
    return torch.cat(out) if st["lse"] is None else (torch.cat(out), torch.cat(lse))
