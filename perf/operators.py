"""The decode-step operators around the quantised projections, as they are measured: appending
rotated keys and values to a paged 8-bit cache, reading cached rows back, attention over that cache,
and the low-rank adapters of many requests beside a shared projection.

`run` computes them in plain torch (own = False) or through the package's calls (own = True).

The cache holds, per page and key/value head, int8 codes [page tokens][head dim] and one f32 scale
for each block of 16 tokens; a cached value is code * scale.  A batch is S sequences; sequence s owns
rows q_start[s] .. q_start[s + 1] - 1 of the call, and has kv_len[s] cached tokens counting them."""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 16  # tokens that share a scale


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    a = dict(op="attention", heads=32, kv_heads=8, dim=128, page=64, rows=1, window=0)
    p = dict(op="append", heads=32, kv_heads=8, dim=128, page=64, rot=128, pairs="halves")
    r = dict(op="read", kv_heads=8, dim=128, page=64)
    lo = dict(op="adapters", dtype="float16")
    return [
        # one request a few tokens in: nothing but latency
        dict(a, name="attend_1x17", seqs=1, len_min=17, len_max=17),
        # one request with a long document in its cache
        dict(a, name="attend_1x32768", seqs=1, len_min=32768, len_max=32768),
        # the eight vectors of one mat-vec call, requests of all ages
        dict(a, name="attend_8_ragged", seqs=8, len_min=1, len_max=4099),
        # a served batch in full swing: the largest read of the cache
        dict(a, name="attend_48_ragged", seqs=48, len_min=2500, len_max=12301),
        # checking four drafted tokens of each request at once (16 rows share a key/value head)
        dict(a, name="attend_verify_4_rows", seqs=8, len_min=700, len_max=2900, rows=4, page=32),
        # small heads, seven to a key/value head, a sliding window, pages of one block
        dict(a, name="attend_64_wide_window", seqs=24, len_min=1, len_max=6000, heads=28, kv_heads=4, dim=64,
             page=16, window=1500),
        # one new token for each of eight requests
        dict(p, name="append_8x1", seqs=8, rows=1, len_min=3, len_max=4000),
        # prompts arriving beside requests that decode; interleaved pairs
        dict(p, name="append_prompts", seqs=6, rows=2777, len_min=0, len_max=900, pairs="adjacent"),
        # a request's cache read back, to be moved or kept
        dict(r, name="read_1x700", seqs=1, rows=700, len_min=0, len_max=0),
        dict(r, name="read_8x4000", seqs=8, rows=4000, len_min=5, len_max=70),
        # one request with a small adapter on the 4096 x 4096 output projection
        dict(lo, name="adapter_1_r8", batch=1, adapters=4, rank=8, K=4096, rows=4096),
        # eight requests, eight adapters (two share one, one has none) on the fused gate|up projection
        dict(lo, name="adapters_8_r64", batch=8, adapters=16, rank=64, K=4096, rows=28672, dtype="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "read", "adapters"])
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (16, 16), (64, 8), (9, 3), (8, 1)])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "attention":
        seqs = _log_int(rng, 1, 64)
        # cached tokens x heads x dim at most those of the largest listed case
        most = min(32768, 48 * 7000 * 8 * 128 // (seqs * kv_heads * dim))
        len_max = _log_int(rng, 1, max(1, most))
        rows = rng.choice([1, 1, 1, 2, 3, 5, 8])
        if rows * heads * dim * len_max * seqs > 48 * 7000 * 32 * 128:
            rows = 1
        return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, rows=rows, seqs=seqs,
                    len_min=rng.randint(0, len_max), len_max=len_max, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]))
    if op == "append":
        rows, seqs = _log_int(rng, 1, 2700), _log_int(rng, 1, 32)
        seqs = max(1, min(seqs, 16000 * 40 * 128 // (rows * (heads + kv_heads) * dim)))
        return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, rows=rows, seqs=seqs, len_min=0,
                    len_max=_log_int(rng, 1, 4000), rot=rng.choice([dim, dim, dim // 2]),
                    pairs=rng.choice(["halves", "adjacent"]))
    if op == "read":
        rows, seqs = _log_int(rng, 1, 4000), _log_int(rng, 1, 32)
        seqs = max(1, min(seqs, 32000 * 8 * 128 // (rows * kv_heads * dim)))
        return dict(op=op, kv_heads=kv_heads, dim=dim, page=page, rows=rows, seqs=seqs, len_min=0,
                    len_max=_log_int(rng, 1, 500))
    return dict(op=op, batch=rng.randint(1, 8), adapters=_log_int(rng, 1, 32), rank=8 * _log_int(rng, 1, 8),
                K=256 * _log_int(rng, 1, 56), rows=_log_int(rng, 64, 28000), dtype=rng.choice(["float16", "bfloat16"]))


def _lengths(case):
    """(cached tokens before the call's rows, rows) of each sequence: part of the case, not of the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lo, hi, n = case["len_min"], case["len_max"], case["rows"]
    out = []
    for s in range(case["seqs"]):
        ln = hi if s == 0 else rng.randint(lo, hi)
        if case["op"] == "attention":
            out.append((ln, n))           # ln counts the rows; fewer tokens than rows leaves rows empty
        elif case["op"] == "append":
            k = n if s == 0 else rng.randint(max(1, n // 2), n)
            out.append((rng.randint(lo, hi) + k, k))
        else:
            out.append((rng.randint(lo, hi) + n, n))
    return out


def work(case):
    if case["op"] == "adapters":
        B, r, K, rows = case["batch"], case["rank"], case["K"], case["rows"]
        idx = _adapter_index(case)
        distinct = len({i for i in idx if i >= 0})
        live = sum(i >= 0 for i in idx)
        return {"bytes": distinct * r * (K + rows) * 2 + B * K * 4 + B * rows * 8, "flops": 2 * live * r * (K + rows)}
    H, D = case["kv_heads"], case["dim"]
    token = 2 * H * (D + 4 / BLOCK)  # codes and scales of K and V
    lens = _lengths(case)
    T = sum(n for _, n in lens)
    if case["op"] == "attention":
        W, nbytes, pairs = case["window"], 0, 0
        for ln, n in lens:
            reach = [(max(0, e - W) if W else 0, max(0, e)) for e in range(ln - n + 1, ln + 1)]
            nbytes += (max(e for _, e in reach) - min(b for b, _ in reach)) * token
            pairs += sum(e - b for b, e in reach)
        return {"bytes": nbytes + 2 * T * case["heads"] * D * 4, "flops": 4 * pairs * case["heads"] * D}
    if case["op"] == "append":
        # q, k, v in; rotated q out; codes in the cache; the table's rows; then the touched blocks read back
        back = sum(ln - (ln - n) // BLOCK * BLOCK for ln, n in lens)
        return {"bytes": T * (2 * case["heads"] * D * 4 + 2 * H * D * 4 + token + case["rot"] * 4) +
                back * (token + 2 * H * D * 4), "flops": T * (case["heads"] + H) * case["rot"] * 3}
    return {"bytes": T * (token + 2 * H * D * 4), "flops": T * 2 * H * D}


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _adapter_index(case):
    """Which adapter each vector uses: different ones, two sharing one, and from four vectors on one with none."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    idx = [rng.randrange(case["adapters"]) for _ in range(case["batch"])]
    if case["batch"] > 1:
        idx[1] = idx[0]
    if case["batch"] > 3:
        idx[3] = -1
    return idx


def _filled(pages, H, page, D, g):
    """Codes and scales of normally distributed values with outlying channels, quantised block by block."""
    codes = torch.empty((pages, H, page, D), dtype=torch.int8, device=DEV)
    scale = torch.empty((pages, H, page // BLOCK), dtype=torch.float32, device=DEV)
    channel = 1 + 3 * (torch.rand(D, device=DEV, generator=g) < 0.04)
    step = max(1, (1 << 27) // (H * page * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn((n, H, page // BLOCK, BLOCK, D), device=DEV, generator=g) * channel
        d = x.abs().amax((-1, -2)) / 127
        codes[a:a + n] = (x / d[..., None, None]).round().clamp(-127, 127).to(torch.int8).view(n, H, page, D)
        scale[a:a + n] = d
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "adapters":
        B, n, r, K, rows = (case[k] for k in ("batch", "adapters", "rank", "K", "rows"))
        t = getattr(torch, case["dtype"])
        st["x"] = torch.randn((B, K), device=DEV, generator=g)
        st["base"] = torch.randn((B, rows), device=DEV, generator=g) * 4
        st["A"] = (torch.randn((n, r, K), device=DEV, generator=g) / math.sqrt(K)).to(t)
        st["B"] = (torch.randn((n, rows, r), device=DEV, generator=g) / math.sqrt(r)).to(t)
        st["scale"] = 0.5 + torch.rand(n, device=DEV, generator=g)
        st["adapter"] = torch.tensor(_adapter_index(case), dtype=torch.int32, device=DEV)
        st["out"] = torch.empty_like(st["base"])
        return st
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
    st["max_q"], st["T"] = max(n for _, n in lens), T
    st["k_codes"], st["k_scale"] = _filled(pages, H, page, D, g)
    st["v_codes"], st["v_scale"] = _filled(pages, H, page, D, g)
    if case["op"] == "append":
        Hq = case["heads"]
        # the three parts of one fused projection's output: rows of (Hq + 2 H) D values
        qkv = torch.randn((T, (Hq + 2 * H) * D), device=DEV, generator=g)
        st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        st["k"] = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        st["v"] = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
        top, half = max(ln for ln, _ in lens), case["rot"] // 2
        f = 500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * f
        st["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()  # [positions][cosines, sines]
        st["q_out"] = torch.empty((T, Hq, D), device=DEV)
        # what is read back after the append: the rows of every block that it touched
        back = [ln - (ln - n) // BLOCK * BLOCK for ln, n in lens]
        bs = [0]
        for n in back:
            bs.append(bs[-1] + n)
        st["back_start"], st["back_max"], st["back_T"] = i32(bs), max(back), bs[-1]
        st["k_out"] = torch.empty((bs[-1], H, D), device=DEV)
        st["v_out"] = torch.empty((bs[-1], H, D), device=DEV)
    elif case["op"] == "attention":
        st["q"] = torch.randn((T, case["heads"], D), device=DEV, generator=g) * 1.5
        st["out"] = torch.empty((T, case["heads"] * D), device=DEV)
    else:
        st["k_out"] = torch.empty((T, H, D), device=DEV)
        st["v_out"] = torch.empty((T, H, D), device=DEV)
    if own:
        import quantised_decode_mat_gb300 as qmd
        st["cache"] = qmd.KVCache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
        st["batch"] = qmd.KVBatch(st["table"], st["kv_len"], st["q_start"], st["max_q"], T)
        if case["op"] == "append":
            st["back"] = qmd.KVBatch(st["table"], st["kv_len"], st["back_start"], st["back_max"], st["back_T"])
        if case["op"] == "attention":
            st["workspace"] = qmd.kv_workspace()
    return st


# ---- the operators, plainly --------------------------------------------------------------------

def _rows(st, q_start, T):
    """Sequence, position and first position of each of T rows."""
    row = torch.arange(T, device=DEV)
    s = torch.searchsorted(q_start[1:].long(), row, right=True)
    start = st["kv_len"].long()[s] - (q_start[1:] - q_start[:-1]).long()[s]
    return s, start + row - q_start.long()[s], start


def _place(st, s, pos):
    """Page, token in the page and block in the page of positions of sequences."""
    page = st["case"]["page"]
    col = (pos // page).clamp(0, st["table"].shape[1] - 1)
    return st["table"].long()[s, col], pos % page, pos % page // BLOCK


def _rotate(x, rope, pos, rot, pairs):
    c, s = rope[pos, None, :rot // 2], rope[pos, None, rot // 2:]
    y = x.clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _codes(x, d):
    inv = torch.where(d > 0, torch.ones_like(d) / d, torch.zeros_like(d))[..., None]
    return (x * inv).round().clamp(-127, 127).to(torch.int8)


def _store(st, codes, scale, x, s, pos, start):
    page, tok, blk = _place(st, s, pos)
    amax = x.abs().amax(-1)
    d_row = torch.where(amax < 1e-30, torch.zeros_like(amax), amax / torch.full_like(amax, 127))  # by a tensor: a true division
    most = torch.zeros_like(scale).transpose(1, 2).flatten(0, 1)  # [page, block][head]: the new rows' scale
    nb = scale.shape[2]
    most.scatter_reduce_(0, (page * nb + blk)[:, None].expand_as(d_row), d_row, "amax")
    # the tokens that the first touched block of each sequence held before
    seq = torch.arange(len(st["kv_len"]), device=DEV)
    n = (st["q_start"][1:] - st["q_start"][:-1]).long()
    first = st["kv_len"].long() - n
    old = first // BLOCK * BLOCK
    p0, _, b0 = _place(st, seq, old)
    d_old = torch.where((first > old)[:, None], scale[p0, :, b0], 0.0)
    d_new = torch.maximum(d_old, most[p0 * nb + b0])
    j = torch.arange(BLOCK, device=DEV)
    page_j, tok_j, _ = _place(st, seq[:, None], old[:, None] + j)
    held = codes[page_j, :, tok_j]  # [sequence][token][head][dim]
    again = _codes(held.float() * d_old[:, None, :, None], d_new[:, None].expand(-1, BLOCK, -1))
    grown = (d_new > d_old)[:, None, :, None] & (old[:, None] + j < first[:, None])[..., None, None] & (n > 0)[:, None, None, None]
    codes[page_j, :, tok_j] = torch.where(grown, again, held)
    begun = (pos // BLOCK * BLOCK >= start)[:, None]  # the block starts within the new rows
    d = torch.maximum(torch.where(begun, 0.0, scale[page, :, blk]), most[page * nb + blk])
    codes[page, :, tok] = _codes(x, d)
    scale[page, :, blk] = d


def _values(codes, scale, page, tok, blk):
    return codes[page, :, tok].float() * scale[page, :, blk][..., None]


def _plain_read(st, q_start, T):
    s, pos, _ = _rows(st, q_start, T)
    at = _place(st, s, pos)
    return _values(st["k_codes"], st["k_scale"], *at), _values(st["v_codes"], st["v_scale"], *at)


def _plain_append(st):
    case = st["case"]
    s, pos, start = _rows(st, st["q_start"], st["T"])
    q = _rotate(st["q"], st["rope"], pos, case["rot"], case["pairs"])
    k = _rotate(st["k"], st["rope"], pos, case["rot"], case["pairs"])
    _store(st, st["k_codes"], st["k_scale"], k, s, pos, start)
    _store(st, st["v_codes"], st["v_scale"], st["v"], s, pos, start)
    return q


def _plain_attention(st):
    case = st["case"]
    H, D, n = case["kv_heads"], case["dim"], st["max_q"]
    G = case["heads"] // H
    L, S = st["table"].shape[1] * case["page"], len(st["kv_len"])

    def cached(codes, scale):  # [sequence][head][token][dim]
        c = codes[st["table"].long()].float().unflatten(3, (-1, BLOCK)) * scale[st["table"].long()][..., None, None]
        return c.transpose(1, 2).reshape(S, H, L, D)

    i = torch.arange(n, device=DEV)
    rows = (st["q_start"][1:] - st["q_start"][:-1]).long()
    at = (st["q_start"][:-1].long()[:, None] + i).clamp(max=st["T"] - 1)
    q = st["q"][at].unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).reshape(S, H, n * G, D)
    last = st["kv_len"].long()[:, None] - rows[:, None] + i  # the newest key that a row sees
    j = torch.arange(L, device=DEV)
    sees = j <= last[..., None]
    if case["window"]:
        sees &= j > last[..., None] - case["window"]
    sees = sees[:, None, :, None].expand(S, 1, n, G, L).reshape(S, 1, n * G, L)
    score = q @ cached(st["k_codes"], st["k_scale"]).transpose(2, 3) * (1 / math.sqrt(D))
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(sees, (score - torch.where(top.isinf(), 0.0, top)).exp(), 0.0)
    o = p @ cached(st["v_codes"], st["v_scale"])
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0).unflatten(2, (n, G)).permute(0, 2, 1, 3, 4).reshape(S, n, -1)
    seq, _, _ = _rows(st, st["q_start"], st["T"])
    return o[seq, torch.arange(st["T"], device=DEV) - st["q_start"].long()[seq]]


def _plain_adapters(st):
    a = st["adapter"].long()
    x, has = st["x"], (a >= 0)[:, None]
    a = a.clamp(min=0)
    t = st["A"][a].float() @ x[:, :, None]
    delta = (st["B"][a].float() @ t)[..., 0] * st["scale"][a][:, None]
    return torch.where(has, st["base"] + delta, st["base"])


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import quantised_decode_mat_gb300 as qmd
        if op == "adapters":
            return qmd.lora_add(st["x"], st["base"], st["A"], st["B"], st["adapter"], st["scale"], out=st["out"])
        if op == "read":
            return qmd.kv_read(st["cache"], st["batch"], st["k_out"], st["v_out"])
        if op == "append":
            q = qmd.kv_append(st["cache"], st["batch"], st["k"], st["v"], rope=st["rope"], q=st["q"], q_out=st["q_out"],
                              pairs=qmd.ROPE_HALVES if st["case"]["pairs"] == "halves" else qmd.ROPE_ADJACENT)
            return (q,) + tuple(qmd.kv_read(st["cache"], st["back"], st["k_out"], st["v_out"]))
        return qmd.kv_attention(st["cache"], st["batch"], st["q"], 1 / math.sqrt(st["case"]["dim"]), st["workspace"],
                                window=st["case"]["window"], out=st["out"])
    if op == "adapters":
        return _plain_adapters(st)
    if op == "read":
        return _plain_read(st, st["q_start"], st["T"])
    if op == "append":
        q = _plain_append(st)
        return (q,) + _plain_read(st, st["back_start"], st["back_T"])
    return _plain_attention(st)


# ---- the definitions, in 64 bits ---------------------------------------------------------------

def _r32(x):
    """x rounded to 32 bits: the append is defined with every operation rounded so (the codes hang on it)."""
    return x.float().double()


def _exact_append(st):
    case = st["case"]
    H, D, page, half = case["kv_heads"], case["dim"], case["page"], case["rot"] // 2
    q_out, k_out, v_out = [], [], []
    for s, (ln, n) in enumerate(_lengths(case)):
        r0 = int(st["q_start"][s])
        c, sn = st["rope"][ln - n:ln].double()[:, None].chunk(2, -1)
        rotated = {}
        for name in ("q", "k"):
            x = st[name][r0:r0 + n].double()
            y = x.clone()
            halves = case["pairs"] == "halves"
            lo = torch.arange(half, device=DEV) * (1 if halves else 2)
            hi = lo + (half if halves else 1)
            y[:, :, lo] = _r32(_r32(x[:, :, lo] * c) - _r32(x[:, :, hi] * sn))
            y[:, :, hi] = _r32(_r32(x[:, :, hi] * c) + _r32(x[:, :, lo] * sn))
            rotated[name] = y
        q_out.append(rotated["q"])
        first = (ln - n) // BLOCK * BLOCK
        where = [(int(st["table"][s, p // page]), p % page) for p in range(first, ln)]
        pg = torch.tensor([w[0] for w in where], device=DEV)
        tk = torch.tensor([w[1] for w in where], device=DEV)
        for x, codes, scale, out in ((rotated["k"], st["k_codes"], st["k_scale"], k_out),
                                     (st["v"][r0:r0 + n].double(), st["v_codes"], st["v_scale"], v_out)):
            m = ln - n - first  # tokens that the first block held
            old_d = scale[pg[0], :, tk[0] // BLOCK].double() if m else torch.zeros(H, device=DEV, dtype=torch.float64)
            top = x.abs().amax(2)
            d_row = torch.where(top < 1e-30, 0.0, _r32(top / 127))
            all_d = torch.cat((old_d.expand(m, H), d_row))
            pad = -len(all_d) % BLOCK
            d = torch.nn.functional.pad(all_d, (0, 0, 0, pad)).unflatten(0, (-1, BLOCK)).amax(1).repeat_interleave(BLOCK, 0)[:len(all_d)]
            d = d[..., None]
            held = codes[pg[:m], :, tk[:m]].double()
            inv = torch.where(d > 0, _r32(1 / d), 0.0)
            new = _r32(torch.cat((_r32(held * old_d[:, None]), x)) * inv).round().clamp(-127, 127)
            new[:m] = torch.where(d[:m] > old_d[:, None], new[:m], held)
            out.append(new * d)
    return torch.cat(q_out), torch.cat(k_out), torch.cat(v_out)


def _sequence(st, s, lo, hi):
    """Keys and values lo .. hi - 1 of sequence s, in 64 bits: [token][head][dim]."""
    page = st["case"]["page"]
    p = torch.arange(lo, hi, device=DEV)
    at = st["table"][s].long()[p // page]
    tok = p % page
    return [c[at, :, tok].double() * d[at, :, tok // BLOCK].double()[..., None]
            for c, d in ((st["k_codes"], st["k_scale"]), (st["v_codes"], st["v_scale"]))]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "adapters":
        rows = []
        for v, a in enumerate(_adapter_index(case)):
            y = st["base"][v].double()
            if a >= 0:
                y = y + st["scale"][a].double() * (st["B"][a].double() @ (st["A"][a].double() @ st["x"][v].double()))
            rows.append(y)
        return torch.stack(rows)
    lens = _lengths(case)
    if case["op"] == "read":
        got = [_sequence(st, s, ln - n, ln) for s, (ln, n) in enumerate(lens)]
        return torch.cat([k for k, _ in got]), torch.cat([v for _, v in got])
    G = case["heads"] // case["kv_heads"]
    out = []
    for s, (ln, n) in enumerate(lens):
        k, v = _sequence(st, s, 0, ln)
        q = st["q"][int(st["q_start"][s]):int(st["q_start"][s]) + n].double()
        for i in range(n):
            end = ln - n + 1 + i
            begin = max(0, end - case["window"]) if case["window"] else 0
            if end <= begin:
                out.append(torch.zeros(case["heads"] * case["dim"], device=DEV, dtype=torch.float64))
                continue
            qi = q[i].unflatten(0, (case["kv_heads"], G))
            w = torch.softmax(torch.einsum("hgd,lhd->hgl", qi, k[begin:end]) / math.sqrt(case["dim"]), -1)
            out.append(torch.einsum("hgl,lhd->hgd", w, v[begin:end]).reshape(-1))
    return torch.stack(out)
