"""Cases of the paged K+V cache operators: appending rotated keys and values to pages held in bf16 or in
8 bits (e4m3 with one power-of-two scale for each page and head), attention over those pages for single
tokens and for several queries of a sequence, and reading rows back.

A cache is kpages, vpages [num_pages][Hkv][page][dh], for e4m3 kscale, vscale [num_pages][Hkv] in fp32, and
table [B][max_pages]: row t of sequence b lies in page table[b][t // page] at row t % page. Rows of several
sequences come packed: sequence b owns rows starts[b] .. starts[b + 1] - 1.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def _case(name, op, kind, B, heads, page, cached, new, rot=0, interleaved=False, mix=1):
    Hq, Hkv, dh = heads
    return {"name": name, "op": op, "kind": kind, "B": B, "Hq": Hq, "Hkv": Hkv, "dh": dh, "page": page,
            "cached_lo": cached[0], "cached_hi": cached[1], "new_lo": new[0], "new_hi": new[1], "rot": rot,
            "interleaved": interleaved, "mix": mix}


def listed():
    return [
        # one generation step of d=1024 H=16 B=8 T=4096: a token for each sequence
        _case("append_token_bf16", "append", "bf16", 8, (16, 16, 64), 64, (4096, 4096), (1, 1), 64),
        # one generation step of a server's batch with grouped heads, ragged lengths, small pages
        _case("append_token_e4m3", "append", "e4m3", 64, (32, 8, 128), 16, (100, 4000), (1, 1), 128),
        # new prompts of several sequences, half of each head rotated, in neighbouring pairs
        _case("append_prompt_bf16", "append", "bf16", 4, (16, 16, 64), 32, (0, 0), (700, 4096), 32, True),
        # prompts and later chunks together: pages that begin and end inside a chunk
        _case("append_prompt_e4m3", "append", "e4m3", 5, (32, 8, 128), 64, (0, 3000), (1, 6000), 128),
        # the 128-token prompt and 16 steps of d=256 H=4, read back for a check
        _case("gather_bf16_small", "gather", "bf16", 1, (4, 4, 64), 16, (0, 0), (144, 144)),
        # sequences taken out of the cache, to be kept elsewhere
        _case("gather_e4m3", "gather", "e4m3", 16, (32, 8, 128), 64, (0, 77), (1000, 6000)),
        # the step of d=256 H=4 after its 128-token prompt: latency
        _case("decode_bf16_one", "decode", "bf16", 1, (4, 4, 64), 16, (143, 143), (1, 1)),
        # the step of d=1024 H=16 B=8 T=4096
        _case("decode_bf16", "decode", "bf16", 8, (16, 16, 64), 64, (4096, 4096), (1, 1)),
        # 32 heads of 128 over 8 shared ones, 16 ragged sequences of 16K to 32K
        _case("decode_e4m3_long", "decode", "e4m3", 16, (32, 8, 128), 64, (16384, 32768), (1, 1)),
        # a whole prompt of 8192 tokens, d=4096 H=32
        _case("prefill_bf16_prompt", "prefill", "bf16", 1, (32, 32, 128), 128, (0, 0), (8192, 8192)),
        # chunks of four prompts behind 16K cached rows
        _case("prefill_e4m3_chunk", "prefill", "e4m3", 4, (32, 8, 128), 64, (16000, 16384), (300, 512)),
        # a few proposed tokens of each sequence verified at once, d=1280 H=20
        _case("prefill_e4m3_few", "prefill", "e4m3", 64, (20, 20, 64), 32, (1000, 1500), (2, 5)),
    ]


_HEADS = [(16, 16, 64), (20, 20, 64), (32, 32, 128), (32, 8, 128), (24, 4, 64), (16, 2, 128), (7, 1, 64),
          (40, 8, 128), (4, 4, 64)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "gather"])
    kind = rng.choice(["bf16", "e4m3"])
    heads = rng.choice(_HEADS)
    Hq, Hkv, dh = heads
    page = rng.choice([16, 32, 64, 128])
    rot = rng.choice([dh, dh // 2, 0]) if op == "append" else 0
    style = rng.random() < 0.3
    width = Hkv * dh
    if op == "decode":
        B = _log(rng, 1, 64)
        hi = min(_log(rng, 1, 32768), max(1, (128 << 20) // (B * width)))
        return _case("", op, kind, B, heads, page, (rng.randint(0, hi), hi), (1, 1), mix=rng.randint(1, 999))
    if op == "prefill":
        B = _log(rng, 1, 16)
        n = _log(rng, 1, 4096)
        L = _log(rng, 1, 16384) - 1
        while B * Hq * n * (n + L) > 32 * 8192 * 8192 or B * (n + L) * width > (128 << 20):
            B, n, L = max(1, B // 2), max(1, n * 3 // 4), L * 3 // 4
        return _case("", op, kind, B, heads, page, (rng.randint(0, L), L), (rng.randint(0, n), n), mix=rng.randint(1, 999))
    if op == "append" and rng.random() < 0.4:
        B, n = _log(rng, 1, 128), 1
        lo = 1
    else:
        B = _log(rng, 1, 16)
        n = max(2, min(_log(rng, 2, 8192), (16 << 20) // (B * width)))
        lo = rng.randint(1, n)
    L = min(_log(rng, 1, 4096) - 1, max(0, (48 << 20) // (B * width) - n))
    return _case("", op, kind, B, heads, page, (rng.randint(0, L), L), (lo, n), rot, style, mix=rng.randint(1, 999))


def _lengths(c):
    """Cached rows and new rows of each sequence, from the case alone."""
    r = random.Random(c["mix"])
    cached = [r.randint(c["cached_lo"], c["cached_hi"]) for _ in range(c["B"])]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    new[-1] = c["new_hi"]
    return cached, new


# ------------------------------------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def _pool(g, num_pages, Hkv, page, dh, kind, spread):
    """Pages of keys or values in use, and their scales: normal values, heads of different magnitude."""
    mag = torch.exp(torch.randn(1, Hkv, 1, 1, generator=g, device=DEV) * spread)
    x = torch.empty(num_pages, Hkv, page, dh, dtype=torch.bfloat16, device=DEV).normal_(generator=g) * mag.bfloat16()
    if kind == "bf16":
        return x, None
    amax = x.abs().amax(dim=(2, 3)).float()
    scale = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(-100, 120))
    return (x / scale.bfloat16()[:, :, None, None]).float().clamp(-448, 448).to(E4M3), scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    cached, new = _lengths(c)
    B, Hq, Hkv, dh, page = c["B"], c["Hq"], c["Hkv"], c["dh"], c["page"]
    need = [-(-(a + n) // page) for a, n in zip(cached, new)]
    width = max(need) + 1
    num_pages = sum(need) + 3
    # pages in the order in which a pool hands them out after some use; -1 where a sequence has none
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32).tolist()
    rows = []
    for k in need:
        rows.append([order.pop() for _ in range(k)] + [-1] * (width - k))
    s = {"case": c, "B": B, "Hq": Hq, "Hkv": Hkv, "dh": dh, "page": page, "max_new": max(new), "table": _i32(rows),
         "lens": _i32(cached), "starts": _i32(_starts(new)), "rows": sum(new), "max_len": max(a + n for a, n in zip(cached, new)),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    s["kpages"], s["kscale"] = _pool(g, num_pages, Hkv, page, dh, c["kind"], 0.3)
    s["vpages"], s["vscale"] = _pool(g, num_pages, Hkv, page, dh, c["kind"], 0.5)
    R = s["rows"]
    if c["op"] == "append":
        # k and v as one projection's output holds them, row by row
        kv = torch.randn(R, 2 * Hkv, dh, generator=g, device=DEV).bfloat16()
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        s["q"] = torch.randn(R, Hq, dh, generator=g, device=DEV).bfloat16()
        s["q_out"] = torch.zeros(R, Hq, dh, dtype=torch.bfloat16, device=DEV)
        if c["rot"]:
            f = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
            a = torch.arange(width * page, dtype=torch.float64, device=DEV)[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        else:
            s["cos"] = s["sin"] = None
        if c["kind"] == "e4m3":
            # 8-bit rows are read back from the first page that a sequence touches: older rows of it may change
            first = [a // page * page for a in cached]
            back = [a + n - f for a, n, f in zip(cached, new, first)]
            s["first"], s["back"], s["back_rows"], s["max_back"] = _i32(first), _i32(_starts(back)), sum(back), max(back)
    elif c["op"] == "decode":
        s["q"] = (2 * torch.randn(B, Hq, dh, generator=g, device=DEV)).bfloat16()
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "prefill":
        s["q"] = (2 * torch.randn(R, Hq, dh, generator=g, device=DEV)).bfloat16()
        s["out"] = torch.zeros_like(s["q"])
    else:
        s["first"], s["back"], s["back_rows"], s["max_back"] = s["lens"], s["starts"], R, s["max_new"]
    if "back_rows" in s:
        s["k_back"] = torch.zeros(s["back_rows"], Hkv, dh, dtype=torch.bfloat16, device=DEV)
        s["v_back"] = torch.zeros_like(s["k_back"])
    if own:
        from only_cache_exact_b200 import slim
        s["slim"] = slim
        s["cache"] = slim.PagedKV(s["kpages"], s["vpages"], s["table"], s["kscale"], s["vscale"])
        if c["op"] == "decode":
            s["ws"] = slim.alloc_paged_decode_workspace(s["cache"], Hq)
        if c["op"] == "prefill":
            s["ws"] = slim.alloc_paged_prefill_workspace(s["cache"], Hq, R, s["max_new"], s["max_len"])
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _rotate(x, pos, s):
    """x [rows][heads][dh] with its first `rot` columns rotated by the angles of `pos`, in 64 bits."""
    x = x.double()
    rot = s["case"]["rot"]
    if rot == 0:
        return x
    c, n = s["cos"].double()[pos][:, None], s["sin"].double()[pos][:, None]
    y = x.clone()
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * n, b * c + a * n
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * n, b * c + a * n
    return y


def _where(starts, first, rows):
    """For each of `rows` packed rows: its sequence and its position, first[b] + its number in the sequence."""
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(starts.long(), r, right=True) - 1
    return b, first.long()[b] + r - starts.long()[b]


def _read(s, which, b, pos):
    """Rows `pos` of sequences `b` of the cache in fp32, [..., Hkv, dh]."""
    pages, scale = s[which + "pages"], s[which + "scale"]
    at = s["table"].long()[b, pos // s["page"]].clamp(min=0)
    x = pages[at, :, pos % s["page"]].float()
    return x if scale is None else x * scale[at].unsqueeze(-1)


def _store(s, which, x, b, pos):
    """Rows x [rows][Hkv][dh] written to the cache, in 8 bits with the pages' scales brought up to date."""
    pages, scale, page = s[which + "pages"], s[which + "scale"], s["page"]
    if scale is None:
        pages[s["table"].long()[b, pos // page], :, pos % page] = x.bfloat16()
        return
    lens, n = s["lens"].long(), s["starts"].long().diff()
    slots = (s["max_new"] + 2 * page - 2) // page  # pages that a sequence can touch
    j = torch.arange(slots, device=DEV)
    last = (lens + n - 1) // page
    at_page = torch.minimum(lens[:, None] // page + j, last[:, None])  # a slot too many repeats the last page
    at = torch.gather(s["table"].long(), 1, at_page)
    block = pages[at].double() * scale[at].double()[..., None, None]  # [B][slots][Hkv][page][dh]
    row = torch.arange(page, device=DEV)
    t = at_page[..., None] * page + row
    is_new = (t >= lens[:, None, None]) & (t < (lens + n)[:, None, None])
    src = (s["starts"].long()[:-1, None, None] + t - lens[:, None, None]).clamp(0, x.shape[0] - 1)
    block = torch.where(is_new[:, :, None, :, None], x[src].transpose(2, 3), block)
    amax = torch.where(is_new[:, :, None, :, None], block.abs(), 0.0).amax(dim=(3, 4))
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), -100).clamp(-100, 120)
    need = torch.exp2(e.double())
    begins = (at_page * page >= lens[:, None])[..., None]
    to = torch.where(begins, need, torch.maximum(need, scale[at].double()))
    pages[at] = (block / to[..., None, None]).clamp(-448, 448).float().to(E4M3)
    scale[at] = to.float()


def _attend(q, K, V, live):
    """q [B][Hkv][m][dh], K, V [B][Hkv][T][dh], live [B][1][m][T]: softmax(q K^T / sqrt(dh)) V in fp32, zero where nothing is live."""
    z = torch.matmul(q * (1.0 / math.sqrt(q.shape[-1])), K.transpose(-1, -2))
    z = torch.where(live, z, -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    return torch.matmul(p, V) / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)


def _dense(s, T, lens):
    """The first T rows of all sequences, [B][Hkv][T][dh] in fp32; rows behind a sequence's length are zero."""
    b = torch.arange(s["B"], device=DEV)[:, None]
    t = torch.arange(T, device=DEV)[None]
    inside = (t < lens.long()[:, None])[..., None, None]
    return [torch.where(inside, _read(s, w, b, t.expand(s["B"], T)), 0.0).transpose(1, 2) for w in ("k", "v")]


def _plain(s):
    op, Hkv, dh = s["case"]["op"], s["Hkv"], s["dh"]
    G = s["Hq"] // Hkv
    if op == "append":
        b, pos = _where(s["starts"], s["lens"], s["rows"])
        _store(s, "k", _rotate(s["k"], pos, s), b, pos)
        _store(s, "v", s["v"].double(), b, pos)
        q = _rotate(s["q"], pos, s).bfloat16()
        if s["kscale"] is None:
            return {"q": q, "k": s["kpages"], "v": s["vpages"]}
        return {"q": q, **_plain_back(s)}
    if op == "gather":
        return _plain_back(s)
    if op == "decode":
        lens = s["lens"] + 1
        K, V = _dense(s, s["max_len"], lens)
        live = (torch.arange(s["max_len"], device=DEV)[None] < lens[:, None])[:, None, None]
        o = _attend(s["q"].float().view(s["B"], Hkv, G, dh), K, V, live)
        return {"out": o.reshape(s["B"], s["Hq"], dh).bfloat16()}
    n = s["max_new"]
    K, V = _dense(s, s["max_len"], s["lens"] + s["starts"].diff())
    j = torch.arange(n, device=DEV)
    at = (s["starts"].long()[:-1, None] + j).clamp(max=s["rows"] - 1)  # [B][n]
    q = s["q"].float()[at].view(s["B"], n, Hkv, G, dh).permute(0, 2, 1, 3, 4).reshape(s["B"], Hkv, n * G, dh)
    live = torch.arange(s["max_len"], device=DEV)[None, None] <= s["lens"].long()[:, None, None] + j[:, None]
    live = live[:, :, None].expand(-1, -1, G, -1).reshape(s["B"], 1, n * G, -1)
    o = _attend(q, K, V, live).view(s["B"], Hkv, n, G, dh).permute(0, 2, 1, 3, 4).reshape(s["B"], n, s["Hq"], dh)
    b, pos = _where(s["starts"], torch.zeros_like(s["lens"]), s["rows"])
    return {"out": o[b, pos].bfloat16()}


def _plain_back(s):
    b, pos = _where(s["back"], s["first"], s["back_rows"])
    return {"k": _read(s, "k", b, pos).bfloat16(), "v": _read(s, "v", b, pos).bfloat16()}


# ------------------------------------------------------------------------------------------------ the framework's
def _own(s):
    S, c, op = s["slim"], s["cache"], s["case"]["op"]
    if op == "append":
        S.slim_mha_paged_append(c, s["k"], s["v"], s["starts"], s["lens"], s["status"], q=s["q"], q_out=s["q_out"],
                                cos=s["cos"], sin=s["sin"], interleaved=s["case"]["interleaved"], max_new=s["max_new"])
        if s["kscale"] is None:
            return {"q": s["q_out"], "k": s["kpages"], "v": s["vpages"]}
        S.slim_mha_paged_gather(c, s["first"], s["back"], s["k_back"], s["v_back"], s["status"], max_new=s["max_back"])
        return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}
    if op == "gather":
        S.slim_mha_paged_gather(c, s["first"], s["back"], s["k_back"], s["v_back"], s["status"], max_new=s["max_back"])
        return {"k": s["k_back"], "v": s["v_back"]}
    if op == "decode":
        S.slim_mha_paged_decode(c, s["q"], s["lens"], s["out"], s["ws"], s["status"], rows_extra=1, t_hint=s["max_len"])
    else:
        S.slim_mha_paged_prefill(c, s["q"], s["starts"], s["lens"], s["out"], s["ws"], s["status"], max_new=s["max_new"],
                                 t_hint=s["max_len"])
    return {"out": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    cached, new = _lengths(c)
    es = 2 if c["kind"] == "bf16" else 1
    Hq, Hkv, dh, page = c["Hq"], c["Hkv"], c["dh"], c["page"]
    w = Hkv * dh
    R = sum(new)
    pages = sum(-(-(a + n) // page) - (a // page if c["op"] in ("append", "gather") else 0) for a, n in zip(cached, new))
    meta = 4 * pages + 4 * (2 * c["B"] + 1) + (8 * Hkv * pages if es == 1 else 0)
    if c["op"] == "append":
        seen = set()
        for a, n in zip(cached, new):
            seen.update(range(a, a + n))
        moved = R * w * 2 * 2 + R * w * es * 2 + R * Hq * dh * 4 + len(seen) * c["rot"] * 4
        if es == 1:  # the rows read back
            back = sum(a % page + n for a, n in zip(cached, new))
            moved += back * w * 2 * (1 + 2)
        return {"bytes": moved + meta, "flops": 3.0 * R * (Hq + Hkv) * c["rot"]}
    if c["op"] == "gather":
        return {"bytes": R * w * 2 * (es + 2) + meta, "flops": 0}
    keys = sum(a + n for a, n in zip(cached, new))
    rows = c["B"] if c["op"] == "decode" else R
    pairs = keys if c["op"] == "decode" else sum(n * a + n * (n + 1) // 2 for a, n in zip(cached, new))
    return {"bytes": keys * w * 2 * es + rows * Hq * dh * 4 + meta, "flops": 4.0 * pairs * Hq * dh}


# ------------------------------------------------------------------------------------------------ 64 bits
def _code_values():
    """The value of each of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits, one NaN for each sign."""
    v = []
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if i & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _grid(x):
    """x rounded to the nearest value of the e4m3 grid, ties to the even one."""
    ulp = torch.exp2((torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3))
    return torch.round(x / ulp) * ulp


def _values(s, which):
    pages, scale = s[which + "pages"], s[which + "scale"]
    if scale is None:
        return lambda ids: pages[ids].double()
    codes = _code_values()
    return lambda ids: codes[pages[ids].view(torch.uint8).long()] * scale[ids].double()[:, :, None, None]


def _turn(x, pos, s):
    """Rotation as a product of complex numbers."""
    rot = s["case"]["rot"]
    x = x.double()
    if rot == 0:
        return x
    w = torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
    h = x[..., :rot]
    pairs = h.unflatten(-1, (rot // 2, 2)) if s["case"]["interleaved"] else h.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    z = z.flatten(-2) if s["case"]["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:]], dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    cached, new = _lengths(case)
    table, page, Hkv, dh = s["table"].tolist(), s["page"], s["Hkv"], s["dh"]
    first = _starts(new)
    ids = [torch.tensor(t[:-(-(a + n) // page)], device=DEV, dtype=torch.long) for t, a, n in zip(table, cached, new)]
    op, e4m3 = case["op"], case["kind"] == "e4m3"

    def sequence(which, b):  # [T][Hkv][dh]
        return _values(s, which)(ids[b]).transpose(1, 2).reshape(-1, Hkv, dh)

    if op == "gather":
        return {w: torch.cat([sequence(w, b)[a:a + n] for b, (a, n) in enumerate(zip(cached, new))]) for w in ("k", "v")}
    if op == "append":
        out = {"q": torch.empty(s["rows"], s["Hq"], dh, dtype=torch.float64, device=DEV)}
        full = {w: s[w + "pages"].double() for w in ("k", "v")} if not e4m3 else {"k": [], "v": []}
        for b, (a, n) in enumerate(zip(cached, new)):
            r = slice(first[b], first[b] + n)
            pos = torch.arange(a, a + n, device=DEV)
            out["q"][r] = _turn(s["q"][r], pos, s)
            for w in ("k", "v"):
                x = _turn(s["k"][r], pos, s) if w == "k" else s["v"][r].double()
                if not e4m3:
                    full[w][ids[b][pos // page], :, pos % page] = x
                    continue
                p0 = a // page
                old = _values(s, w)(ids[b][p0:]).transpose(1, 2).reshape(-1, Hkv, dh)
                old_scale = s[w + "scale"][ids[b][p0:]].double()
                k = len(ids[b]) - p0
                lead = a - p0 * page
                new_rows = torch.zeros_like(old)
                new_rows[lead:lead + n] = x
                amax = new_rows.view(k, page, Hkv, dh).abs().amax(dim=(1, 3))
                up = torch.ceil(torch.log2(amax / 448).clamp(-100, 120))
                sc = torch.exp2(up)
                if lead:
                    sc[0] = torch.maximum(sc[0], old_scale[0])
                    new_rows[:lead] = old[:lead]
                each = sc[:, None, :, None]
                full[w].append((_grid(new_rows.view(k, page, Hkv, dh) / each) * each).reshape(-1, Hkv, dh)[:lead + n])
        for w in ("k", "v"):
            out[w] = torch.cat(full[w]) if e4m3 else full[w]
        return out
    G = s["Hq"] // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (a, n) in enumerate(zip(cached, new)):
        K, V = sequence("k", b), sequence("v", b)
        for h in range(Hkv):
            r = slice(b, b + 1) if op == "decode" else slice(first[b], first[b] + n)
            q = s["q"][r, h * G:(h + 1) * G].double()  # [m][G][dh]
            m = q.shape[0]
            z = torch.einsum("mgd,td->mgt", q, K[:a + n, h]) / math.sqrt(dh)
            seen = torch.arange(a + n, device=DEV)[None] <= a + torch.arange(m, device=DEV)[:, None]
            z.masked_fill_(~seen[:, None], -math.inf)
            out[r, h * G:(h + 1) * G] = torch.softmax(z, dim=-1) @ V[:a + n, h] if m else out[r, h * G:(h + 1) * G]
    return {"out": out}
