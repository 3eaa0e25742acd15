"""The paged 4-bit KV cache's operators: what is measured, and their plain forms.

Four operators of a batched decoding stage, which a serving loop calls one after another:

  plan       block tables and slot maps from request lengths
  append     K and V rows quantised to 4 bits and written to their slots (then read back: a cache of
             4 bits is returned as the values it stands for)
  read       the rows at some slots as values
  attention  softmax(q k^T / sqrt(D)) v over the pages, causal, one or more query tokens per sequence

The cache: pages of `page` positions, a tensor of bytes [page][kv head][tile of 16 positions][bytes of a tile], each
tile K codes, K scales, V codes, V scales.  A block of 32 dims has one fp16 scale s; a code c of 4 bits stands for s * (c - 8).
K codes of a tile: [position 16][dim / 8 % 4][block][4 bytes], the low nibble the lower dim.
V codes of a tile: [position / 8][dim / 4 % 8][position / 2 % 4][position % 2][block][2 bytes].
Scales: [position 16][block].
"""
import math
import random

import torch

own = False

SCRATCH = 64 << 20  # bytes of the attention's scratch, kept by the program (zero at the start)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 requests, each one token further
        {"name": "plan decode 64", "op": "plan", "kind": "decode", "seqs": 64, "page": 64, "len_max": 4096, "new_max": 1, "mix": 1},
        # a step of a busy server: finished requests leave, prompts enter, drafts are rolled back
        {"name": "plan mixed 1021", "op": "plan", "kind": "mixed", "seqs": 1021, "page": 16, "len_max": 8192, "new_max": 512, "mix": 2},
        # the K and V rows of a decode step of 64 sequences (the 70B shape's heads)
        {"name": "append decode 64", "op": "append", "tokens": 64, "run": 1, "hkv": 8, "hd": 128, "page": 64, "dtype": "f32", "mix": 3},
        # the rows of a prompt batch, some of them padding
        {"name": "append prompt 16411", "op": "append", "tokens": 16411, "run": 731, "hkv": 8, "hd": 128, "page": 64, "dtype": "bf16", "mix": 4},
        # a short prefix copied out of the cache
        {"name": "read prefix 100", "op": "read", "tokens": 100, "run": 100, "hkv": 4, "hd": 64, "page": 16, "dtype": "f32", "mix": 5},
        # a long context handed over to a 16-bit cache
        {"name": "read context 32768", "op": "read", "tokens": 32768, "run": 4096, "hkv": 8, "hd": 128, "page": 64, "dtype": "f16", "mix": 6},
        # the first tokens of one sequence: latency
        {"name": "attend one short", "op": "attention", "seqs": 1, "q_min": 1, "q_max": 1, "len_min": 17, "len_max": 17, "hq": 4, "hkv": 2, "hd": 64, "page": 16, "dtype": "f32", "mix": 7},
        # one sequence far into its context (the 8B shape's heads)
        {"name": "attend one long", "op": "attention", "seqs": 1, "q_min": 1, "q_max": 1, "len_min": 131001, "len_max": 131001, "hq": 32, "hkv": 8, "hd": 128, "page": 64, "dtype": "f32", "mix": 8},
        # the 70B shape's batched decode: 64 ragged sequences
        {"name": "attend ragged 64", "op": "attention", "seqs": 64, "q_min": 1, "q_max": 1, "len_min": 128, "len_max": 4096, "hq": 64, "hkv": 8, "hd": 128, "page": 64, "dtype": "f32", "mix": 9},
        # drafts of a few tokens verified at once, in 16 bits
        {"name": "attend drafts 16", "op": "attention", "seqs": 16, "q_min": 1, "q_max": 5, "len_min": 100, "len_max": 2000, "hq": 32, "hkv": 8, "hd": 128, "page": 32, "dtype": "bf16", "mix": 10},
        # the 8B shape's prefill: four prompts of 512 tokens in one step
        {"name": "attend prompts 4x512", "op": "attention", "seqs": 4, "q_min": 512, "q_max": 512, "len_min": 512, "len_max": 512, "hq": 32, "hkv": 8, "hd": 128, "page": 64, "dtype": "f32", "mix": 11},
        # chunks of long prompts, whose beginnings are in the cache
        {"name": "attend chunks 2x1024", "op": "attention", "seqs": 2, "q_min": 900, "q_max": 1024, "len_min": 6000, "len_max": 8192, "hq": 32, "hkv": 8, "hd": 128, "page": 64, "dtype": "bf16", "mix": 12},
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "read", "attention", "attention", "attention"])
    page, mix = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 30)
    if op == "plan":
        kind = rng.choice(["decode", "mixed"])
        seqs = _log(rng, 1, 1500)
        new = 1 if kind == "decode" else _log(rng, 2, max(2, min(2048, 300000 // seqs)))
        return {"op": op, "kind": kind, "seqs": seqs, "page": page, "len_max": _log(rng, 16, 8192), "new_max": new, "mix": mix}
    if op in ("append", "read"):
        tokens = _log(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "run": _log(rng, 1, tokens), "hkv": rng.choice([1, 2, 3, 4, 8]), "hd": rng.choice([64, 128]), "page": page,
                "dtype": rng.choice(["f32", "f16", "bf16"]), "mix": mix}
    hkv, group, hd, dtype = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([64, 128]), rng.choice(["f32", "f32", "f16", "bf16"])
    kind = rng.choice(["decode", "decode", "drafts", "chunks"])
    if kind == "decode":
        seqs = _log(rng, 1, 128)
        length = _log(rng, 16, 131072 // seqs)
        q = 1
    elif kind == "drafts":
        seqs, q = _log(rng, 1, 32), rng.randrange(2, 9)
        length = _log(rng, q, min(16384, 131072 // seqs))
    else:
        seqs, q = rng.randrange(1, 5), _log(rng, 16, 640)
        length = q + rng.choice([0, _log(rng, 1, 4096)])
        group = min(group, max(1, 32 // hkv))
    return {"op": op, "seqs": seqs, "q_min": rng.randrange(1, q + 1), "q_max": q, "len_min": rng.randrange(1, length + 1), "len_max": length, "hq": hkv * group,
            "hkv": hkv, "hd": hd, "page": page, "dtype": dtype, "mix": mix}


# ------------------------------------------------------------------------------------------- inputs

def _requests(case):
    """The lengths of a case's requests: plan: (cached, kept, new); attention: (query tokens, positions)."""
    r = random.Random(case["mix"])
    if case["op"] == "plan":
        rows = []
        for _ in range(case["seqs"]):
            n = r.randrange(1, case["len_max"] + 1)
            what = r.random() if case["kind"] == "mixed" else 1.0
            if what < 0.1:
                rows.append((n, 0, 0))  # finished
            elif what < 0.3:
                rows.append((0, 0, r.randrange(1, case["new_max"] + 1)))  # a prompt
            elif what < 0.5:
                rows.append((n, n - min(n, r.randrange(0, 8)), r.randrange(1, 1 + min(8, case["new_max"]))))  # a draft rolled back
            else:
                rows.append((n, n, 1))
        return rows
    rows = []
    for i in range(case["seqs"]):
        q = case["q_max"] if i == 0 else r.randrange(case["q_min"], case["q_max"] + 1)
        n = case["len_max"] if i == 0 else r.randrange(case["len_min"], case["len_max"] + 1)
        rows.append((q, max(q, n)))
    return rows


def _runs(case):
    """Lengths of the runs of neighbouring positions that an append or a read goes through."""
    r, left, runs = random.Random(case["mix"]), case["tokens"], []
    while left:
        n = min(left, max(1, int(case["run"] * r.uniform(0.5, 1.5))))
        runs.append(n)
        left -= n
    return runs


def _pages(n, page):
    return -(-n // page)


def _tile_bytes(hd):
    return 16 * (hd // 2 + hd // 16) * 2


def _quantise(x):
    """Scales (fp16) and codes (0..15) of x [..., 32 * n]: [..., n] and [..., n, 32]."""
    b = x.float().unflatten(-1, (-1, 32))
    m = torch.gather(b, -1, b.abs().argmax(-1, keepdim=True))  # the lowest index where several are the largest
    s = (m / -8).to(torch.float16)
    s64 = s.double()
    c = torch.where(s64 != 0, torch.round(b.double() / torch.where(s64 != 0, s64, 1.0)), 0.0) + 8  # in 64 bits: next to a half
    return s.squeeze(-1), c.clamp(0, 15).to(torch.uint8)


def _k_bytes(c):
    """Codes [..., pos 16, block, 32] to the bytes of a tile's K."""
    c = c.unflatten(-1, (4, 4, 2))  # dim / 8, byte, nibble
    return (c[..., 0] | c[..., 1] << 4).transpose(-3, -2).flatten(-4)


def _v_bytes(c):
    """Codes [..., pos 16, block, 32] to the bytes of a tile's V."""
    c = c.unflatten(-1, (8, 2, 2)).unflatten(-5, (2, 4, 2))  # half, pair, parity, block, dim / 4, byte, nibble
    b = c[..., 0] | c[..., 1] << 4
    n = b.dim()
    return b.permute(*range(n - 6), n - 6, n - 2, n - 5, n - 4, n - 3, n - 1).flatten(-6)


def _fill(g, n_pages, page, hkv, hd):
    """A cache of n_pages pages of quantised rows, as bytes; K has some channels larger than the others."""
    tiles, nb = page // 16, hd // 32
    wide = 1 + 3 * (torch.rand(hkv, 1, hd, device="cuda", generator=g) < 0.05)
    cache = torch.empty(n_pages, hkv, tiles, _tile_bytes(hd), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (hkv * page * hd))
    for a in range(0, n_pages, step):
        n = min(step, n_pages - a)
        parts = []
        for wider, pack in ((wide, _k_bytes), (1, _v_bytes)):
            x = torch.randn(n, hkv, page, hd, device="cuda", generator=g) * wider
            s, c = _quantise(x)
            parts += [pack(c.unflatten(2, (tiles, 16))), s.unflatten(2, (tiles, 16)).flatten(-2).contiguous().view(torch.uint8)]
        cache[a:a + n] = torch.cat(parts, -1)
    return cache


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    page = case["page"]
    if case["op"] == "plan":
        rows = _requests(case)
        n, stride = len(rows), max(_pages(max(l, k + w), page) for l, k, w in rows)
        have = [_pages(l, page) for l, _, _ in rows]
        more = sum(max(0, _pages(k + w, page) - h) for (_, k, w), h in zip(rows, have))
        total = sum(have) + more + 7
        ids = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)  # every page once: in a table, or free
        table = torch.full((n, stride), -1, dtype=torch.int32, device="cuda")
        h = _i32(have)
        at = torch.arange(stride, device="cuda")[None, :] < h[:, None]
        table[at] = ids[: sum(have)]
        head = int(torch.randint(0, total, (1,), device="cuda", generator=g))
        ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        free = total - sum(have)
        ring[(head + torch.arange(free, device="cuda")) % total] = ids[sum(have):]
        tokens = sum(w for _, _, w in rows)
        cap = tokens + 5  # a program's buffers are a little longer than a step's tokens
        s |= {"len": _i32([r[0] for r in rows]), "keep": _i32([r[1] for r in rows]), "new": _i32([r[2] for r in rows]), "table": table, "ring": ring,
              "free": _i32([head, free]), "len_out": _i32([0] * n), "free_out": _i32([0, 0]), "cu": _i32([0] * (n + 1)), "status": _i32([0])}
        s |= {k: _i32([0] * cap) for k in ("slot", "pos", "seq")}
        return s
    hkv, hd = case["hkv"], case["hd"]
    if case["op"] in ("append", "read"):
        runs = _runs(case)
        pages = [_pages(n + 3, page) for n in runs]
        n_pages = sum(pages) + 3
        ids = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
        first = torch.tensor([3 * (i % 2) for i in range(len(runs))], device="cuda")  # where in its first page a run begins
        runs_d, base = torch.tensor(runs, device="cuda"), torch.tensor(pages, device="cuda").cumsum(0) - torch.tensor(pages, device="cuda")
        of = torch.repeat_interleave(torch.arange(len(runs), device="cuda"), runs_d)
        at = torch.arange(case["tokens"], device="cuda") - (runs_d.cumsum(0) - runs_d)[of] + first[of]
        slot = ids[base[of] + at // page] * page + (at % page).to(torch.int32)
        if case["tokens"] > 8:
            slot[-case["tokens"] // 9:: 2] = -1  # padding
        s |= {"slot": slot.to(torch.int32).contiguous(), "n_pages": n_pages}
        s["cache"] = _fill(g, n_pages, page, hkv, hd) if case["op"] == "read" else torch.zeros(n_pages, hkv, page // 16, _tile_bytes(hd), dtype=torch.uint8, device="cuda")
        shape = (case["tokens"], hkv, hd)
        if case["op"] == "append":
            s |= {k: torch.randn(shape, device="cuda", generator=g).to(TYPES[case["dtype"]]) for k in ("k", "v")}
            s["k"][..., 5:: 31] *= 4
        out = torch.float32 if case["op"] == "append" else TYPES[case["dtype"]]
        s |= {k: torch.zeros(shape, dtype=out, device="cuda") for k in ("k_out", "v_out")}
        return s
    rows = _requests(case)
    pages = [_pages(n, page) for _, n in rows]
    n_pages, stride = sum(pages) + 2, max(pages)
    ids = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((len(rows), stride), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(stride, device="cuda")[None, :] < _i32(pages)[:, None]] = ids[: sum(pages)]
    cu = [0]
    for q, _ in rows:
        cu.append(cu[-1] + q)
    q = torch.randn(cu[-1], case["hq"], hd, device="cuda", generator=g).to(TYPES[case["dtype"]])
    s |= {"cache": _fill(g, n_pages, page, hkv, hd), "n_pages": n_pages, "table": table, "cu": _i32(cu), "len": _i32([n for _, n in rows]), "q": q, "out": torch.zeros_like(q),
          "longest": max(n for _, n in rows), "most": max(q for q, _ in rows), "scratch": torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda")}
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _tiles(s):
    """The cache's parts as views: K codes, K scales, V codes, V scales, each [tile, kv head, ...]."""
    hd = s["hd"]
    t = s["cache"].transpose(1, 2)  # [page, tile, head, bytes]
    a, b = 16 * hd // 2, 16 * hd // 16
    return t, (slice(0, a), slice(a, a + b), slice(a + b, 2 * a + b), slice(2 * a + b, 2 * a + 2 * b))


def _rows(s, tile):
    """K and V (fp32, exact) of the tiles with the given numbers (any shape): [..., 16, kv head, hd]."""
    t, (kc, ks, vc, vs) = _tiles(s)
    hd, nb = s["hd"], s["hd"] // 32
    x = t[tile // (s["page"] // 16), tile % (s["page"] // 16)]  # [..., head, bytes]
    lead = x.shape[:-1]

    def nibbles(b):
        return torch.stack((b & 15, b >> 4), -1).float() - 8

    k = nibbles(x[..., kc].reshape(*lead, 16, 4, nb, 4)).transpose(-4, -3).reshape(*lead, 16, nb, 32)
    v = nibbles(x[..., vc].reshape(*lead, 2, 8, 4, 2, nb, 2))
    n = len(lead)
    v = v.permute(*range(n), n, n + 2, n + 3, n + 4, n + 1, n + 5, n + 6).reshape(*lead, 16, nb, 32)
    out = []
    for c, at in ((k, ks), (v, vs)):
        scale = x[..., at].contiguous().view(torch.float16).reshape(*lead, 16, nb, 1).float()
        out.append((c * scale).flatten(-2).transpose(-3, -2))
    return out


def _plain_plan(s):
    n, stride = s["table"].shape
    page, cap, tokens = s["page"], s["ring"].numel(), s["slot"].numel()
    have, need = (s["len"].long() + page - 1) // page, (s["keep"].long() + s["new"] + page - 1) // page
    head, count = s["free"][0].long(), s["free"][1].long()
    take, give = (need - have).clamp(min=0), (have - need).clamp(min=0)
    col = torch.arange(stride, device="cuda")[None, :]
    taken = s["ring"][(head + (take.cumsum(0) - take)[:, None] + (col - have[:, None]).clamp(min=0)) % cap]
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), taken, s["table"])
    back = (col >= need[:, None]) & (col < have[:, None])
    to = (head + count + (give.cumsum(0) - give)[:, None] + col - need[:, None]) % cap
    ring = torch.cat((s["ring"], s["ring"][:1])).index_put((torch.where(back, to, cap),), s["table"])[:cap]  # the last entry takes what stays
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), s["new"].long().cumsum(0)))
    t = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    pos = s["keep"].long()[seq] + t - cu[seq]
    real = t < cu[n]
    slot = table[seq, (pos // page).clamp(0, stride - 1)].long() * page + pos % page
    a, b = take.sum(), give.sum()
    return {"len": s["keep"] + s["new"], "table": table, "ring": ring, "free": torch.stack(((head + a) % cap, count - a + b)).int(), "cu": cu.int(),
            "slot": torch.where(real, slot, -1).int(), "pos": torch.where(real, pos, -1).int(), "seq": torch.where(real, seq, -1).int(),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _plain_append(s):
    vc, cache = _tiles(s)[1][2], s["cache"].view(-1)
    hd, page, nb = s["hd"], s["page"], s["hd"] // 32
    slot = s["slot"].long()
    real = (slot >= 0) & (slot < s["n_pages"] * page)
    at = torch.where(real, slot, 0)
    where = (at // page, at % page // 16)
    p = (at % 16)[:, None, None, None]
    dev = slot.device
    tok, head, block = (torch.arange(x, device=dev).view(v) for x, v in ((slot.numel(), (-1, 1, 1, 1)), (s["hkv"], (1, -1, 1, 1)), (nb, (1, 1, -1, 1))))
    codes = hd // 2 * 16
    for x, base, is_k in ((s["k"], 0, True), (s["v"], vc.start, False)):
        scale, c = _quantise(x)
        b = c[..., 0::2] | c[..., 1::2] << 4  # [token, head, block, 16 bytes]
        j = torch.arange(16, device=dev).view(1, 1, 1, -1)
        if is_k:
            off = p * (hd // 2) + j // 4 * (4 * nb) + block * 4 + j % 4
        else:
            off = (((p // 8 * 8 + j // 2) * 4 + p // 2 % 4) * 2 + p % 2) * (2 * nb) + block * 2 + j % 2
        full = ((where[0][:, None, None, None] * s["hkv"] + head) * (page // 16) + where[1][:, None, None, None]) * _tile_bytes(hd)
        keep = real.view(-1, 1, 1, 1).expand(b.shape)
        cache[(full + base + off)[keep]] = b[keep]
        sb = scale.contiguous().view(torch.uint8).unflatten(-1, (nb, 2))
        off = base + codes + (p * nb + block) * 2 + torch.arange(2, device=dev).view(1, 1, 1, -1)
        keep = real.view(-1, 1, 1, 1).expand(sb.shape)
        cache[(full + off)[keep]] = sb[keep]
    return _plain_read(s, torch.float32)


def _plain_read(s, dtype):
    slot = s["slot"].long()
    real = ((slot >= 0) & (slot < s["n_pages"] * s["page"])).view(-1, 1, 1)
    at = slot.clamp(0, s["n_pages"] * s["page"] - 1)
    k, v = _rows(s, at // 16)  # [token, 16, head, hd]
    i = torch.arange(slot.numel(), device=slot.device)
    return {"k": torch.where(real, k[i, at % 16].to(dtype), s["k_out"]), "v": torch.where(real, v[i, at % 16].to(dtype), s["v_out"])}


def _plain_attention(s):
    n, hq, hkv, hd, page = s["table"].shape[0], s["hq"], s["hkv"], s["hd"], s["page"]
    per = page // 16
    tiles = (s["table"].clamp(min=0).long()[:, :, None] * per + torch.arange(per, device="cuda")).flatten(1)
    tiles = tiles[:, : -(-s["longest"] // 16)]
    k, v = (x.flatten(1, 2) for x in _rows(s, tiles))  # [seq, position, head, hd]
    j = torch.arange(k.shape[1], device="cuda")
    start, length = s["cu"][:-1].long(), s["len"].long()
    count = s["cu"][1:].long() - start
    i = torch.arange(s["most"], device="cuda")
    token = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1)  # [seq, i]
    q = s["q"].float()[token].unflatten(2, (hkv, hq // hkv))  # [seq, i, head, group, hd]
    scores = torch.matmul(q.permute(0, 2, 3, 1, 4), k.permute(0, 2, 3, 1)[:, :, None]) / math.sqrt(hd)  # [seq, head, group, i, position]
    last = (length - count)[:, None] + i  # the position of query token i
    seen = j <= last[:, :, None]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    o = torch.matmul(e, v.permute(0, 2, 1, 3)[:, :, None])
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [seq, i, hq, hd]
    t = torch.arange(s["q"].shape[0], device="cuda")
    of = torch.searchsorted(s["cu"][1:].long(), t, right=True).clamp(max=n - 1)
    return o[of, t - start[of]].to(s["q"].dtype)


def run(s):
    if not own:
        if s["op"] == "plan":
            return _plain_plan(s)
        if s["op"] == "append":
            return _plain_append(s)
        if s["op"] == "read":
            return _plain_read(s, TYPES[s["dtype"]])
        return _plain_attention(s)
    import layer_range_stage_gb300 as L

    if s["op"] == "plan":
        L.stage_op_kv4_plan(s["page"], s["len"], s["new"], s["table"], s["ring"], s["free"], s["len_out"], s["free_out"], s["cu"], s["slot"], s["pos"], s["seq"], s["status"],
                            keep_len=s["keep"])
        return {"len": s["len_out"], "table": s["table"], "ring": s["ring"], "free": s["free_out"], "cu": s["cu"], "slot": s["slot"], "pos": s["pos"], "seq": s["seq"],
                "status": s["status"]}
    if s["op"] == "append":
        L.stage_op_kv4_append(s["cache"], s["k"], s["v"], s["slot"])
    if s["op"] in ("append", "read"):
        L.stage_op_kv4_read(s["cache"], s["slot"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    L.stage_op_kv4_attention(s["cache"], s["q"], s["cu"], s["len"], s["table"], s["out"], max_q=s["most"], max_len=s["longest"], workspace=s["scratch"])
    return s["out"]


# ------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    page = case["page"]
    if case["op"] == "plan":
        rows = _requests(case)
        tokens = sum(w for _, _, w in rows)
        moved = sum(abs(_pages(k + w, page) - _pages(l, page)) for l, k, w in rows)
        touched = sum(_pages(k + w, page) - k // page for _, k, w in rows if w)
        return {"bytes": 4 * (5 * len(rows) + 3 * (tokens + 5) + 2 * moved + touched + 6), "flops": 0}
    if case["op"] in ("append", "read"):
        n = case["tokens"] * case["hkv"] * case["hd"] * 2
        wide = 4 if case["dtype"] == "f32" else 2
        packed = n // 2 + n // 16
        if case["op"] == "append":
            return {"bytes": n * wide + packed + n * 4 + 4 * case["tokens"], "flops": 4 * n}
        return {"bytes": n * wide + packed + 4 * case["tokens"], "flops": 2 * n}
    rows = _requests(case)
    wide = 4 if case["dtype"] == "f32" else 2
    tokens = sum(q for q, _ in rows)
    cache = sum(n for _, n in rows) * case["hkv"] * 2 * (case["hd"] // 2 + case["hd"] // 16)
    pairs = sum(sum(range(n - q + 1, n + 1)) for q, n in rows)
    return {"bytes": cache + 2 * tokens * case["hq"] * case["hd"] * wide + 4 * sum(_pages(n, page) for _, n in rows), "flops": 4 * pairs * case["hq"] * case["hd"]}


# ------------------------------------------------------------------------------------------- 64 bits

def _value(s, slot, head, dim, is_v):
    """The number at (slot, kv head, dim) of the cache, in 64 bits, by the address of its nibble."""
    hd, page = s["hd"], s["page"]
    nb, p = hd // 32, slot % 16
    block, j = dim // 32, dim % 32
    base = ((slot // page * s["hkv"] + head) * (page // 16) + slot % page // 16) * (36 * hd // 2)
    half = 9 * hd  # bytes of a tile's K, and of its V
    if is_v:
        at = base + half + p // 8 * (4 * hd) + j // 4 * (hd // 2) + p // 2 % 4 * (hd // 8) + p % 2 * (hd // 16) + block * 2 + j // 2 % 2
    else:
        at = base + p * (hd // 2) + j // 8 * (hd // 8) + block * 4 + j // 2 % 4
    code = s["cache"].view(-1)[at].long() >> (4 * (j % 2)) & 15
    scales = s["cache"].view(-1).view(torch.float16)[(base + (half if is_v else 0) + 8 * hd) // 2 + p * nb + block]
    return scales.double() * (code - 8)


def _rows64(s, slots, is_v):
    at = (slots[:, None, None], torch.arange(s["hkv"], device="cuda")[None, :, None], torch.arange(s["hd"], device="cuda"))
    return _value(s, *at, is_v)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] in ("append", "read"):
        real = (s["slot"] >= 0)[:, None, None]
        found = {}
        for name in ("k", "v"):
            if case["op"] == "read":
                x = _rows64(s, s["slot"].long().clamp(min=0), name == "v")
            else:
                b = s[name].double().reshape(case["tokens"], case["hkv"], -1, 32)
                big, low = b.max(-1).values, b.min(-1).values
                first_high = (b == big[..., None]).int().argmax(-1)
                first_low = (b == low[..., None]).int().argmax(-1)
                m = torch.where(big > -low, big, torch.where(big < -low, low, torch.where(first_high < first_low, big, low)))
                step = (m / -8).float().half().double()[..., None]
                n = torch.where(step == 0, 0.0, torch.round(b / torch.where(step == 0, 1.0, step)).clamp(-8, 7))
                x = (n * step).flatten(-2)
            found[name] = torch.where(real, x, 0.0)
        return found
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // case["hkv"]
    cu = s["cu"].tolist()
    for i, n in enumerate(s["len"].tolist()):
        at = torch.arange(n, device="cuda")
        slots = s["table"][i].long()[at // case["page"]] * case["page"] + at % case["page"]
        count = cu[i + 1] - cu[i]
        hidden = at[None, :] > (n - count + torch.arange(count, device="cuda"))[:, None]
        for h in range(case["hkv"]):
            k, v = (_value(s, slots[:, None], h, torch.arange(case["hd"], device="cuda"), is_v) for is_v in (False, True))
            for j in range(h * group, h * group + group):
                z = (s["q"][cu[i]:cu[i + 1], j].double() @ k.T) / case["hd"] ** 0.5
                z[hidden] = -math.inf
                out[cu[i]:cu[i + 1], j] = torch.softmax(z, -1) @ v
    return out
