"""A step's operators around the projections: what is measured, and their plain forms.

Four operators that a program which puts a decoder's step together from single calls makes one after another:

  norm      the residual's addition, a root-mean-square norm, and rows of 8 bits (e4m3) with a scale for each 128 columns
  product   rows of 8 bits times a weight matrix of 8 bits with a scale for each block of 128 x 128
  rope      rotary positions of the query and key heads
  logprobs  log probabilities of given tokens, the entropy, the tokens' ranks, and the likeliest tokens

Scales of rows lie block by block: [block of 128 columns][row].  Scales of weights: [block of 128 rows][block of 128 columns].
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
EPS = 1e-5


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of the 8B shape, between two blocks: latency
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 4096, "x": "f32", "resid": "f32", "gamma": True, "y": False, "mix": 1},
        # four prompts of the 8B shape, sums of projections in 16 bits on a residual stream of 32
        {"name": "norm prompts 2048", "op": "norm", "rows": 2048, "cols": 4096, "x": "bf16", "resid": "f32", "gamma": True, "y": False, "mix": 2},
        # a long ragged prompt batch of the 70B shape
        {"name": "norm ragged 16411", "op": "norm", "rows": 16411, "cols": 8192, "x": "bf16", "resid": "bf16", "gamma": True, "y": False, "mix": 3},
        # one token's q, k and v of the 8B shape
        {"name": "product one token", "op": "product", "rows": 1, "k": 4096, "n": 6144, "out": "bf16", "mix": 4},
        # a decode step of 64 sequences through the 70B shape's up and gate
        {"name": "product step 64", "op": "product", "rows": 64, "k": 8192, "n": 57344, "out": "bf16", "mix": 5},
        # a ragged batch through the 8B shape's down projection, onto a stream of 32 bits
        {"name": "product ragged 777", "op": "product", "rows": 777, "k": 14336, "n": 4096, "out": "f32", "mix": 6},
        # four prompts through the 8B shape's up and gate
        {"name": "product prompts 2048", "op": "product", "rows": 2048, "k": 4096, "n": 28672, "out": "bf16", "mix": 7},
        # a decode step of 64 sequences (the 70B shape's heads)
        {"name": "rope step 64", "op": "rope", "rows": 64, "hq": 64, "hkv": 8, "hd": 128, "rot": 128, "pairs": "half", "far": 4096, "scaling": "none", "dtype": "f32", "mix": 8},
        # a prompt batch far into long contexts, half of each head rotated
        {"name": "rope prompts 16384", "op": "rope", "rows": 16384, "hq": 32, "hkv": 8, "hd": 128, "rot": 64, "pairs": "interleaved", "far": 1000000, "scaling": "parts",
         "dtype": "bf16", "mix": 9},
        # one answer's next token over the MoE shape's vocabulary, with 20 alternatives: latency
        {"name": "logprobs one row", "op": "logprobs", "rows": 1, "vocab": 151936, "top": 20, "dtype": "f32", "mix": 10},
        # a decode step of 64 sequences over the 70B shape's vocabulary
        {"name": "logprobs step 64", "op": "logprobs", "rows": 64, "vocab": 128256, "top": 5, "dtype": "f32", "mix": 11},
        # prompts scored over the 8B shape's vocabulary
        {"name": "logprobs prompts 4099", "op": "logprobs", "rows": 4099, "vocab": 32000, "top": 1, "dtype": "bf16", "mix": 12},
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op, mix = rng.choice(["norm", "product", "product", "rope", "logprobs"]), rng.randrange(1 << 30)
    if op == "norm":
        cols = rng.choice([256, 688, 768, 1000, 2048, 4096, 8192, 14336, 28672, _log(rng, 64, 28672)])
        x = rng.choice(["f32", "f16", "bf16", "bf16"])
        return {"op": op, "rows": _log(rng, 1, min(16411, 55000000 // cols)), "cols": cols, "x": x, "resid": rng.choice(["none", "f32", x, x]),
                "gamma": rng.random() < 0.8, "y": rng.random() < 0.3, "mix": mix}
    if op == "product":
        k, n = rng.choice([256, 688, 1000, 2048, 4096, 8192, _log(rng, 64, 14336)]), rng.choice([512, 1001, 4096, 6144, 10240, 32000, _log(rng, 16, 32000)])
        return {"op": op, "rows": _log(rng, 1, max(1, min(4096, 200000000000 // (k * n)))), "k": k, "n": n, "out": rng.choice(["f32", "f16", "bf16", "bf16"]), "mix": mix}
    if op == "rope":
        hkv, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 64, 80, 128, 128, 256])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        rot = rng.choice([hd, hd, hd // 2, hd // 4])
        return {"op": op, "rows": _log(rng, 1, min(16384, 40000000 // ((hq + hkv) * hd))), "hq": hq, "hkv": hkv, "hd": hd, "rot": rot, "pairs": rng.choice(["half", "interleaved"]),
                "far": _log(rng, 64, 2000000), "scaling": rng.choice(["none", "linear", "bands", "parts"]), "dtype": rng.choice(["f32", "f16", "bf16"]), "mix": mix}
    vocab = rng.choice([1024, 32000, 50257, 128256, 151936, _log(rng, 1000, 262144)])
    return {"op": op, "rows": _log(rng, 1, max(1, min(8192, 65000000 // vocab))), "vocab": vocab, "top": rng.choice([0, 1, 2, 5, 8, 20, rng.randrange(0, 33)]),
            "dtype": rng.choice(["f32", "f32", "f16", "bf16"]), "mix": mix}


# ------------------------------------------------------------------------------------------- inputs

def _up(n, m):
    return -(-n // m) * m


def _blocks(n):
    return -(-n // 128)


def _rows8(x):
    """Rows of 8 bits and their scales of x [rows, cols], as a program that quantises would hold them: a row stride of a multiple of 16 bytes."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, _blocks(cols) * 128 - cols)).unflatten(1, (-1, 128))
    s = b.abs().amax(-1).clamp(min=1e-30) / 448
    q = torch.zeros(rows, _up(cols, 16), dtype=F8, device=x.device)
    q[:, :cols] = (b / s[..., None]).flatten(1)[:, :cols].clamp(-448, 448).to(F8)
    return q[:, :cols], s.t().contiguous()


def _weights8(n, k, g):
    """A weight matrix [n, k] of 8 bits and its scales, some rows larger than the others."""
    q = torch.zeros(n, _up(k, 16), dtype=F8, device="cuda")
    s = torch.empty(_blocks(n), _blocks(k), device="cuda")
    for a in range(0, n, 4096):  # a part at a time
        m = min(4096, n - a)
        w = torch.randn(m, k, device="cuda", generator=g) * 0.02
        w[::37] *= 3
        b = torch.nn.functional.pad(w, (0, _blocks(k) * 128 - k, 0, _blocks(m) * 128 - m)).unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
        t = b.abs().amax((1, 3)) / 448
        q[a:a + m, :k] = (b / t[:, None, :, None]).flatten(2).flatten(0, 1)[:m, :k].clamp(-448, 448).to(F8)
        s[a // 128: a // 128 + t.shape[0]] = t
    return q[:, :k], s


def _freqs(case):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated values."""
    r, theta, factor, first = case["rot"], 10000.0, 8.0, 4096.0
    f = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "bands":  # long waves are stretched, short ones kept, those between mixed by their length
        mix = [min(1.0, max(0.0, (first * x / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for x in f]
        return [x * (m + (1 - m) / factor) for x, m in zip(f, mix)], 1.0
    if case["scaling"] == "parts":  # the same by the pair's number, between those that turn 32 times and once
        at = [r * math.log(first / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (32.0, 1.0)]
        low, high = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(r // 2)]
        return [x * (m / factor + 1 - m) for x, m in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    rows = case["rows"]
    if case["op"] == "norm":
        cols = case["cols"]
        # a stream with a few strong channels, as deep blocks have
        strong = 1 + 20 * (torch.rand(cols, device="cuda", generator=g) < 0.01)
        s["in"] = (torch.randn(rows, cols, device="cuda", generator=g) * 0.5).to(TYPES[case["x"]])
        s["stream"] = s["stream_out"] = None
        if case["resid"] != "none":
            s["stream"] = (torch.randn(rows, cols, device="cuda", generator=g) * strong).to(TYPES[case["resid"]])
            s["stream_out"] = torch.zeros_like(s["stream"])
        s["weight"] = 1 + 0.1 * torch.randn(cols, device="cuda", generator=g) if case["gamma"] else None
        s["q"] = torch.zeros(rows, _up(cols, 16), dtype=F8, device="cuda")[:, :cols]
        s["scale"] = torch.zeros(_blocks(cols), rows, device="cuda")
        s["plain"] = torch.zeros(rows, cols, dtype=TYPES[case["x"]], device="cuda") if case["y"] else None
        return s
    if case["op"] == "product":
        x = torch.randn(rows, case["k"], device="cuda", generator=g)
        x[:, 5::61] *= 8
        s["a"], s["a_scale"] = _rows8(x)
        s["w"], s["w_scale"] = _weights8(case["n"], case["k"], g)
        s["out_"] = torch.zeros(rows, case["n"], dtype=TYPES[case["out"]], device="cuda")
        return s
    if case["op"] == "rope":
        hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
        qkv = torch.randn(rows, hq + 2 * hkv, hd, device="cuda", generator=g).to(TYPES[case["dtype"]])  # one projection's output
        pos = torch.randint(0, case["far"] + 1, (rows,), device="cuda", generator=g).to(torch.int32)
        if rows > 16:
            pos[5::17] = -1  # padding
        f, s["factor"] = _freqs(case)
        s |= {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "pos": pos, "freqs": torch.tensor(f, dtype=torch.float64, device="cuda")}
        s |= {n + "_out": torch.zeros(rows, h, hd, dtype=TYPES[case["dtype"]], device="cuda") for n, h in (("q", hq), ("k", hkv))}
        return s
    vocab, top = case["vocab"], case["top"]
    z = torch.randn(rows, vocab, device="cuda", generator=g) * 2.5
    if case["mix"] % 2 == 0:  # banned tokens, in the two ways that programs write
        z[:, 3::29] = -math.inf
        z[:, 7::31] = torch.finfo(TYPES[case["dtype"]]).min
    likely = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    z[torch.arange(rows, device="cuda"), likely] = 12.0 + 4 * torch.rand(rows, device="cuda", generator=g)
    given = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    banned = (given % 29 == 3) | (given % 31 == 7)  # a program gives tokens that it allows
    given = torch.where((torch.rand(rows, device="cuda", generator=g) < 0.7) | banned, likely, given)
    s |= {"logits": z.to(TYPES[case["dtype"]]), "tokens": given.to(torch.int32)}
    s |= {k: torch.zeros(rows, device="cuda") for k in ("logprob", "entropy")}
    s |= {"rank": torch.zeros(rows, dtype=torch.int32, device="cuda"), "ids": torch.zeros(rows, top, dtype=torch.int32, device="cuda"), "best": torch.zeros(rows, top, device="cuda")}
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _plain_norm(s):
    """32 bits but for the mean of squares; y, the scales and the codes are defined by their roundings to 32 bits."""
    h = s["in"].float()
    if s["stream"] is not None:
        h = (h + s["stream"].float()).to(s["stream"].dtype)
        s["stream_out"].copy_(h)
        h = h.float()
    y, cols = h, s["cols"]
    if s["weight"] is not None:
        eps = torch.tensor(EPS, device="cuda").double()
        r = (1 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + eps)).float()
        y = h * r * s["weight"]
    b = torch.nn.functional.pad(y, (0, _blocks(cols) * 128 - cols)).unflatten(1, (-1, 128))
    top = b.abs().amax(-1).clamp(min=2.0 ** -100)
    full = torch.full_like(top, 448)
    s["scale"].copy_((top / full).t())
    s["q"].copy_((b * (full / top)[..., None]).flatten(1)[:, :cols].to(F8))
    if s["plain"] is not None:
        s["plain"].copy_(y)


def _plain_product(s):
    a = s["a"].float() * s["a_scale"].repeat_interleave(128, 0)[:s["k"]].t()
    w = s["w"].float() * s["w_scale"].repeat_interleave(128, 0)[:s["n"]].repeat_interleave(128, 1)[:, :s["k"]]
    s["out_"].copy_(torch.matmul(a, w.t()))


def _plain_rope(s):
    angle = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    live, r = (s["pos"] >= 0)[:, None, None], s["rot"]
    for name in ("q", "k"):
        x, out = s[name].float(), s[name + "_out"]
        u, v = (x[..., :r // 2], x[..., r // 2:r]) if s["pairs"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
        u, v = u * cos - v * sin, v * cos + u * sin
        turned = torch.cat((u, v), -1) if s["pairs"] == "half" else torch.stack((u, v), -1).flatten(-2)
        out.copy_(torch.where(live, torch.cat((turned, x[..., r:]), -1).to(out.dtype), out))


def _plain_logprobs(s):
    z, t = s["logits"].float(), s["tokens"].long()[:, None]
    top = z.amax(-1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    log = torch.log(total)
    s["logprob"].copy_((d.gather(1, t) - log)[:, 0])
    s["entropy"].copy_((log - torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / total)[:, 0])
    at = z.gather(1, t)
    s["rank"].copy_(((z > at) | ((z == at) & (torch.arange(s["vocab"], device="cuda") < t))).sum(-1))
    if s["top"]:
        ids = torch.argsort(z, dim=-1, descending=True, stable=True)[:, :s["top"]]  # equal ones by their index
        s["ids"].copy_(ids)
        s["best"].copy_(d.gather(1, ids) - log)


def run(s):
    op = s["op"]
    if not own:
        {"norm": _plain_norm, "product": _plain_product, "rope": _plain_rope, "logprobs": _plain_logprobs}[op](s)
    if own:
        import layer_range_stage_gb300 as L

        if op == "norm":
            L.stage_op_norm_f8(s["in"], s["q"], s["scale"], gamma=s["weight"], eps=EPS, resid=s["stream"], resid_out=s["stream_out"], y=s["plain"])
        elif op == "product":
            L.stage_op_f8_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out_"])
        elif op == "rope":
            L.stage_op_rope(s["q"], s["k"], s["pos"], s["freqs"], q_out=s["q_out"], k_out=s["k_out"], interleaved=s["pairs"] == "interleaved", scale=s["factor"])
        else:
            L.stage_op_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], rank=s["rank"], top_ids=s["ids"], top_logprobs=s["best"])
    if op == "norm":
        return {"stream": s["stream_out"], "q": s["q"], "scale": s["scale"], "y": s["plain"]}
    if op == "product":
        return s["out_"]
    if op == "rope":
        return {"q": s["q_out"], "k": s["k_out"]}
    return {"logprob": s["logprob"], "entropy": s["entropy"], "rank": s["rank"], "ids": s["ids"], "best": s["best"]}


# ------------------------------------------------------------------------------------------- what a pass needs

def _bytes(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    rows = case["rows"]
    if case["op"] == "norm":
        cols = case["cols"]
        each = _bytes(case["x"]) * (2 if case["y"] else 1) + (0 if case["resid"] == "none" else 2 * _bytes(case["resid"])) + 1
        return {"bytes": rows * cols * each + 4 * rows * _blocks(cols) + (4 * cols if case["gamma"] else 0), "flops": 8 * rows * cols}
    if case["op"] == "product":
        k, n = case["k"], case["n"]
        return {"bytes": rows * k + n * k + rows * n * _bytes(case["out"]) + 4 * _blocks(k) * (rows + _blocks(n)), "flops": 2 * rows * n * k}
    if case["op"] == "rope":
        live = rows - (len(range(5, rows, 17)) if rows > 16 else 0)
        heads = case["hq"] + case["hkv"]
        return {"bytes": live * heads * case["hd"] * 2 * _bytes(case["dtype"]) + 4 * rows + 4 * case["rot"], "flops": 3 * live * heads * case["rot"]}
    return {"bytes": rows * (case["vocab"] * _bytes(case["dtype"]) + 16 + 8 * case["top"]), "flops": 5 * rows * case["vocab"]}


# ------------------------------------------------------------------------------------------- 64 bits

def _32(x):
    """x (64 bits) rounded to 32, where the definition rounds."""
    return x.to(torch.float32).double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        stream = None
        found = {"q": torch.empty(case["rows"], case["cols"], dtype=torch.float64, device="cuda"), "scale": torch.empty(_blocks(case["cols"]), case["rows"], dtype=torch.float64, device="cuda")}
        if s["stream"] is not None:
            stream = (s["in"].double() + s["stream"].double()).float().to(s["stream"].dtype).double()  # a sum of two 32-bit numbers, then the stream's type
        h = s["in"].double() if stream is None else stream
        if case["gamma"]:
            scale = torch.rsqrt((h * h).sum(1) / case["cols"] + torch.tensor(EPS).double().item())
            h = _32(_32(h * _32(scale)[:, None]) * s["weight"].double())
        for b in range(_blocks(case["cols"])):
            part = h[:, 128 * b: 128 * b + 128]
            most = torch.maximum(part.max(1).values, -part.min(1).values).clamp(min=2.0 ** -100)
            found["scale"][b] = _32(most / torch.tensor(448.0, dtype=torch.float64, device="cuda"))
            v = _32(part * _32(torch.tensor(448.0, dtype=torch.float64, device="cuda") / most)[:, None])
            # the nearest number of 4 significant bits, or multiple of 2^-9; ties to even
            step = torch.exp2(torch.clamp(torch.frexp(v).exponent - 4, min=-9).double())
            found["q"][:, 128 * b: 128 * b + 128] = torch.round(v / step) * step
        return {"stream": stream, "q": found["q"], "scale": found["scale"], "y": h if case["y"] else None}
    if case["op"] == "product":
        k = case["k"]
        out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        for b in range(_blocks(k)):  # a block of the sum at a time, its scales behind its product
            at = slice(128 * b, min(k, 128 * b + 128))
            part = s["a"][:, at].double() @ s["w"][:, at].double().T
            out += part * s["a_scale"][b].double()[:, None] * s["w_scale"][:, b].double()[torch.arange(case["n"], device="cuda") // 128]
        return out
    if case["op"] == "rope":
        found = {}
        i = torch.arange(case["hd"], device="cuda")
        half = case["rot"] // 2
        first = i < half if case["pairs"] == "half" else i % 2 == 0
        other = torch.where(first, i + half, i - half) if case["pairs"] == "half" else i ^ 1
        pair = i % max(1, half) if case["pairs"] == "half" else i // 2
        angle = s["pos"].double()[:, None] * s["freqs"][pair.clamp(max=half - 1)]
        turn = i < case["rot"]
        c = torch.where(turn, angle.cos() * s["factor"], 1.0)[:, None]
        d = torch.where(turn, angle.sin() * torch.where(first, -1.0, 1.0) * s["factor"], 0.0)[:, None]
        for name in ("q", "k"):
            x = s[name].double()
            found[name] = (x * c + x[..., torch.where(turn, other, i)] * d) * (s["pos"] >= 0)[:, None, None]
        return found
    rows, top = case["rows"], case["top"]
    found = {n: torch.empty(rows, dtype=torch.float64, device="cuda") for n in ("logprob", "entropy")} | {"best": torch.empty(rows, top, dtype=torch.float64, device="cuda")}
    for a in range(0, rows, 512):
        z = s["logits"][a:a + 512].double()
        lse = torch.logsumexp(z, 1, keepdim=True)
        logp = z - lse
        found["logprob"][a:a + 512] = logp[torch.arange(len(z), device="cuda"), s["tokens"][a:a + 512].long()]
        found["entropy"][a:a + 512] = -(logp.exp() * logp.clamp(min=-1e300)).sum(1)
        found["best"][a:a + 512] = torch.sort(logp, 1, descending=True).values[:, :top]
    return {**found, "rank": None, "ids": None}
