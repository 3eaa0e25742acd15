"""The paged 4-bit cache's kernels against the float64 oracle (oracle/kv4.py).

Plan, append and read (float32) are exact: whole numbers, and values that float32 holds exactly.  Read in a
16-bit type is one rounding of an exact value: equal to numpy's.

Attention, per output value: with A = sum_j p_j |v_j| and X = max_j sum_d |q_d k_jd| / sqrt(D) (both from the
oracle) a score is off by at most 2^-19 X -- the fp16 pairs hold q to 2^-22 and products are exact; a score is
then at most 128 / 16 + 4 float32 additions, some truncating, of terms that add up to X in magnitude: under 2^-20 X
for the sums and 2^-20 X for the operands, the block scales' products and the scaling by log2(e) / sqrt(D).
exp of it is off by a factor 1 + 2^-19 X + 2^-20 (the exponential unit's 2^-22 and the argument's rounding,
which X covers), in numerator and denominator: 2 (2^-19 X + 2^-20).  The probabilities' fp16 pairs (2^-21, or
2^-38 of the largest), the sums (chains of at most 64 truncating additions, 64 * 2^-24 = 2^-18, then chains of
additions to nearest over the rest: 2^-18 again at these lengths), the merge and the division (2^-21) add under 2^-16.  So
    |got - want| <= (2^-18 X + 2^-16) A.
The low halves of the pairs end at fp16's smallest step, 2^-24: with x_j = 2^(z_j - r) s_j (s_j: the block's V scale, e_j the
least integer with s_j < 2^(e_j) for the row's largest scale, at least -14; r <= max_j (z_j + e_j) - 11) each x_j is off by at most
2^-25 more, times |c - 8| <= 8.  The sum that divides it is at least 2^(z_j - r) / p_j >= 2^(11 - e_j) / p_j for the
position j that sets r, so this adds at most, over N positions,
    N 2^-22 2^(e_j - 11) p_j <= N p_j max(2^-35 (8 s_j), 2^-47) <= N (2^-34 max_jd p_j |v_jd| + 2^-47):
2^(e_j) <= 2 s_j, or 2^-14 where s_j is subnormal, and a block's largest |v| is at least 4 s_j at any s_j (8 s_j
rounded to a code, a code cut off at 15 still 7 s_j).
Chunks hold V as two fp16 values relative to a power of two above its position's largest scale s_j (2^(e_j) <= 2 s_j, s_j's
subnormal steps included, or 2^-14): the low one ends at 2^-24, so each value is off by at most 2^-25 2^(e_j) <= 2^-26 max_d |v_jd|,
or 2^-39 at subnormal scales, and the sum by N (2^-26 max_jd p_j |v_jd| + 2^-39 max_j p_j).
In the 16-bit types a probability may be rounded once to fp16 (2^-11 A), and the output is rounded once: eps / 2 of its
value.  Chunks of many tokens in bfloat16 also round K and V to fp16 once each: V adds 2^-11 A; K moves a score by up to
2^-11 X, its exponential by that factor in numerator and denominator: 2^-10 X A.
"""
import numpy as np
import pytest

from oracle import kv4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def B(cuda):
    from layer_range_stage_gb300 import binding
    return binding


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def as_given(x, dtype):
    """float64 of the numbers a tensor of this type holds."""
    return torch.as_tensor(x).to(DT[dtype]).double().numpy()


def same(a, b):
    a, b = np.asarray(a), np.asarray(b)
    assert a.shape == b.shape
    assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), (np.argwhere((a != b) & ~((a != a) & (b != b)))[:5], a.dtype)


def check_attention(got, ref, dtype, rows=None, chunk=False):
    out, weight, spread, peak, seen = ref
    got = got.detach().double().cpu().numpy()
    tol = (2.0 ** -18 * spread[..., None] + 2.0 ** -16) * weight + (seen * (2.0 ** -34 * peak + 2.0 ** -47))[..., None]
    if chunk:
        tol = tol + (seen * (2.0 ** -26 * peak + 2.0 ** -39))[..., None]
    if dtype != "f32":
        tol = tol + 2.0 ** -11 * weight + torch.finfo(DT[dtype]).eps / 2 * np.abs(out)
    if dtype == "bf16":
        tol = tol + (2.0 ** -11 + 2.0 ** -10 * spread[..., None]) * weight
    some = ~np.isnan(out) if rows is None else rows
    err = np.abs(got - out)[some]
    assert (err <= tol[some]).all(), (float((err / np.maximum(tol[some], 1e-300)).max()), np.argwhere(~(np.abs(got - out) <= tol) & some)[:4])


def random_cache(rng, pages, page, hkv, d, wide=1.0):
    """Cache with normal rows everywhere, as numpy and on the device."""
    cache = kv4.cache_array(pages, page, hkv, d)
    n = pages * page
    k = (rng.standard_normal((n, hkv, d)) * wide).astype(np.float32)
    v = (rng.standard_normal((n, hkv, d)) * wide).astype(np.float32)
    for is_v, x in ((False, k), (True, v)):
        bits, codes = kv4.quantise(x)
        p, dims, blocks = np.arange(n) % 16, np.arange(d), np.arange(d // 32)
        flat = cache.reshape(pages, hkv, page // 16, 18 * d).transpose(0, 2, 1, 3)       # [page, tile, head, bytes]
        flat = flat.reshape(pages * page // 16, hkv, 18 * d).copy()
        at, _ = kv4.code_place(p[:, None], dims[0::2], d, is_v)
        sp = kv4.scale_place(p[:, None], blocks, d, is_v)
        tile = np.arange(n) // 16
        for h in range(hkv):
            flat[tile[:, None], h, at] = codes[:, h, 0::2] | codes[:, h, 1::2] << 4
            flat[tile[:, None], h, sp] = bits[:, h] & 255
            flat[tile[:, None], h, sp + 1] = bits[:, h] >> 8
        cache = np.ascontiguousarray(flat.reshape(pages, page // 16, hkv, 18 * d).transpose(0, 2, 1, 3))
    return cache, torch.from_numpy(cache).cuda()


# ------------------------------------------------------------------------------------------- append, read

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,hkv,page,n", [(128, 8, 64, 70), (64, 3, 16, 41), (128, 1, 32, 1), (64, 1, 48, 5), (64, 5, 16, 17)])
def test_append_and_read_are_exact(B, dtype, d, hkv, page, n):
    rng = np.random.default_rng(d + hkv + n)
    pages = n // page + 3
    cache = rng.integers(0, 256, kv4.cache_array(pages, page, hkv, d).shape).astype(np.uint8)   # what lies there is kept
    k, v = (as_given(rng.standard_normal((n, hkv, d)) * 10.0 ** rng.integers(-4, 4, (n, hkv, 1)), dtype) for _ in range(2))
    k[0, 0, :32] = rng.integers(-16, 17, 32) / 2.0                 # ties of the rounding
    v[n // 2, -1, 3] = np.inf
    k[n // 2, 0, 32:40] = np.nan
    v[n - 1, 0, :32] = 0
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    if n > 4:
        slots[[1, 3, 4]] = [-1, pages * page, 2 ** 31 - 1]
    dev = torch.from_numpy(cache).cuda()
    # rows inside a fused buffer: 16 bytes between them
    pad = 16 // torch.finfo(DT[dtype]).bits * 8 + hkv * d
    fused = torch.zeros(n, 2 * pad, dtype=DT[dtype], device="cuda")
    kd, vd = (fused[:, i * pad: i * pad + hkv * d].unflatten(1, (hkv, d)) for i in (0, 1))
    kd.copy_(torch.as_tensor(k))
    vd.copy_(torch.as_tensor(v))
    B.stage_op_kv4_append(dev, kd, vd, i32(slots))
    torch.cuda.synchronize()
    kv4.append(cache, k, v, slots)
    same(dev.cpu().numpy(), cache)

    live = (slots >= 0) & (slots < pages * page)
    ko, vo = (torch.full((n, hkv, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    B.stage_op_kv4_read(dev, i32(slots), ko, vo)
    torch.cuda.synchronize()
    for got, is_v in ((ko, False), (vo, True)):
        want = np.full((n, hkv, d), 7.0)
        want[live] = torch.as_tensor(kv4.rows(cache, slots[live], is_v)).to(DT[dtype]).double().numpy()
        same(got.double().cpu().numpy(), want)


def test_read_of_any_bytes_and_one_slot_many_times(B):
    rng = np.random.default_rng(9)
    cache = rng.integers(0, 256, kv4.cache_array(4, 16, 2, 128).shape).astype(np.uint8)
    slots = np.array([5] * 9 + list(range(64)) + [-5, 64], np.int32)
    ko, vo = (torch.zeros(len(slots), 2, 128, device="cuda") for _ in range(2))
    B.stage_op_kv4_read(torch.from_numpy(cache).cuda(), i32(slots), ko, vo)
    with np.errstate(all="ignore"):
        for got, is_v in ((ko, False), (vo, True)):
            want = np.zeros((len(slots), 2, 128))
            want[:-2] = kv4.rows(cache, slots[:-2], is_v)
            same(got.double().cpu().numpy(), want)


def test_offsets_beyond_32_bits(B):
    """A cache of 4.8 GB: slots, pages and bytes past 2^32 (the last pages), and their attention."""
    rng = np.random.default_rng(11)
    hkv, d, page = 8, 128, 64
    pages = 4_800_000_000 // (page // 16 * hkv * 18 * d)
    dev = torch.empty((pages, hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
    assert dev.numel() > 1 << 32
    used = np.array([pages - 1, pages - 2, 3], np.int32)
    n = 150
    slots = used[np.arange(n) // page] * page + np.arange(n) % page
    k, v = (rng.standard_normal((n, hkv, d)).astype(np.float32) for _ in range(2))
    B.stage_op_kv4_append(dev, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(slots))
    small = kv4.cache_array(3, page, hkv, d)
    kv4.append(small, k, v, np.arange(n))
    same(dev[torch.as_tensor(used.astype(np.int64)).cuda()].cpu().numpy(), small)
    ko, vo = (torch.zeros(n, hkv, d, device="cuda") for _ in range(2))
    B.stage_op_kv4_read(dev, i32(slots), ko, vo)
    same(ko.double().cpu().numpy(), kv4.rows(small, np.arange(n), False))
    same(vo.double().cpu().numpy(), kv4.rows(small, np.arange(n), True))
    q = rng.standard_normal((2, 32, d)).astype(np.float32)
    out = torch.zeros(2, 32, d, device="cuda")
    ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(1, 32, hkv, d, 2, n), dtype=torch.uint8, device="cuda")
    B.stage_op_kv4_attention(dev, torch.from_numpy(q).cuda(), i32([0, 2]), i32([n]), i32(used[None]), out, 2, n, ws)
    check_attention(out, kv4.attention(small, q, [0, 2], [n], np.array([[0, 1, 2]])), "f32")


# ------------------------------------------------------------------------------------------- plan

def run_plan(B, page, length, new, table, ring, free, n_tok, pages, keep=None, alias=False):
    n = len(length)
    t = {"len_in": i32(length), "table": i32(table), "ring": i32(ring), "free_in": i32(free)}
    out = {k: torch.full((m,), -77, dtype=torch.int32, device="cuda") for k, m in
           (("len", n), ("free", 2), ("cu", n + 1), ("slot", n_tok), ("pos", n_tok), ("seq", n_tok), ("status", 1))}
    if alias:
        out["len"], out["free"] = t["len_in"], t["free_in"]
    B.stage_op_kv4_plan(page, t["len_in"], i32(new), t["table"], t["ring"], t["free_in"], out["len"], out["free"], out["cu"], out["slot"], out["pos"],
                        out["seq"], out["status"], keep_len=None if keep is None else i32(keep), n_pages=pages)
    torch.cuda.synchronize()
    r = {k: x.cpu().numpy() for k, x in out.items()}
    r["table"], r["ring"], r["status"] = t["table"].cpu().numpy(), t["ring"].cpu().numpy(), int(r["status"][0])
    return r


def check_plan(got, want):
    assert got["status"] == want["status"]
    for k in ("len", "free", "cu", "slot", "pos", "seq", "table", "ring"):
        same(got[k], np.asarray(want[k], np.int32))


@pytest.mark.parametrize("n,page,new_max,n_tok", [(1, 16, 1, 1), (7, 64, 3, 40), (600, 16, 40, 20000), (1500, 32, 3, 3000), (5000, 16, 9, 25000), (64, 128, 5000, 200000)])
def test_plan_over_steps(B, n, page, new_max, n_tok):
    rng = np.random.default_rng(n)
    stride = -(-4 * new_max // page) + 2
    pages = n * stride // 2 + stride
    table = np.full((n, stride), -1, np.int32)
    ring, free, length = rng.permutation(pages).astype(np.int32), np.array([pages // 3, pages], np.int32), np.zeros(n, np.int32)
    for step in range(6):
        keep = np.where(rng.random(n) < 0.2, 0, length - np.minimum(length, rng.integers(0, 5, n))).astype(np.int32)
        new = np.where(rng.random(n) < 0.5, rng.integers(0, new_max + 1, n), 1).astype(np.int32)
        new = np.minimum(new, stride * page - keep).astype(np.int32)
        want = kv4.plan(page, length, new, table, ring, free, n_tok, pages, keep)
        check_plan(run_plan(B, page, length, new, table, ring, free, n_tok, pages, keep, alias=step % 2 == 1), want)
        length, table, ring, free = want["len"], want["table"], want["ring"], want["free"]


def test_plan_refuses_a_step_as_a_whole(B):
    page, table = 16, np.arange(12, dtype=np.int32).reshape(3, 4)
    ring, ok = np.arange(12, 20, dtype=np.int32), [3, 8]
    cases = [  # length, keep, new, free state, n_tok
        ([10, 20, 64], None, [1, 1, 0], ok, 9),              # fine
        ([10, 20, 64], None, [1, 1, 1], ok, 9),              # the third is beyond its row
        ([10, -1, 0], None, [1, 1, 1], ok, 9),
        ([10, 20, 0], [10, 21, 0], [1, 1, 1], ok, 9),        # keeps more than it has
        ([10, 20, 0], [10, -1, 0], [1, 1, 1], ok, 9),
        ([10, 20, 0], None, [1, -1, 1], ok, 9),
        ([10, 20, 0], None, [4, 5, 1], ok, 9),               # ten tokens
        ([10, 20, 0], None, [4, 2 ** 31 - 1, 1], ok, 9),
        ([0, 0, 0], None, [30, 30, 30], [3, 5], 99),         # six pages of five
        ([0, 0, 0], None, [30, 30, 30], [3, 6], 99),         # fine: all of them
        ([10, 20, 0], None, [1, 1, 1], [8, 1], 9),           # a head beyond the ring
        ([10, 20, 0], None, [1, 1, 1], [0, 9], 9),
        ([10, 20, 0], [0, 0, 0], [0, 0, 0], [0, 6], 9),      # three pages back: one more than fits
        ([10, 20, 0], [0, 0, 0], [0, 0, 0], [2, 5], 9),      # fine
        ([2 ** 31 - 1, 20, 0], None, [1, 1, 1], ok, 9),
        ([0, 20, 0], None, [0, 0, 0], ok, 9),                # no token at all
        ([0, 20, 0], None, [0, 0, 0], ok, 0),                # and no slot map
    ]
    seen = []
    for length, keep, new, free, n_tok in cases:
        want = kv4.plan(page, np.array(length, np.int32), new, table, ring, np.array(free, np.int32), n_tok, 20, keep)
        check_plan(run_plan(B, page, length, new, table, ring, free, n_tok, 20, keep), want)
        seen.append(want["status"])
    assert seen == [0, 2, 2, 2, 2, 2, 3, 3, 1, 0, 2, 2, 2, 0, 2, 0, 0]


@pytest.mark.parametrize("n", [40, 3000, 9000])
def test_plan_with_long_runs_of_idle_requests(B, n):
    """A few requests with hundreds of tokens and pages each, among thousands without any."""
    rng = np.random.default_rng(n)
    page, stride = 16, 64
    length = np.where(rng.random(n) < 0.5, rng.integers(0, 200, n), 0).astype(np.int32)
    have = -(-length // page)
    table = np.full((n, stride), -1, np.int32)
    ids = rng.permutation(int(have.sum()) + 600).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(have)])
    for i in range(n):
        table[i, :have[i]] = ids[at[i]:at[i + 1]]
    ring = np.full(len(ids), -9, np.int32)
    ring[5:605] = ids[at[-1]:]
    new, keep = np.zeros(n, np.int32), length.copy()
    busy = rng.choice(n, 12, replace=False)
    new[busy[:8]] = rng.integers(300, 800, 8)
    keep[busy[6:]] = 0
    want = kv4.plan(page, length, new, table, ring, np.array([5, 600], np.int32), 7000, len(ids), keep)
    assert want["status"] == 0
    check_plan(run_plan(B, page, length, new, table, ring, [5, 600], 7000, len(ids), keep), want)


def test_a_large_plan_captured_and_replayed(B):
    """A cluster launch in a graph; lengths and ring go on from replay to replay."""
    rng = np.random.default_rng(17)
    n, page, stride, n_tok = 1500, 16, 8, 3000
    length = rng.integers(0, 60, n).astype(np.int32)
    have = -(-length // page)
    ids = rng.permutation(n * stride).astype(np.int32)
    table, at = np.full((n, stride), -1, np.int32), np.concatenate([[0], np.cumsum(have)])
    for i in range(n):
        table[i, :have[i]] = ids[at[i]:at[i + 1]]
    ring, free = np.resize(ids[at[-1]:], n * stride).astype(np.int32), np.array([0, n * stride - at[-1]], np.int32)
    new = rng.integers(0, 4, n).astype(np.int32)
    new[np.cumsum(new) > n_tok] = 0
    t = {k: i32(x) for k, x in (("len", length), ("new", new), ("table", table), ("ring", ring), ("free", free), ("cu", np.zeros(n + 1)),
                                ("slot", np.zeros(n_tok)), ("pos", np.zeros(n_tok)), ("seq", np.zeros(n_tok)), ("status", np.full(1, -1)))}

    def step():
        B.stage_op_kv4_plan(page, t["len"], t["new"], t["table"], t["ring"], t["free"], t["len"], t["free"], t["cu"], t["slot"], t["pos"], t["seq"],
                            t["status"])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        want = kv4.plan(page, length, new, table, ring, free, n_tok, n * stride)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: x.cpu().numpy() for k, x in t.items()}
        check_plan({**got, "status": int(got["status"][0])}, want)
        length, table, ring, free = want["len"], want["table"], want["ring"], want["free"]
    assert want["status"] == 0


def test_plan_refuses_positions_beyond_31_bits(B):
    """Table rows may be wider than positions can be counted."""
    page, stride = 4096, (1 << 31) // 4096 + 1
    table, ring = np.zeros((1, stride), np.int32), np.arange(2, dtype=np.int32)
    for new, status in ((1, 0), (2, 2), (5, 2)):
        length = np.array([2 ** 31 - 2], np.int32)
        want = kv4.plan(page, length, [new], table, ring, np.array([0, 2], np.int32), 8, 2)
        assert want["status"] == status
        check_plan(run_plan(B, page, length, [new], table, ring, [0, 2], 8, 2), want)


def test_plan_gives_no_slot_of_a_page_outside_the_cache(B):
    table = np.array([[5, 99, -3, 7]], np.int32)
    length, new = np.array([10], np.int32), [50]
    want = kv4.plan(16, length, new, table, np.array([1, 99, 2, 3], np.int32), np.array([0, 4], np.int32), 60, 8)
    got = run_plan(B, 16, length, new, table, np.array([1, 99, 2, 3], np.int32), [0, 4], 60, 8)
    check_plan(got, want)
    assert (got["slot"][22:38] == -1).all() and (got["slot"][:22] >= 0).all()


def test_plan_of_no_request(B):
    got = run_plan(B, 16, np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 4), np.int32), np.arange(3, dtype=np.int32), [1, 2], 4, 3)
    assert got["status"] == 0 and got["cu"].tolist() == [0] and (got["slot"] == -1).all() and got["free"].tolist() == [1, 2]


# ------------------------------------------------------------------------------------------- attention

def attention_case(rng, hkv, group, d, page, rows, dtype, wide=1.0, extra=3, qwide=1.0):
    """rows: (query tokens, positions) per sequence; pages shuffled; what lies behind a sequence's last position is noise
    with NaN scales among it."""
    need = [-(-n // page) for _, n in rows]
    pages = sum(need) + 2
    cache, _ = random_cache(rng, pages, page, hkv, d, wide)
    ids = rng.permutation(pages)
    table = np.full((len(rows), max(need + [1]) + 1), -1, np.int32)
    at = 0
    dims, blocks = np.arange(d), np.arange(d // 32)
    for i, (_, n) in enumerate(rows):
        table[i, :need[i]] = ids[at:at + need[i]]
        at += need[i]
        for p in range(n, need[i] * page):
            page_id, off = table[i, p // page], p % page
            for is_v in (False, True):
                sp = kv4.scale_place(off % 16, blocks, d, is_v)
                cache[page_id, :, off // 16, sp] = 0xFF
                cache[page_id, :, off // 16, sp + 1] = rng.choice([0x7F, 0x7C, 0xFF, 0x40])
    cu = np.concatenate([[0], np.cumsum([q for q, _ in rows])]).astype(np.int32)
    q = as_given(rng.standard_normal((cu[-1] + extra, hkv * group, d)) * qwide, dtype)
    return cache, table, cu, np.array([n for _, n in rows], np.int32), q


def run_attention(B, cache, table, cu, length, q, dtype, max_q=None, max_len=None, ws=None, dev=None):
    dev = torch.from_numpy(cache).cuda() if dev is None else dev
    n_tok, hq, d = q.shape
    pad = hq * d + 16
    fused = torch.zeros(n_tok, pad, dtype=DT[dtype], device="cuda")
    qd = fused[:, 8: 8 + hq * d].unflatten(1, (hq, d))
    qd.copy_(torch.as_tensor(q))
    out = torch.full((n_tok, pad), 3.0, dtype=DT[dtype], device="cuda")
    od = out[:, 16:].unflatten(1, (hq, d))
    max_q = max_q or max(1, int(np.diff(cu).max()))
    max_len = max_len or max(1, int(length.max()))
    if ws is None:
        ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(len(length), hq, cache.shape[1], d, max_q, max_len), dtype=torch.uint8, device="cuda")
    B.stage_op_kv4_attention(dev, qd, i32(cu), i32(length), i32(table), od, max_q, max_len, ws)
    torch.cuda.synchronize()
    assert (out[:, :16] == 3).all()
    assert (od[int(cu[-1]):] == 3).all()            # rows behind the last sequence stay
    return od


CASES = [
    # hkv, group, d, page, (query tokens, positions)
    (2, 4, 128, 16, [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17)]),
    (1, 8, 128, 64, [(1, 63), (1, 64), (1, 65), (1, 300)]),
    (2, 1, 64, 16, [(1, 33), (0, 20), (1, 500)]),
    (3, 2, 64, 48, [(1, 100), (1, 47)]),
    (1, 3, 128, 32, [(1, 77), (2, 31)]),
    (1, 7, 64, 32, [(1, 200), (3, 90)]),
    (1, 16, 128, 64, [(1, 129), (2, 70)]),
    (2, 5, 128, 16, [(4, 4), (5, 50), (1, 1)]),
    (2, 4, 128, 32, [(3, 40), (8, 300), (0, 9), (1, 0), (2, 1), (4, 2)]),     # tokens before the first position
    (1, 40, 64, 16, [(1, 50)]),
    (8, 4, 128, 64, [(1, 1000), (1, 37)]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hkv,group,d,page,rows", CASES)
def test_attention_matches_oracle(B, hkv, group, d, page, rows, dtype):
    rng = np.random.default_rng(hkv * 1000 + group * 10 + d)
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype)
    out = run_attention(B, cache, table, cu, length, q, dtype)
    check_attention(out, kv4.attention(cache, q, cu, length, table), dtype)


CHUNKS = [
    (2, 4, 128, 64, [(130, 130), (97, 300)]),
    (1, 8, 128, 16, [(64, 64), (33, 33), (1, 200)]),
    (2, 1, 64, 32, [(200, 257)]),
    (1, 4, 64, 64, [(150, 100), (70, 70)]),               # more tokens than positions
    (1, 3, 128, 48, [(61, 190), (0, 5), (129, 129)]),
    (1, 2, 128, 128, [(65, 700)]),
    (1, 16, 64, 16, [(40, 90)]),
    (1, 1, 128, 16, [(300, 300)]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hkv,group,d,page,rows", CHUNKS)
def test_chunks_match_oracle(B, hkv, group, d, page, rows, dtype):
    rng = np.random.default_rng(hkv * 1000 + group * 10 + d + 7)
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype)
    out = run_attention(B, cache, table, cu, length, q, dtype)
    check_attention(out, kv4.attention(cache, q, cu, length, table), dtype)


@pytest.mark.parametrize("rows", [[(1, 600)], [(40, 600)]])
@pytest.mark.parametrize("hkv,group,d", [(1, 4, 128), (1, 8, 64)])
def test_scales_and_scores_over_a_wide_range(B, hkv, group, d, rows):
    """V rows from 1e-6 to 1e5 and scores up to a few hundred: the largest scale does not swallow what the
    probabilities single out."""
    rng = np.random.default_rng(21)
    page, n = 32, 600
    cache = kv4.cache_array(20, page, hkv, d)
    slots = rng.permutation(20 * page)[:page * 19]
    table = rng.permutation(20)[None, :19].astype(np.int32)
    slots = (table[0][np.arange(n) // page] * page + np.arange(n) % page)
    k = rng.standard_normal((n, hkv, d)) * 3
    v = rng.standard_normal((n, hkv, d)) * 10.0 ** rng.integers(-6, 6, (n, hkv, 1))
    kv4.append(cache, k.astype(np.float32), v.astype(np.float32), slots)
    c = rows[0][0]
    q = as_given(rng.standard_normal((c, hkv * group, d)) * 10.0 ** rng.integers(-3, 2, (c, hkv * group, 1)), "f32")
    q[0, 0] = 0
    cu, length = np.array([0, c], np.int32), np.array([n], np.int32)
    out = run_attention(B, cache, table, cu, length, q, "f32")
    check_attention(out, kv4.attention(cache, q, cu, length, table), "f32", chunk=c > 1)


@pytest.mark.parametrize("qtok", [1, 33])
def test_nan_rows_stay_where_they_belong(B, qtok):
    """A NaN in K makes its KV head's outputs NaN; one in V only its own block of dims; other heads and
    sequences, and tokens that do not see it, keep their values."""
    rng = np.random.default_rng(31)
    hkv, group, d, page, n = 2, 2, 128, 16, 100
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, [(qtok, n), (qtok, 60)], "f32")
    clean = kv4.attention(cache, q, cu, length, table)
    last = n - 1
    tile = cache[table[0, last // page], :, last % page // 16]
    ks, vs = (int(kv4.scale_place(last % 16, 1, d, is_v)) for is_v in (False, True))
    tile[0, ks:ks + 2] = [0xFF, 0x7F]
    tile[1, vs:vs + 2] = [0xFF, 0x7F]
    got = run_attention(B, cache, table, cu, length, q, "f32").cpu().numpy()
    hit = np.zeros(q.shape, bool)
    hit[qtok - 1, :group] = True                        # K of head 0: the last token sees it
    hit[qtok - 1, group:, 32:64] = True                 # V of head 1, block 1
    assert np.isnan(got[hit]).all()
    some = ~np.isnan(clean[0]) & ~hit
    check_attention(torch.from_numpy(got), clean, "f32", some)


def test_bad_page_ids_count_as_absent(B):
    rng = np.random.default_rng(41)
    for rows in ([(1, 150), (2, 100)], [(40, 150), (35, 100)]):
        cache, table, cu, length, q = attention_case(rng, 2, 4, 128, 16, rows, "f32")
        table[0, [1, 4]] = [-1, cache.shape[0]]
        table[1, :] = [2 ** 31 - 1, -2 ** 31, -7, 10 ** 6, -1, 1 << 30, -1] + [-1] * (table.shape[1] - 7)
        out = run_attention(B, cache, table, cu, length, q, "f32")
        check_attention(out, kv4.attention(cache, q, cu, length, table), "f32")
        assert (out[int(cu[1]):int(cu[2])] == 0).all()


def test_lengths_beyond_the_stated_bounds(B):
    """seq_len counts as at most max_len and the table's positions; tokens behind max_q get no output."""
    rng = np.random.default_rng(43)
    cache, table, cu, length, q = attention_case(rng, 1, 4, 64, 16, [(1, 90), (6, 40)], "f32")
    out = run_attention(B, cache, table, cu, length, q, "f32", max_q=2, max_len=64)
    ref = kv4.attention(cache, q, cu, np.array([64, 40]), table, max_q=2)
    check_attention(out, ref, "f32")
    assert (out[3:7] == 3).all()
    out = run_attention(B, cache, table[:, :3].copy(), cu, np.array([10 ** 9, 40], np.int32), q, "f32", max_len=1 << 20)
    check_attention(out, kv4.attention(cache, q, cu, np.array([48, 40]), table[:, :3]), "f32")
    out = run_attention(B, cache, table, cu, np.array([-5, 40], np.int32), q, "f32", max_len=64)
    assert (out[0] == 0).all()


def test_one_long_sequence(B):
    """20011 positions, split over the GPU; twice the same bits, also with another call in between."""
    rng = np.random.default_rng(51)
    cache, table, cu, length, q = attention_case(rng, 2, 4, 128, 64, [(1, 20011)], "f32", extra=0)
    dev = torch.from_numpy(cache).cuda()
    ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(1, 8, 2, 128, 1, 20011), dtype=torch.uint8, device="cuda")
    out = run_attention(B, cache, table, cu, length, q, "f32", ws=ws, dev=dev)
    check_attention(out, kv4.attention(cache, q, cu, length, table), "f32")
    run_attention(B, cache, table, cu, np.array([777], np.int32), q, "f32", max_len=20011, ws=ws, dev=dev)
    again = run_attention(B, cache, table, cu, length, q, "f32", ws=ws, dev=dev)
    same(out.cpu().numpy(), again.cpu().numpy())


def test_many_ragged_sequences(B):
    rng = np.random.default_rng(61)
    rows = [(1, int(n)) for n in rng.integers(1, 700, 60)]
    cache, table, cu, length, q = attention_case(rng, 2, 8, 128, 32, rows, "f32")
    out = run_attention(B, cache, table, cu, length, q, "f32")
    check_attention(out, kv4.attention(cache, q, cu, length, table), "f32")


def test_two_streams_with_a_workspace_each(B):
    rng = np.random.default_rng(71)
    cases = [attention_case(rng, 2, 4, 128, 32, [(1, 3000)], "f32", extra=0) for _ in range(2)]
    streams, work, held = [torch.cuda.Stream() for _ in cases], [], []
    for cache, table, cu, length, q in cases:
        ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(1, 8, 2, 128, 1, 3000), dtype=torch.uint8, device="cuda")
        work.append((torch.from_numpy(cache).cuda(), torch.as_tensor(q).float().cuda(), i32(cu), i32(length), i32(table), ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (dev, q, cu, length, table, ws) in zip(streams, work):
            out = torch.zeros_like(q)
            torch.cuda.synchronize()
            held.append(out)
        for s, (dev, q, cu, length, table, ws), out in zip(streams, work, held[-2:]):
            B.stage_op_kv4_attention(dev, q, cu, length, table, out, 1, 3000, ws, stream=s)
    torch.cuda.synchronize()
    for i, out in enumerate(held):
        cache, table, cu, length, q = cases[i % 2]
        check_attention(out, kv4.attention(cache, q, cu, length, table), "f32")


def test_one_workspace_for_chunks_and_decode_in_turn(B):
    """A workspace of the larger size serves calls of both sizes one after another: each leaves it ready for the next."""
    rng = np.random.default_rng(75)
    few = attention_case(rng, 2, 4, 128, 32, [(1, 3000)], "f32", extra=0)
    many = attention_case(rng, 2, 4, 128, 32, [(60, 2100)], "f32", extra=0)
    size = max(B.stage_op_kv4_attention_workspace_bytes(1, 8, 2, 128, q, 3000) for q in (1, 60))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for cache, table, cu, length, q in (few, many, few, many, many, few):
        out = run_attention(B, cache, table, cu, length, q, "f32", ws=ws)
        check_attention(out, kv4.attention(cache, q, cu, length, table), "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hkv,group,d,rows", [(1, 4, 128, [(70, 1500)]), (2, 1, 64, [(40, 2000), (0, 7), (36, 500)]), (1, 8, 128, [(40, 40), (33, 3000)])])
def test_few_row_tiles_share_their_positions_out(B, hkv, group, d, rows, dtype):
    """Few row tiles over long contexts: the positions of a tile are shared out, some parts are empty for short sequences,
    and a NaN in V reaches the rows and dims that it reaches otherwise."""
    rng = np.random.default_rng(77 + d)
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, 16, rows, dtype)
    out = run_attention(B, cache, table, cu, length, q, dtype)
    want = kv4.attention(cache, q, cu, length, table)
    check_attention(out, want, dtype)
    at = int(length[0]) // 2
    vs = int(kv4.scale_place(at % 16, 0, d, True))
    cache[table[0, at // 16], 0, 0, vs:vs + 2] = [0xFF, 0x7F]
    got = run_attention(B, cache, table, cu, length, q, dtype).double().cpu().numpy()
    hit = np.zeros(q.shape, bool)
    first = max(0, at - (int(length[0]) - rows[0][0]))
    hit[first:rows[0][0], :group, :32] = True
    assert np.isnan(got[hit]).all()
    check_attention(torch.from_numpy(got), want, dtype, ~np.isnan(want[0]) & ~hit)


def with_loose_bounds(monkeypatch, empty):
    """Attention called with a bound on the lengths far above them, and with `empty` sequences more that have no token: the
    launch is chosen by the bounds, so chunks of any length run on the tiles for many columns -- their positions shared out
    over the GPU without empty sequences, in one part each with many."""
    tight = run_attention

    def loose(B, cache, table, cu, length, q, dtype, max_q=None, max_len=None, **kw):
        max_q = max_q or max(1, int(np.diff(cu).max()))
        cu = np.concatenate([cu, np.full(empty, cu[-1], np.int32)])
        length = np.concatenate([length, np.zeros(empty, np.int32)])
        table = np.concatenate([table, np.full((empty, table.shape[1]), -1, np.int32)])
        return tight(B, cache, table, cu, length, q, dtype, max_q=max_q, max_len=max_len or 1 << 28, **kw)

    monkeypatch.setitem(globals(), "run_attention", loose)


@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hkv,group,d,page,rows", CHUNKS)
def test_chunks_match_oracle_under_loose_bounds(B, monkeypatch, hkv, group, d, page, rows, dtype, empty):
    rng = np.random.default_rng(hkv * 1000 + group * 10 + d + 9)
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype)
    with_loose_bounds(monkeypatch, empty)
    out = run_attention(B, cache, table, cu, length, q, dtype)
    check_attention(out, kv4.attention(cache, q, cu, length, table), dtype, chunk=True)


@pytest.mark.parametrize("empty", [0, 160])
def test_hard_chunks_under_loose_bounds(B, monkeypatch, empty):
    """Wide ranges, NaN rows and bad pages, on the tiles for many columns."""
    with_loose_bounds(monkeypatch, empty)
    test_scales_and_scores_over_a_wide_range(B, 1, 4, 128, [(40, 600)])
    test_scales_and_scores_over_a_wide_range(B, 1, 8, 64, [(40, 600)])
    test_nan_rows_stay_where_they_belong(B, 33)
    test_bad_page_ids_count_as_absent(B)
    for dtype in DT:
        test_few_row_tiles_share_their_positions_out(B, 1, 4, 128, [(70, 1500)], dtype)
        test_few_row_tiles_share_their_positions_out(B, 2, 1, 64, [(40, 2000), (0, 7), (36, 500)], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,max_len", [([(1, 3000), (2, 40)], 3000), ([(40, 900), (33, 33)], 1 << 28)])
def test_the_output_in_the_place_of_q(B, rows, max_len, dtype):
    """Rows that several CTAs share (long, and chunks in parts) read their q before any of it is written."""
    rng = np.random.default_rng(91)
    cache, table, cu, length, q = attention_case(rng, 2, 4, 128, 16, rows, dtype)
    apart = run_attention(B, cache, table, cu, length, q, dtype, max_len=max_len)
    qd, most = torch.as_tensor(q).to(DT[dtype]).cuda(), max(c for c, _ in rows)
    ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(2, 8, 2, 128, most, max_len), dtype=torch.uint8, device="cuda")
    B.stage_op_kv4_attention(torch.from_numpy(cache).cuda(), qd, i32(cu), i32(length), i32(table), qd, most, max_len, ws)
    same(qd[:int(cu[-1])].float().cpu().numpy(), apart[:int(cu[-1])].float().cpu().numpy())


@pytest.mark.parametrize("max_q", [1, 1 << 20])
def test_a_loose_bound_on_the_tokens(B, max_q):
    """Each of 200 sequences has one token, whatever the bound says: at most the call's tokens count."""
    rng = np.random.default_rng(81)
    rows = [(1, int(n)) for n in rng.integers(1, 90, 200)]
    cache, table, cu, length, q = attention_case(rng, 2, 4, 64, 16, rows, "f32")
    out = run_attention(B, cache, table, cu, length, q, "f32", max_q=max_q)
    check_attention(out, kv4.attention(cache, q, cu, length, table), "f32", chunk=True)


# ------------------------------------------------------------------------------------------- refusals through the binding

def test_binding_refusals(B):
    dev = torch.zeros(B.stage_op_kv4_cache_shape(4, 16, 2, 64), dtype=torch.uint8, device="cuda")
    k = torch.zeros(3, 2, 64, device="cuda")
    slot = torch.zeros(3, dtype=torch.int32, device="cuda")
    good = dict(cache=dev, k=k, v=k, slot=slot)
    for kw in (dict(slot=slot.long()), dict(slot=slot[:2]), dict(v=k.half()), dict(v=k[:2]), dict(k=k.double()), dict(k=k[..., :32]), dict(v=k.cpu()),
               dict(k=torch.zeros(3, 64, 2, device="cuda").transpose(1, 2)), dict(cache=dev[:, :1])):
        with pytest.raises(B.StageError) as e:
            B.stage_op_kv4_append(**{**good, **kw})
        assert e.value.code == B.STAGE_E_INVALID, kw
    q = torch.zeros(3, 4, 64, device="cuda")
    ws = torch.zeros(B.STAGE_KV4_SCRATCH_MAX, dtype=torch.uint8, device="cuda")
    good = dict(cache=dev, q=q, cu_q=i32([0, 1, 3]), seq_len=i32([5, 6]), table=i32([[0], [1]]), out=torch.zeros_like(q), max_q=2, max_len=16, workspace=ws)
    B.stage_op_kv4_attention(**good)
    for kw in (dict(cu_q=i32([0, 3])), dict(out=q.half()), dict(out=q[:2]), dict(table=i32([[0]])), dict(table=i32([0, 1])), dict(workspace=ws[:0]),
               dict(max_q=0), dict(max_len=0), dict(q=q[:, :3], out=torch.zeros_like(q)[:, :3]), dict(seq_len=i32([5, 6]).long()), dict(workspace=ws.cpu())):
        with pytest.raises(B.StageError) as e:
            B.stage_op_kv4_attention(**{**good, **kw})
        assert e.value.code == B.STAGE_E_INVALID, kw
    one = i32([0])
    good = dict(page_len=16, seq_len=one, new_len=one, table=i32([[0]]), free_ring=i32([0, 1]), free_state=i32([0, 1]), seq_len_out=i32([0]), free_state_out=i32([0, 0]),
                cu_new=i32([0, 0]), slot=i32([0]), pos=i32([0]), seq=i32([0]), status=i32([0]))
    B.stage_op_kv4_plan(**good)
    for kw in (dict(page_len=15), dict(cu_new=one), dict(status=i32([0, 0])), dict(pos=i32([0, 0])), dict(table=i32([0])), dict(new_len=one.long()),
               dict(keep_len=i32([0, 0])), dict(n_pages=0), dict(free_state=i32([0]))):
        with pytest.raises(B.StageError) as e:
            B.stage_op_kv4_plan(**{**good, **kw})
        assert e.value.code == B.STAGE_E_INVALID, kw
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------- together

class Server:
    """The device state of a small serving loop: plan, append and attention of one block, step after step."""

    def __init__(self, B, n, page, hkv, group, d, pages, stride, n_tok, dtype, max_q, seed):
        self.B, self.page, self.dtype, self.max_q, self.max_len = B, page, dtype, max_q, stride * page
        rng = np.random.default_rng(seed)
        self.cache = torch.full(B.stage_op_kv4_cache_shape(pages, page, hkv, d), 0xFF, dtype=torch.uint8, device="cuda")
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.len, self.keep, self.new, self.table = z(n), z(n), z(n), torch.full((n, stride), -1, dtype=torch.int32, device="cuda")
        self.ring, self.free = i32(rng.permutation(pages)), i32([0, pages])
        self.cu, self.slot, self.pos, self.seq, self.status = z(n + 1), z(n_tok), z(n_tok), z(n_tok), z(1)
        self.k, self.v = (torch.zeros(n_tok, hkv, d, dtype=DT[dtype], device="cuda") for _ in range(2))
        self.q = torch.zeros(n_tok, hkv * group, d, dtype=DT[dtype], device="cuda")
        self.out = torch.zeros_like(self.q)
        self.ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(n, hkv * group, hkv, d, max_q, self.max_len), dtype=torch.uint8, device="cuda")

    def launch(self):
        B = self.B
        B.stage_op_kv4_plan(self.page, self.len, self.new, self.table, self.ring, self.free, self.len, self.free, self.cu, self.slot, self.pos, self.seq,
                            self.status, keep_len=self.keep)
        B.stage_op_kv4_append(self.cache, self.k, self.v, self.slot)
        B.stage_op_kv4_attention(self.cache, self.q, self.cu, self.len, self.table, self.out, self.max_q, self.max_len, self.ws)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,hkv,group,d,page", [("f32", 2, 4, 128, 32), ("bf16", 1, 8, 64, 16)])
def test_a_serving_loop(B, graph, dtype, hkv, group, d, page):
    """Prompts enter, tokens are decoded, drafts rolled back, requests leave; eagerly and as one captured graph replayed
    while everything grows.  The expected output comes from lists of rows per request, which know no pages."""
    n, stride, n_tok, max_q = 5, 10, 160, 100
    pages = 5 * stride - 9
    s = Server(B, n, page, hkv, group, d, pages, stride, n_tok, dtype, max_q, 81)
    s.launch()                                     # nothing to do: no request has a token
    torch.cuda.synchronize()
    assert s.status.item() == 0 and (s.out == 0).all()
    g = None
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.launch()
    rng = np.random.default_rng(82)
    rows = [[] for _ in range(n)]                  # per request: (k, v) rows as given
    refused = 0
    for step in range(24):
        keep = np.array([len(r) for r in rows])
        new = np.ones(n, int)
        for i in range(n):
            what = rng.random()
            if not rows[i] or what < 0.12:         # leave, and another prompt enters
                keep[i], new[i] = 0, rng.integers(1, 60 if step else max_q)
            elif what < 0.3:
                keep[i], new[i] = max(0, keep[i] - 3), rng.integers(0, 6)
            new[i] = min(new[i], stride * page - keep[i])
        total = int(new.sum())
        k, v, q = (as_given(rng.standard_normal((n_tok, h, d)), dtype) for h in (hkv, hkv, hkv * group))
        s.k.copy_(torch.as_tensor(k)), s.v.copy_(torch.as_tensor(v)), s.q.copy_(torch.as_tensor(q))
        s.keep.copy_(i32(keep)), s.new.copy_(i32(new))
        s.out.fill_(5)
        g.replay() if graph else s.launch()
        torch.cuda.synchronize()
        if s.status.item():                        # refused as a whole: nothing changed
            refused += 1
            assert (s.out == 5).all() and s.len.tolist() == [len(r) for r in rows]
            continue
        cu = np.concatenate([[0], np.cumsum(new)])
        assert s.cu.tolist() == cu.tolist() and s.len.tolist() == (keep + new).tolist()
        for i in range(n):
            rows[i] = rows[i][:keep[i]] + [(k[t], v[t]) for t in range(cu[i], cu[i + 1])]
        flat = kv4.cache_array(n * stride, page, hkv, d)
        table = np.arange(n * stride, dtype=np.int32).reshape(n, stride)
        for i in range(n):
            if rows[i]:
                kv4.append(flat, np.stack([r[0] for r in rows[i]]), np.stack([r[1] for r in rows[i]]), i * stride * page + np.arange(len(rows[i])))
        want = kv4.attention(flat, q[:total], cu, [len(r) for r in rows], table)
        check_attention(s.out[:total], want, dtype)
        assert (s.out[total:] == 5).all()
    assert refused < 12


def test_captured_graphs_with_their_own_workspaces_replayed_in_turn(B):
    rng = np.random.default_rng(91)
    graphs = []
    for i in range(2):
        cache, table, cu, length, q = attention_case(rng, 1, 4, 128, 32, [(1, 2000 + 50 * i)], "f32", extra=0)
        dev, qd, args = torch.from_numpy(cache).cuda(), torch.as_tensor(q).float().cuda(), (i32(cu), i32(length), i32(table))
        out = torch.zeros_like(qd)
        ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(1, 4, 1, 128, 1, 2100), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.stage_op_kv4_attention(dev, qd, *args, out, 1, 2100, ws)
        graphs.append((g, out, kv4.attention(cache, q, cu, length, table), (dev, qd, args, ws)))
    for _ in range(3):
        for g, out, want, _ in graphs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, out, want, _ in graphs:
            check_attention(out, want, "f32")
