"""Attention over the paged 4-bit cache where scales are infinite or spread far, where positions that a row does not see
hold large values, and where a CTA of the tiles for many columns goes from item to item.

The tolerances are those of tests/test_gpu_kv4.py, derived there, with two changes for the tiles for many columns.  K and V
are exact there (STAGE_BF16: rounded once to fp16, 2^-11 of themselves), whatever the block's scale, unless a scale of 4096 or
more shares the position; then a value is off by at most 2^-33 of the position's largest.  And the fp16 probabilities end at
2^-25 (half of the smallest step): with T_j the largest scale of position j (at least 2^-14), a probability stands as
x_j = 2^(z_j - r + e_j) against values v_j 2^-(e_j), where T_j is in 2^(e_j) * [2^10, 2^12) if each position has its own power and in
2^(e_j) * [2^7, 2^12) if a tile's positions share one.  The largest x_j is at least 2^11 (two fp16 values) or 2^7 (one), at a position
m, and divides by p_m 2^(e_m) / x_m at most, so dim d is off by at most
    sum_j 2^-25 |v_jd| 2^-(e_j) p_m 2^(e_m) / x_m <= 2^-34 max_j(p_j T_j) sum_j |v_jd| / T_j          (two)
                                                  <= 2^-27 max_j(p_j T_j) sum_j |v_jd| / T_j          (one).
"""
import numpy as np
import pytest

from oracle import kv4

torch = pytest.importorskip("torch")
from test_gpu_kv4 import DT, Server, as_given, attention_case, i32, run_attention, same  # noqa: E402

pytestmark = pytest.mark.gpu

WIDE_BOUND = 1 << 28   # a bound on the lengths that sends more than 24 columns to the tiles for many columns


@pytest.fixture(scope="module")
def B(cuda):
    from layer_range_stage_gb300 import binding
    return binding


def scales(cache, slots, is_v):
    """|scale| [n, heads, blocks] in float64 at valid slots."""
    tiles, nbytes = cache.shape[2:]
    d, page_len = nbytes // 18, tiles * 16
    slots = np.asarray(slots, np.int64)
    tile = cache[slots // page_len, :, slots % page_len // 16]
    sp = kv4.scale_place((slots % 16)[:, None], np.arange(d // 32)[None], d, is_v)[:, None]
    pick = lambda x: np.take_along_axis(tile, np.broadcast_to(x, tile.shape[:2] + (d // 32,)), -1).astype(np.uint16)  # noqa: E731
    return np.abs((pick(sp) | pick(sp + 1) << 8).view(np.float16).astype(np.float64))


def reference(cache, q, cu, seq_len, table):
    """As kv4.attention, a sequence and head at a time on the GPU in float64, and `small` [rows, heads, d]:
    max_j(p_j T_j) sum_j |v_jd| / T_j."""
    n_pages, hkv, tiles, nbytes = cache.shape
    d, page_len = nbytes // 18, tiles * 16
    group = q.shape[1] // hkv
    out = np.full(q.shape, np.nan)
    weight, small = np.zeros(q.shape), np.zeros(q.shape)
    spread = np.zeros(q.shape[:2])
    for i, n in enumerate(map(int, seq_len)):
        a, b = int(cu[i]), int(cu[i + 1])
        if a == b:
            continue
        at = np.arange(max(0, min(n, table.shape[1] * page_len)))
        page = table[i][at // page_len].astype(np.int64)
        at = at[(page >= 0) & (page < n_pages)]
        slots = table[i][at // page_len].astype(np.int64) * page_len + at % page_len
        with np.errstate(all="ignore"):
            k, v = (torch.from_numpy(kv4.rows(cache, slots, is_v)).cuda() for is_v in (False, True))
        top = torch.from_numpy(np.maximum(np.nan_to_num(scales(cache, slots, True)).max(-1, initial=0), 2.0 ** -14)).cuda()
        hidden = torch.from_numpy(at[None] > (n - (b - a) + np.arange(b - a))[:, None]).cuda()
        none = hidden.all(1)
        for h in range(q.shape[1]):
            kh, vh, th = k[:, h // group], v[:, h // group], top[:, h // group]
            qh = torch.from_numpy(np.ascontiguousarray(q[a:b, h])).cuda()
            if not len(at):
                out[a:b, h] = 0
                continue
            z = (qh @ kh.T / np.sqrt(d)).masked_fill(hidden, -np.inf)
            p = torch.softmax(z, -1).masked_fill(none[:, None], 0)
            seen = (~hidden).double()
            out[a:b, h] = (p @ vh).cpu().numpy()
            weight[a:b, h] = (p @ vh.abs()).cpu().numpy()
            spread[a:b, h] = ((qh.abs() @ kh.abs().T / np.sqrt(d)) * seen).amax(-1).cpu().numpy()
            small[a:b, h] = ((p * th).amax(-1, keepdim=True) * (seen @ (vh.abs() / th[:, None]))).cpu().numpy()
    return out, weight, spread, small


def check(got, ref, dtype, rows=None):
    out, weight, spread, small = ref
    got = got.detach().double().cpu().numpy() if torch.is_tensor(got) else got
    # 2^-33 of a position's largest, which only scales from 4096 on leave, is at most 2^-31 T_j: inside the terms of `small`
    tol = (2.0 ** -18 * spread[..., None] + 2.0 ** -16) * weight + 2.0 ** (-33 if dtype == "f32" else -27) * small
    if dtype != "f32":
        tol = tol + 2.0 ** -11 * weight + torch.finfo(DT[dtype]).eps / 2 * np.abs(out)
    if dtype == "f16":  # the output's own smallest step
        tol = tol + 2.0 ** -25
    if dtype == "bf16":
        tol = tol + (2.0 ** -11 + 2.0 ** -10 * spread[..., None]) * weight
    some = ~np.isnan(out) if rows is None else rows
    err = np.abs(got - out)[some]
    assert (err <= tol[some]).all(), (float((err / np.maximum(tol[some], 1e-300)).max()), np.argwhere(~(np.abs(got - out) <= tol) & some)[:4])


def tiled(B, cache, table, cu, length, q, dtype, empty=0, **kw):
    """The call on the tiles for many columns: in parts of the positions where there are few row tiles, in one part each with
    `empty` sequences more that have no token."""
    cu = np.concatenate([cu, np.full(empty, cu[-1], np.int32)])
    length = np.concatenate([length, np.zeros(empty, np.int32)])
    table = np.concatenate([table, np.full((empty, table.shape[1]), -1, np.int32)])
    return run_attention(B, cache, table, cu, length, q, dtype, max_len=WIDE_BOUND, **kw)


def put_scale(cache, table, i, pos, head, block, is_v, bits):
    d, page = cache.shape[3] // 18, cache.shape[2] * 16
    at = int(kv4.scale_place(pos % 16, block, d, is_v))
    cache[table[i, pos // page], head, pos % page // 16, at:at + 2] = [bits & 255, bits >> 8]


# ------------------------------------------------------------------------------------------- infinite scales

@pytest.mark.parametrize("bits", [0x7C00, 0xFC00])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("qtok,n,empty", [(1, 100, None), (1, 3000, None), (3, 200, None), (40, 200, 0), (40, 200, 160)])
def test_infinite_scales_count_as_nan(B, bits, dtype, qtok, n, empty):
    """An infinite scale in K makes NaN of the outputs that see it, of its KV head; one in V of its block's dims; other heads,
    sequences, dims and tokens keep their values, and the sign does not matter."""
    rng = np.random.default_rng(n + qtok)
    hkv, group, d = 2, 2, 128
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, 16, [(qtok, n), (qtok, 60)], dtype)
    clean = reference(cache, q, cu, length, table)
    put_scale(cache, table, 0, n - 1, 0, 1, False, bits)   # only the last token sees it
    put_scale(cache, table, 0, n - 1, 1, 1, True, bits)
    put_scale(cache, table, 1, 7, 0, 2, True, bits)        # all tokens of the second sequence
    run = run_attention if empty is None else lambda *a: tiled(*a, empty=empty)
    got = run(B, cache, table, cu, length, q, dtype).double().cpu().numpy()
    hit = np.zeros(q.shape, bool)
    hit[qtok - 1, :group] = True
    hit[qtok - 1, group:, 32:64] = True
    hit[qtok:2 * qtok, :group, 64:96] = True
    assert np.isnan(got[hit]).all()
    check(got, clean, dtype, ~np.isnan(clean[0]) & ~hit)


# ------------------------------------------------------------------------------------------- positions that a row does not see

@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,size", [(128, 2e-3), (64, 0.08), (128, 0.4)])
def test_large_keys_of_later_positions(B, dtype, d, size, empty):
    """The last tokens of a chunk have keys near the largest that the cache holds; the tokens before them, in the same tile of
    positions, do not see them and get what they get without them."""
    rng = np.random.default_rng(101)
    hkv, group, page, rows = 2, 4, 16, [(40, 61), (33, 126)]
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype, extra=0)
    for i, (c, n) in enumerate(rows):
        k = rng.standard_normal((n, hkv, d)) * size
        k[n - 3:] = rng.standard_normal((3, hkv, d)) * 1e5
        k = np.clip(k, -5e5, 5e5)
        v = rng.standard_normal((n, hkv, d))
        at = np.arange(n)
        kv4.append(cache, k.astype(np.float32), v.astype(np.float32), table[i][at // page] * page + at % page)
    q = as_given(q * (0.5 / size), dtype)      # scores of order 1 before the large keys
    out = tiled(B, cache, table, cu, length, q, dtype, empty=empty)
    check(out, reference(cache, q, cu, length, table), dtype)


@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_values_of_later_positions(B, dtype, d, empty):
    """The same for values: 1e-4 beside 4e5 that only the last tokens see."""
    rng = np.random.default_rng(103)
    hkv, group, page, rows = 2, 4, 16, [(40, 61), (33, 126)]
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype, extra=0)
    for i, (c, n) in enumerate(rows):
        v = rng.standard_normal((n, hkv, d)) * 1e-4
        v[n - 3:] = np.clip(rng.standard_normal((3, hkv, d)) * 1e5, -4e5, 4e5)
        if dtype == "f16":
            v[n - 3:] /= 16        # outputs that float16 holds
        at = np.arange(n)
        kv4.append(cache, rng.standard_normal((n, hkv, d)).astype(np.float32), v.astype(np.float32), table[i][at // page] * page + at % page)
    out = tiled(B, cache, table, cu, length, q, dtype, empty=empty)
    check(out, reference(cache, q, cu, length, table), dtype)


@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,by", [(128, "position"), (64, "position"), (128, "block"), (64, "block"), (128, "tile")])
def test_values_over_a_wide_range(B, dtype, d, by, empty):
    """V from 1e-6 to 1e4 from position to position, block to block or tile to tile, with scores that single positions out."""
    rng = np.random.default_rng(105)
    hkv, group, page, rows = 2, 4, 32, [(40, 300), (35, 130)]
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype, extra=0)
    for i, (c, n) in enumerate(rows):
        shape = {"position": (n, hkv, 1, 1), "block": (n, hkv, d // 32, 1), "tile": (n, hkv, 1, 1)}[by]
        power = rng.integers(-6, 4, shape)
        if by == "tile":
            power = power[np.arange(n) // 64 * 64]
        v = rng.standard_normal((n, hkv, d // 32, 32)) * 10.0 ** power
        v = np.clip(v, -3e4, 3e4).reshape(n, hkv, d)
        at = np.arange(n)
        kv4.append(cache, (2 * rng.standard_normal((n, hkv, d))).astype(np.float32), v.astype(np.float32), table[i][at // page] * page + at % page)
    q = as_given(q * 10.0 ** rng.integers(-2, 2, q.shape[:2] + (1,)), dtype)
    out = tiled(B, cache, table, cu, length, q, dtype, empty=empty)
    check(out, reference(cache, q, cu, length, table), dtype)


@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_keys_and_values_of_many_sizes(B, dtype, empty):
    """Keys and values from 1e-6 to 1e5: scores far beyond float32's exponentials, rows of zeros, subnormal scales."""
    rng = np.random.default_rng(107)
    hkv, group, d, page, rows = 2, 4, 128, 16, [(40, 300), (50, 64)]
    cache, table, cu, length, q = attention_case(rng, hkv, group, d, page, rows, dtype, extra=0)
    for i, (c, n) in enumerate(rows):
        k, v = (rng.standard_normal((n, hkv, d)) * 10.0 ** rng.integers(-6, 5, (n, hkv, 1)) for _ in range(2))
        k[n // 3], v[n // 2] = 0, 0
        if dtype == "f16":
            v = np.clip(v, -3e4, 3e4)
        at = np.arange(n)
        kv4.append(cache, k.astype(np.float32), v.astype(np.float32), table[i][at // page] * page + at % page)
    q = as_given(q * 10.0 ** rng.integers(-4, 1, q.shape[:2] + (1,)), dtype)
    out = tiled(B, cache, table, cu, length, q, dtype, empty=empty)
    check(out, reference(cache, q, cu, length, table), dtype)


# ------------------------------------------------------------------------------------------- from item to item

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_many_items_on_every_cta(B, dtype, d):
    """40 sequences of 8 KV heads, several hundred items: items without a tile, of one, two and more than sixteen follow one another
    on a CTA, with NaN in V, a K scale far above the others and absent pages in some of them."""
    rng = np.random.default_rng(109 + d)
    rows = [(int(rng.integers(40, 131)), int(rng.integers(60, 701))) for _ in range(36)]
    rows += [(100, 30), (0, 50), (1, 1300), (70, 1400)]
    rows = [rows[i] for i in rng.permutation(len(rows))]
    cache, table, cu, length, q = attention_case(rng, 8, 4, d, 16, rows, dtype)
    put_scale(cache, table, 3, int(length[3]) // 2, 2, 1, False, 0x7800)       # 32768
    at = rows.index((70, 1400))
    table[at, 40:44] = [-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31]
    bad, block = next(i for i in range(15, 40) if rows[i][0] > 60 and rows[i][1] > 200), 1
    want = reference(cache, q, cu, length, table)
    pos = rows[bad][1] - 30
    put_scale(cache, table, bad, pos, 5, block, True, 0x7FFF)
    out = run_attention(B, cache, table, cu, length, q, dtype).double().cpu().numpy()
    hit = np.zeros(q.shape, bool)
    hit[int(cu[bad]) + pos - (rows[bad][1] - rows[bad][0]):int(cu[bad + 1]), 20:24, 32 * block:32 * block + 32] = True
    assert np.isnan(out[hit]).all()
    check(out, want, dtype, ~np.isnan(want[0]) & ~hit)
    again = run_attention(B, cache, table, cu, length, q, dtype).double().cpu().numpy()
    same(out, again)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_long_items_follow_one_another(B, dtype):
    """Fewer sequences with long contexts: each CTA has a few items of dozens of tiles."""
    rng = np.random.default_rng(113)
    rows = [(300, 2500), (420, 420), (333, 1111), (512, 2000)]
    cache, table, cu, length, q = attention_case(rng, 8, 4, 128, 64, rows, dtype)
    out = run_attention(B, cache, table, cu, length, q, dtype)
    check(out, reference(cache, q, cu, length, table), dtype)


# ------------------------------------------------------------------------------------------- long sums

@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_sums_over_millions_of_positions(B, dtype, d, empty):
    """One page of values between 0.5 and 1, 4096 times in the table: with q = 0 every position weighs the same (an exact
    probability), so the output is the page's mean.  The tensor cores' additions drop 6e-7 of the sum per tile of 64 positions (as
    measured: 15 % over these when a chain of them had no end), 128 tiles 2^-13; the chains' sums are then added up in float32,
    2048 additions of 2^-24 each: 2^-13.  64 more tokens or fewer than the whole page move the mean by less than
    2^-18; bfloat16 rounds V to fp16, 2^-12 of itself; 2^-14 for the probabilities' sum and the division.  The output's rounding
    comes on top."""
    page, n = 4096, 4096 * 4096
    rng = np.random.default_rng(127)
    cache = kv4.cache_array(1, page, 1, d)
    kv4.append(cache, np.zeros((page, 1, d), np.float32), rng.uniform(0.5, 1, (page, 1, d)).astype(np.float32), np.arange(page))
    want = kv4.rows(cache, np.arange(page), True).mean(0)
    table = np.zeros((1, n // page), np.int32)
    out = tiled(B, cache, table, np.array([0, 40], np.int32), np.array([n], np.int32), np.zeros((40, 1, d)), dtype, empty=empty)
    got = out.double().cpu().numpy()
    tol = 2.0 ** -12 + 2.0 ** -14 + 2.0 ** -18 + (2.0 ** -12 if dtype == "bf16" else 0) + torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(got - want) <= tol * want).all(), (np.abs(got - want) / want).max()


# ------------------------------------------------------------------------------------------- one after another, captured, together

def on_tiles(B, n, n_tok, hq, hkv, d, dtype, max_q, max_len):
    return B.stage_op_kv4_attention_many(n, n_tok, hq, hkv, d, DT[dtype], max_q, max_len)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_workspace_for_both_kernels_in_turn(B, dtype):
    """Decode rows cut over the GPU, chunks in parts and chunks of many items one after another on one workspace: each leaves the
    arrival counters zero, and each call's rows are right."""
    rng = np.random.default_rng(131)
    few = attention_case(rng, 2, 4, 128, 32, [(1, 3000)], dtype, extra=0)
    parts = attention_case(rng, 2, 4, 128, 32, [(60, 2100)], dtype, extra=0)
    items = attention_case(rng, 2, 4, 128, 32, [(60, 300 + i) for i in range(160)], dtype, extra=0)
    size = max(B.stage_op_kv4_attention_workspace_bytes(160, 8, 2, 128, q, WIDE_BOUND) for q in (1, 60))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = {id(c): reference(c[0], c[4], c[2], c[3], c[1]) for c in (few, parts, items)}
    for case in (few, parts, few, items, few, items, parts, few):
        cache, table, cu, length, q = case
        bound = 3000 if case is few else WIDE_BOUND
        assert on_tiles(B, len(length), len(q), 8, 2, 128, dtype, int(np.diff(cu).max()), bound) == (case is not few)
        out = run_attention(B, cache, table, cu, length, q, dtype, ws=ws, max_len=bound)
        check(out, want[id(case)], dtype)
        assert (ws[:2048] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_chunks_with_their_own_workspaces_on_two_streams(B, dtype):
    """Chunk calls in two graphs, one in parts with its join, replayed at the same time; then with other lengths and queries."""
    rng = np.random.default_rng(137)
    graphs = []
    for rows in ([(60, 2000)], [(50, 300 + i) for i in range(90)]):
        cache, table, cu, length, q = attention_case(rng, 2, 4, 128, 32, rows, dtype, extra=0)
        n, most = len(rows), rows[0][0]
        assert on_tiles(B, n, len(q), 8, 2, 128, dtype, most, WIDE_BOUND)
        dev, qd, args = torch.from_numpy(cache).cuda(), torch.as_tensor(q).to(DT[dtype]).cuda(), (i32(cu), i32(length), i32(table))
        out = torch.zeros_like(qd)
        ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(n, 8, 2, 128, most, WIDE_BOUND), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.stage_op_kv4_attention(dev, qd, *args, out, most, WIDE_BOUND, ws)
        graphs.append((g, out, (cache, table, cu, length, q), (dev, qd, args, ws), torch.cuda.Stream()))
    for shorter in (0, 7):
        for g, out, (cache, table, cu, length, q), (dev, qd, args, ws), st in graphs:
            args[1].copy_(i32(length - shorter))
            qd.copy_(torch.as_tensor(np.roll(q, shorter, 0)))
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, out, case, held, st in graphs:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for g, out, (cache, table, cu, length, q), held, st in graphs:
            check(out, reference(cache, np.roll(q, shorter, 0), cu, length - shorter, table), dtype)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,hkv,group,d,page", [("f32", 2, 4, 128, 32), ("f16", 2, 4, 64, 16), ("bf16", 1, 8, 64, 16)])
def test_a_serving_loop_of_chunks(B, graph, dtype, hkv, group, d, page):
    """plan, append and attention on the tiles for many columns: prompts enter in chunks beside tokens and rolled-back drafts, eagerly
    and as one captured graph.  The expected output comes from lists of rows per request."""
    n, stride, n_tok, max_q = 4, 12, 200, 90
    s = Server(B, n, page, hkv, group, d, n * stride, stride, n_tok, dtype, max_q, 139)
    s.max_len = WIDE_BOUND
    s.ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(n, hkv * group, hkv, d, max_q, s.max_len), dtype=torch.uint8, device="cuda")
    assert on_tiles(B, n, n_tok, hkv * group, hkv, d, dtype, max_q, s.max_len)
    s.launch()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.launch()
    rng = np.random.default_rng(149)
    rows = [[] for _ in range(n)]
    for step in range(10):
        keep = np.array([len(r) for r in rows])
        new = np.ones(n, int)
        for i in range(n):
            what = rng.random()
            if what < 0.15:
                keep[i], new[i] = 0, 0                                   # leaves
            elif what < 0.6 or not rows[i]:
                new[i] = rng.integers(20, 50)                            # a prompt's next chunk
            elif what < 0.8:
                keep[i], new[i] = max(0, keep[i] - 3), rng.integers(1, 6)
            new[i] = min(new[i], stride * page - keep[i])
        total = int(new.sum())
        assert total <= n_tok
        k, v, q = (as_given(rng.standard_normal((n_tok, h, d)), dtype) for h in (hkv, hkv, hkv * group))
        s.k.copy_(torch.as_tensor(k)), s.v.copy_(torch.as_tensor(v)), s.q.copy_(torch.as_tensor(q))
        s.keep.copy_(i32(keep)), s.new.copy_(i32(new))
        s.out.fill_(5)
        g.replay() if graph else s.launch()
        torch.cuda.synchronize()
        assert s.status.item() == 0
        cu = np.concatenate([[0], np.cumsum(new)])
        for i in range(n):
            rows[i] = rows[i][:keep[i]] + [(k[t], v[t]) for t in range(cu[i], cu[i + 1])]
        flat = kv4.cache_array(n * stride, page, hkv, d)
        table = np.arange(n * stride, dtype=np.int32).reshape(n, stride)
        for i in range(n):
            if rows[i]:
                kv4.append(flat, np.stack([r[0] for r in rows[i]]), np.stack([r[1] for r in rows[i]]), i * stride * page + np.arange(len(rows[i])))
        check(s.out[:total], reference(flat, q[:total], cu, [len(r) for r in rows], table), dtype)
        assert (s.out[total:] == 5).all()


# ------------------------------------------------------------------------------------------- a wait that runs out

@pytest.mark.parametrize("dtype,rows", [("f32", [(60, 2000)]), ("f32", [(60, 300 + i) for i in range(160)]), ("f16", [(60, 2000)]),
                                        ("bf16", [(60, 2000)]), ("bf16", [(60, 300 + i) for i in range(160)])])
def test_a_wait_that_runs_out_gives_nan_and_the_error_word(B, dtype, rows):
    """The next call copies nothing of the cache: every wait for it runs out.  Its rows are NaN and the error word is set, the rows behind
    the last sequence stay, and the call after it is right on the same workspace."""
    rng = np.random.default_rng(151)
    cache, table, cu, length, q = attention_case(rng, 2, 4, 128, 32, rows, dtype)
    n = len(rows)
    assert on_tiles(B, n, len(q), 8, 2, 128, dtype, 60, WIDE_BOUND)
    ws = torch.zeros(B.stage_op_kv4_attention_workspace_bytes(n, 8, 2, 128, 60, WIDE_BOUND), dtype=torch.uint8, device="cuda")
    word = ws[B.STAGE_KV4_ERROR_AT:B.STAGE_KV4_ERROR_AT + 4].view(torch.int32)
    want = reference(cache, q, cu, length, table)
    B.stage_op_kv4_debug_stall(1)
    out = run_attention(B, cache, table, cu, length, q, dtype, ws=ws, max_len=WIDE_BOUND)
    assert torch.isnan(out[:int(cu[-1])].float()).all() and word.item() == 1
    for _ in range(2):
        out = run_attention(B, cache, table, cu, length, q, dtype, ws=ws, max_len=WIDE_BOUND)
        check(out, want, dtype)
        assert word.item() == 1                    # no call clears it
    word.zero_()
    out = run_attention(B, cache, table, cu, length, q, dtype, ws=ws, max_len=WIDE_BOUND)
    check(out, want, dtype)
    assert word.item() == 0


def test_stall_refuses_other_counts(B):
    for calls in (-1, 17):
        with pytest.raises(B.StageError) as e:
            B.stage_op_kv4_debug_stall(calls)
        assert e.value.code == B.STAGE_E_INVALID
    B.stage_op_kv4_debug_stall(3)
    B.stage_op_kv4_debug_stall(0)


# ------------------------------------------------------------------------------------------- one prompt among many tokens

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,bound", [(128, None), (64, None), (128, 1 << 20)])
def test_one_prompt_among_many_decoding_sequences(B, dtype, d, bound):
    """One bound for a prompt's chunk and single tokens: of the row tiles that it allows for, few are there.  `bound`: far above even the
    chunk's tokens.  NaN in V in one of the sequences, another without positions for its token."""
    rng = np.random.default_rng(157)
    rows = [(1, int(n)) for n in rng.integers(1, 150, 300)]
    rows[171], rows[40], rows[41], rows[299] = (260, 500), (1, 0), (0, 30), (9, 80)
    cache, table, cu, length, q = attention_case(rng, 2, 4, d, 16, rows, dtype)
    assert on_tiles(B, len(rows), len(q), 8, 2, d, dtype, bound or 260, WIDE_BOUND)
    want = reference(cache, q, cu, length, table)
    put_scale(cache, table, 171, 300, 1, 0, True, 0x7FFF)
    out = run_attention(B, cache, table, cu, length, q, dtype, max_q=bound, max_len=WIDE_BOUND).double().cpu().numpy()
    hit = np.zeros(q.shape, bool)
    hit[int(cu[171]) + 60:int(cu[172]), 4:, :32] = True
    assert np.isnan(out[hit]).all()
    check(out, want, dtype, ~np.isnan(want[0]) & ~hit)


def test_thousands_of_sequences(B):
    """3000 sequences of a token and one prompt: 375 thousand places for items of which 6 thousand are there."""
    rng = np.random.default_rng(163)
    rows = [(1, 1 + i % 20) for i in range(3000)]
    rows[2000] = (1000, 1000)
    cache, table, cu, length, q = attention_case(rng, 1, 8, 64, 16, rows, "bf16")
    assert on_tiles(B, len(rows), len(q), 8, 1, 64, "bf16", 1000, WIDE_BOUND)
    out = run_attention(B, cache, table, cu, length, q, "bf16", max_len=WIDE_BOUND)
    check(out, reference(cache, q, cu, length, table), "bf16")


# ------------------------------------------------------------------------------------------- bounds, and rows by the thousand

@pytest.mark.parametrize("empty", [0, 160])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_chunks_beyond_the_stated_bounds(B, dtype, empty):
    """On the tiles for many columns too, tokens behind max_q get no output and keep their positions, seq_len counts as at most the
    table's positions, and one below zero as none."""
    rng = np.random.default_rng(167)
    cache, table, cu, length, q = attention_case(rng, 2, 4, 64, 16, [(70, 150), (40, 300), (33, 40)], dtype)
    out = tiled(B, cache, table, cu, length, q, dtype, empty=empty, max_q=45)
    ref = reference(cache, q, cu, length, table)
    done = np.zeros(q.shape, bool)
    for i in range(3):
        done[cu[i]:min(cu[i] + 45, cu[i + 1])] = True
    check(out, ref, dtype, done)
    assert (out[45:70] == 3).all()
    short = table[:, :5].copy()
    out = tiled(B, cache, short, cu, np.array([10 ** 9, 2 ** 31 - 1, -7], np.int32), q, dtype, empty=empty)
    ref = reference(cache, q, cu, [80, 80, 0], short)
    check(out, ref, dtype)
    assert (out[int(cu[2]):int(cu[3])] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,hkv", [(128, 8), (128, 3), (128, 1), (64, 8), (64, 5), (64, 1)])
def test_thousands_of_rows_are_written_and_read_as_few_are(B, dtype, d, hkv):
    """From 4096 rows on a warp goes through all heads of its row, below through some: the same bytes, and the same values back.  The calls
    of few rows are those that tests/test_gpu_kv4.py holds against the oracle."""
    g = torch.Generator(device="cuda").manual_seed(d + hkv)
    n, page = 4099, 32
    pages = n // page + 20
    slot = torch.randperm(pages * page, device="cuda", generator=g)[:n].to(torch.int32)
    slot[::17] = -1
    slot[5] = pages * page
    power = torch.randint(-30, 18, (n, hkv, 1), device="cuda", generator=g)
    k, v = ((torch.randn(n, hkv, d, device="cuda", generator=g) * 2.0 ** power).to(DT[dtype]) for _ in range(2))
    k[7, 0, 3], v[9, -1, 40] = float("inf"), float("nan")
    start = torch.randint(0, 256, B.stage_op_kv4_cache_shape(pages, page, hkv, d), device="cuda", generator=g).to(torch.uint8)
    one, some = start.clone(), start.clone()
    B.stage_op_kv4_append(one, k, v, slot)
    for a in range(0, n, 1000):
        B.stage_op_kv4_append(some, k[a:a + 1000], v[a:a + 1000], slot[a:a + 1000])
    assert torch.equal(one, some) and not torch.equal(one, start)
    got = [torch.full((n, hkv, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(4)]
    B.stage_op_kv4_read(one, slot, got[0], got[1])
    for a in range(0, n, 1000):
        B.stage_op_kv4_read(one, slot[a:a + 1000], got[2][a:a + 1000], got[3][a:a + 1000])
    for x, y in ((got[0], got[2]), (got[1], got[3])):
        same(x.double().cpu().numpy(), y.double().cpu().numpy())
    assert (got[0][::17] == 7).all()
