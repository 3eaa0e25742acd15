"""Attention over the paged 4-bit cache at the edges of its range, against a float64 reference.

The tolerances are those of tests/test_gpu_kv4.py, derived there; `small` bounds what fp16's smallest step takes from a probability.
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
@pytest.mark.parametrize("qtok,n,empty", [(1, 100, None), (1, 3000, None), (3, 200, None)])
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
