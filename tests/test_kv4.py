"""The paged 4-bit cache without a GPU: the oracle pinned against exact arithmetic and invariants, and every
refusal of the entry points of include/stage_kv4.h before any device call."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import layer_range_stage_gb300 as L
from layer_range_stage_gb300 import build as lbuild
from oracle import kv4


@pytest.fixture(scope="module", autouse=True)
def built():
    lbuild.build()


@pytest.mark.parametrize("d", [64, 128])
def test_every_nibble_and_scale_has_one_place(d):
    p, dim = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    seen = np.zeros(18 * d, dtype=int)
    for is_v in (False, True):
        at, sh = kv4.code_place(p, dim, d, is_v)
        np.add.at(seen, at.ravel(), 1 << sh.ravel())            # two nibbles: 1 + 16
        sp = kv4.scale_place(*np.meshgrid(np.arange(16), np.arange(d // 32), indexing="ij"), d, is_v)
        np.add.at(seen, sp.ravel(), 17)
        np.add.at(seen, sp.ravel() + 1, 17)
    assert (seen == 17).all()


def test_quantise_against_exact_rationals():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal((200, 32)), rng.standard_normal((50, 32)) * 1e-6, rng.standard_normal((50, 32)) * 1e4,
                        rng.integers(-16, 17, (200, 32)) / 2.0]).astype(np.float32)   # the last: many ties
    bits, codes = kv4.quantise(x)
    for row, b, c in zip(x, bits[:, 0], codes):
        m = row[np.abs(row).argmax()]
        s = np.float16(np.float32(m) / np.float32(-8))
        assert b == s.view(np.uint16)
        if s == 0:
            assert (c == 8).all()
            continue
        for xi, ci in zip(row, c):
            want = round(Fraction(float(xi)) / Fraction(float(s)))   # ties to even
            assert int(ci) == min(15, max(0, want + 8))


def test_quantise_edges():
    x = np.zeros((6, 32), np.float32)
    x[1, 3], x[1, 7] = 2.0, -2.0             # a tie of magnitudes: the lower index gives the sign
    x[2, 0] = np.inf
    x[3, 5] = np.nan
    x[4, 1] = 6e5                            # 6e5 / 8 is beyond fp16
    x[5, 2] = 1e-9                           # its scale is 0
    bits, codes = kv4.quantise(x)
    assert bits[0, 0] & 0x7FFF == 0 and (codes[0] == 8).all()
    assert bits[1, 0] == np.float16(-0.25).view(np.uint16) and codes[1, 3] == 0 and codes[1, 7] == 15  # 16 clamped
    assert (bits[2:5, 0] == kv4.NAN_SCALE).all() and (codes[2:5] == 8).all()
    assert bits[5, 0] & 0x7FFF == 0 and (codes[5] == 8).all()


@pytest.mark.parametrize("d", [64, 128])
def test_append_then_rows_within_half_a_step(d):
    rng = np.random.default_rng(d)
    cache = kv4.cache_array(5, 32, 3, d)
    slots = rng.permutation(5 * 32)[:40]
    slots[7] = -1
    slots[9] = 5 * 32
    k, v = (rng.standard_normal((40, 3, d)).astype(np.float32) for _ in range(2))
    kv4.append(cache, k, v, slots)
    live = (slots >= 0) & (slots < 160)
    for is_v, x in ((False, k), (True, v)):
        got = kv4.rows(cache, slots[live], is_v)
        top = np.abs(x[live]).reshape(-1, 3, d // 32, 32).max(-1).repeat(32, -1)
        # half a step of top / 8, a whole one at the clamped end, and the scale's own rounding of 8 steps
        assert (np.abs(got - x[live]) <= top / 8 * (1 + 8 * 2.0 ** -11)).all()
        assert np.abs(got - x[live]).mean() < 0.3 * (top / 8).mean()
    untouched = np.setdiff1d(np.arange(160), slots)
    assert (kv4.rows(cache, untouched, True) == 0).all()


def test_attention_of_equal_scores_is_the_mean():
    rng = np.random.default_rng(5)
    cache = kv4.cache_array(3, 16, 2, 64)
    table = np.array([[2, 0, -1]], np.int32)
    slots = np.concatenate([32 + np.arange(16), np.arange(5)])
    kv4.append(cache, np.zeros((21, 2, 64), np.float32), rng.standard_normal((21, 2, 64)).astype(np.float32), slots)
    q = rng.standard_normal((3, 4, 64))
    out, *_ = kv4.attention(cache, q, [0, 3], [21], table)
    v = kv4.rows(cache, slots, True)
    for j in range(3):
        for h in range(4):
            assert np.allclose(out[j, h], v[:19 + j, h // 2].mean(0), atol=1e-14)
    out, *_ = kv4.attention(cache, q, [0, 3], [1], table)   # two tokens before the first position
    assert (out[:2] == 0).all() and np.allclose(out[2, 0], v[0, 0])


def test_plan_keeps_every_page_once():
    rng = np.random.default_rng(3)
    page, n, stride, pages = 16, 9, 12, 22
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((n, stride), -1, np.int32)
    ring = ids.copy()
    free = np.array([0, pages], np.int32)
    length = np.zeros(n, np.int32)
    seen = set()
    for step in range(200):
        keep = np.where(rng.random(n) < 0.15, 0, length - np.minimum(length, rng.integers(0, 5, n))).astype(np.int32)
        new = np.where(rng.random(n) < 0.1, rng.integers(0, 90, n), rng.integers(0, 3, n)).astype(np.int32)
        new = np.minimum(new, stride * page - keep).astype(np.int32)
        r = kv4.plan(page, length, new, table, ring, free, 400, pages, keep)
        seen.add(r["status"])
        length, table, ring, free = r["len"], r["table"], r["ring"], r["free"]
        held = [p for i in range(n) for p in table[i, : -(-length[i] // page)]]
        loose = [ring[(free[0] + j) % pages] for j in range(free[1])]
        assert sorted(held + loose) == list(range(pages))
        if r["status"] == 0:
            assert r["cu"][-1] == new.sum() and len(set(r["slot"][: new.sum()])) == new.sum()
    assert seen == {0, 1}


def test_entry_points_refuse_bad_arguments_before_any_device_call():
    lib, v = L.lib(), ctypes.c_void_p
    buf = ctypes.create_string_buffer(4096 + 64)
    p = v((ctypes.addressof(buf) + 63) // 64 * 64)
    odd, off4 = v(p.value + 2), v(p.value + 4)

    def rows(fn, cache=p, n_pages=4, page=16, hkv=2, d=64, k=p, vv=p, dtype=0, stride=128, slot=p, n=3):
        if fn is lib.stage_op_kv4_append:
            return fn(cache, n_pages, page, hkv, d, k, vv, dtype, stride, slot, n, None)
        return fn(cache, n_pages, page, hkv, d, slot, n, k, vv, dtype, stride, None)

    for fn in (lib.stage_op_kv4_append, lib.stage_op_kv4_read):
        for kw in (dict(cache=None), dict(cache=off4), dict(n_pages=0), dict(n_pages=1 << 27, page=16), dict(page=8), dict(page=24), dict(page=4112),
                   dict(hkv=0), dict(hkv=1025), dict(d=96), dict(k=None), dict(vv=None), dict(k=off4), dict(vv=off4), dict(dtype=3), dict(dtype=-1),
                   dict(stride=127), dict(stride=130), dict(dtype=1, stride=132), dict(stride=1 << 40), dict(slot=None), dict(slot=odd), dict(n=-1),
                   dict(n=(1 << 24) + 1)):
            assert rows(fn, **kw) == L.STAGE_E_INVALID, kw
            assert lib.stage_op_last_error().decode()
        assert rows(fn, k=None, vv=None, slot=None, n=0) == L.STAGE_OK       # an empty step

    def attend(cache=p, n_pages=4, page=16, hkv=2, d=64, q=p, dtype=0, qs=256, n_tok=3, hq=4, cu=p, sl=p, table=p, ts=2, n=2, mq=2, ml=32, out=p, os_=256, ws=p,
               wb=1 << 30):
        return lib.stage_op_kv4_attention(cache, n_pages, page, hkv, d, q, dtype, qs, n_tok, hq, cu, sl, table, ts, n, mq, ml, out, os_, ws, wb, None)

    for kw in (dict(cache=None), dict(cache=off4), dict(page=20), dict(d=32), dict(q=None), dict(q=off4), dict(dtype=7), dict(qs=255), dict(qs=258),
               dict(n_tok=-1), dict(n_tok=1 << 25), dict(hq=3), dict(hq=0), dict(hq=1026), dict(cu=None), dict(sl=None), dict(table=None), dict(cu=odd),
               dict(ts=0), dict(ts=1 << 21), dict(n=-1), dict(n=65536), dict(mq=0), dict(ml=0), dict(mq=1 << 21), dict(ml=(1 << 30) + 1), dict(out=None),
               dict(out=off4), dict(os_=192), dict(ws=None), dict(ws=off4), dict(wb=0)):
        assert attend(**kw) == L.STAGE_E_INVALID, kw
        assert lib.stage_op_last_error().decode()
    assert attend(n_tok=0, q=None, out=None) == L.STAGE_OK and attend(n=0, cu=None) == L.STAGE_OK

    def plan(n=2, page=16, pages=4, sl=p, kl=None, nl=p, table=p, ts=2, ring=p, rl=4, fs=p, slo=p, fso=p, nt=3, cu=p, slot=p, pos=p, seq=p, st=p):
        return lib.stage_op_kv4_plan(n, page, pages, sl, kl, nl, table, ts, ring, rl, fs, slo, fso, nt, cu, slot, pos, seq, st, None)

    for kw in (dict(n=-1), dict(n=65537), dict(page=0), dict(page=17), dict(page=8192), dict(pages=0), dict(pages=1 << 40), dict(sl=None), dict(kl=odd),
               dict(nl=None), dict(table=None), dict(ts=0), dict(ts=(1 << 20) + 1), dict(ring=None), dict(rl=0), dict(fs=None), dict(slo=None),
               dict(fso=None), dict(nt=-1), dict(nt=(1 << 24) + 1), dict(cu=None), dict(slot=None), dict(pos=None), dict(seq=None), dict(st=None), dict(st=odd)):
        assert plan(**kw) == L.STAGE_E_INVALID, kw
        assert lib.stage_op_last_error().decode()


def test_sizes():
    assert L.stage_op_kv4_cache_bytes(10, 64, 8, 128) == 10 * 8 * 4 * 2304
    assert L.stage_op_kv4_cache_shape(10, 64, 8, 128) == (10, 8, 4, 2304)
    assert L.stage_op_kv4_cache_bytes((1 << 31) // 16, 16, 1, 64) == 0 and L.stage_op_kv4_cache_bytes(1, 16, 1, 96) == 0
    with pytest.raises(L.StageError):
        L.stage_op_kv4_cache_shape(1, 8, 1, 64)
    assert L.stage_op_kv4_attention_workspace_bytes(4, 6, 4, 128, 1, 100) == 0   # 6 heads over 4
    assert L.stage_op_kv4_attention_workspace_bytes(4, 8, 4, 128, 1, 0) == 0
    for n, hq, hkv, d, mq, ml in ((1, 32, 8, 128, 1, 1 << 20), (65535, 1024, 8, 128, 1 << 20, 1 << 30), (64, 64, 8, 128, 1, 4096), (3, 7, 1, 64, 5, 17)):
        assert 0 < L.stage_op_kv4_attention_workspace_bytes(n, hq, hkv, d, mq, ml) <= 64 << 20


def test_binding_refuses_host_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    cache = torch.zeros(L.stage_op_kv4_cache_shape(4, 16, 2, 64), dtype=torch.uint8)
    k = torch.zeros(3, 2, 64)
    slot = torch.zeros(3, dtype=torch.int32)
    for bad in (cache.flatten(), cache.to(torch.int32), cache[..., :-1], cache.transpose(0, 1)):
        with pytest.raises(L.StageError) as e:
            L.stage_op_kv4_append(bad, k, k, slot)
        assert e.value.code == L.STAGE_E_INVALID
    with pytest.raises(L.StageError, match="device tensors"):
        L.stage_op_kv4_append(cache, k, k, slot)


def test_binding_refuses_sizes_that_a_c_int_would_cut_off():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, dtype=torch.int32)
    for max_q, max_len in ((0, 5), ((1 << 32) + 1, 5), (1, 0), (1, (1 << 32) + 5), (-1, 5), ((1 << 20) + 1, 5)):
        with pytest.raises(L.StageError, match="max_q"):
            L.stage_op_kv4_attention(x, x, x, x, x, x, max_q, max_len, x)
    for page_len in (0, -16, 8192, (1 << 32) + 16):
        with pytest.raises(L.StageError, match="page_len"):
            L.stage_op_kv4_plan(page_len, *[x] * 12)
