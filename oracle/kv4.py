"""Plain oracle of the paged 4-bit KV cache (include/stage_kv4.h): float64 numpy, test infrastructure only.

The cache is a uint8 array [n_pages, n_kv_heads, page_len / 16, 18 * head_dim]; everything here goes by the
address of single nibbles, one rule per function, and shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

NAN_SCALE = 0x7FFF


def cache_array(n_pages: int, page_len: int, n_kv_heads: int, head_dim: int) -> np.ndarray:
    return np.zeros((n_pages, n_kv_heads, page_len // 16, 18 * head_dim), dtype=np.uint8)


def code_place(p, d, head_dim: int, is_v: bool):
    """(byte inside the tile, shift) of the code of position p (0..15) and dim d."""
    p, d = np.asarray(p), np.asarray(d)
    nb, block, j = head_dim // 32, d // 32, d % 32
    if is_v:
        at = ((((p // 8) * 8 + j // 4) * 4 + (p // 2) % 4) * 2 + p % 2) * nb + block
        return 9 * head_dim + 2 * at + (j // 2) % 2, 4 * (d % 2)
    at = (p * 4 + j // 8) * nb + block
    return 4 * at + (j // 2) % 4, 4 * (d % 2)


def scale_place(p, block, head_dim: int, is_v: bool):
    """Byte inside the tile of the fp16 scale of position p and block."""
    return (9 * head_dim if is_v else 0) + 8 * head_dim + 2 * (np.asarray(p) * (head_dim // 32) + np.asarray(block))


def quantise(x: np.ndarray):
    """x [..., 32 * n] (the values as given: float32 or less) -> scale bits uint16 [..., n], codes uint8 [..., 32 * n]."""
    b = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(all="ignore"):
        mag = np.where(np.isnan(b), np.inf, np.abs(b))
        m = np.take_along_axis(b, mag.argmax(-1)[..., None], -1)
        s = (m / -8).astype(np.float32).astype(np.float16)   # m / 8 is exact in float32 wherever fp16 can hold it
        bad = ~np.isfinite(s.astype(np.float64))
        s64 = np.where(bad | (s == 0), 1.0, s.astype(np.float64))
        c = np.clip(np.rint(np.where(bad | (s == 0), 0.0, b) / s64) + 8, 0, 15).astype(np.uint8)
    bits = np.where(bad, np.uint16(NAN_SCALE), s.view(np.uint16))[..., 0]
    return bits, c.reshape(x.shape)


def append(cache: np.ndarray, k, v, slots) -> None:
    """Write rows k, v [n, heads, head_dim] (any float type; taken as they are) at their slots."""
    n_pages, heads, tiles, nbytes = cache.shape
    d, page_len = nbytes // 18, tiles * 16
    dims, blocks = np.arange(d), np.arange(d // 32)
    for is_v, x in ((False, k), (True, v)):
        bits, codes = quantise(x)
        for t, slot in enumerate(slots):
            if not 0 <= slot < n_pages * page_len:
                continue
            page, off = divmod(int(slot), page_len)
            p = off % 16
            at, sh = code_place(p, dims, d, is_v)
            sp = scale_place(p, blocks, d, is_v)
            for h in range(heads):
                tile = cache[page, h, off // 16]
                tile[at[0::2]] = codes[t, h, 0::2] | codes[t, h, 1::2] << 4
                tile[sp], tile[sp + 1] = bits[t, h] & 255, bits[t, h] >> 8


def rows(cache: np.ndarray, slots, is_v: bool) -> np.ndarray:
    """Values [n, heads, head_dim] float64 at valid slots."""
    heads, tiles, nbytes = cache.shape[1:]
    d, page_len = nbytes // 18, tiles * 16
    slots = np.asarray(slots, np.int64)
    page, off = slots // page_len, slots % page_len
    tile = cache[page, :, off // 16].astype(np.int64)               # [n, heads, bytes]
    p = off % 16
    at, sh = code_place(p[:, None], np.arange(d), d, is_v)          # [n, d]
    code = np.take_along_axis(tile, np.broadcast_to(at[:, None], tile.shape[:2] + (d,)), -1) >> sh[None, None] & 15
    sp = np.broadcast_to(scale_place(p[:, None], np.arange(d) // 32, d, is_v)[:, None], tile.shape[:2] + (d,))
    bits = (np.take_along_axis(tile, sp, -1) | np.take_along_axis(tile, sp + 1, -1) << 8).astype(np.uint16)
    return bits.view(np.float16).astype(np.float64) * (code - 8)


def attention(cache, q, cu, seq_len, table, max_q=None, max_len=None):
    """Softmax attention in float64, and what rounding errors are relative to, as
    (out, weight, spread, peak, seen): out [rows, heads, d], NaN in rows that get no output; weight the same for
    sum_j p_j |v_j|; per row and head: spread, the largest sum_d |q_d k_jd| / sqrt(D); peak, the largest
    p_j max_d |v_jd|; seen, the number of positions."""
    n_pages, hkv, tiles, nbytes = cache.shape
    d, page_len = nbytes // 18, tiles * 16
    q = np.asarray(q, np.float64)
    group = q.shape[1] // hkv
    out = np.full(q.shape, np.nan)
    weight = np.zeros(q.shape)
    spread, peak, count = (np.zeros(q.shape[:2]) for _ in range(3))
    for i, n in enumerate(seq_len):
        c = int(cu[i + 1]) - int(cu[i])
        n = min(int(n), table.shape[1] * page_len, max_len or 1 << 60)
        at = np.arange(max(n, 0))
        page = table[i][at // page_len].astype(np.int64)
        at = at[(page >= 0) & (page < n_pages)]
        slots = table[i][at // page_len].astype(np.int64) * page_len + at % page_len
        k, v = rows(cache, slots, False), rows(cache, slots, True)
        for j in range(min(c, max_q or c)):
            t = int(cu[i]) + j
            seen = at <= n - c + j
            for h in range(q.shape[1]):
                kh, vh = k[seen, h // group], v[seen, h // group]
                if not len(kh):
                    out[t, h] = 0
                    continue
                with np.errstate(all="ignore"):
                    s = kh @ q[t, h] / np.sqrt(d)
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out[t, h] = p @ vh
                    weight[t, h] = p @ np.abs(vh)
                    spread[t, h] = (np.abs(kh) @ np.abs(q[t, h])).max() / np.sqrt(d)
                    peak[t, h] = (p * np.abs(vh).max(-1)).max()
                    count[t, h] = len(kh)
    return out, weight, spread, peak, count


def plan(page_len, seq_len, new_len, table, ring, free_state, n_tok, n_pages, keep_len=None):
    """The step's outputs as a dict (table and ring as copies), one request after another."""
    n, stride = table.shape
    head, count = (int(x) for x in free_state)
    keep_len = seq_len if keep_len is None else keep_len
    r = {"len": np.array(seq_len), "table": table.copy(), "ring": ring.copy(), "free": np.array(free_state), "cu": np.zeros(n + 1, np.int32),
         "slot": np.full(n_tok, -1, np.int32), "pos": np.full(n_tok, -1, np.int32), "seq": np.full(n_tok, -1, np.int32), "status": 0}
    bad = not (0 <= head < len(ring) and 0 <= count <= len(ring))
    have, need = [], []
    for length, keep, new in zip(map(int, seq_len), map(int, keep_len), map(int, new_len)):
        ok = length >= 0 and 0 <= keep <= length and new >= 0
        have.append(-(-length // page_len) if ok else 0)
        need.append(-(-(keep + new) // page_len) if ok else 0)
        bad |= not ok or have[-1] > stride or (need[-1] > stride and new <= n_tok) or keep + min(new, n_tok + 1) >= 2 ** 31
    give = sum(max(0, h - w) for h, w in zip(have, need))
    if bad or count + give > len(ring):
        r["status"] = 2
    elif sum(map(int, new_len)) > n_tok:
        r["status"] = 3
    elif sum(max(0, w - h) for h, w in zip(have, need)) > count:
        r["status"] = 1
    if r["status"]:
        return r
    tail, t = head + count, 0
    for i in range(n):
        for col in range(have[i], need[i]):
            r["table"][i, col] = ring[head % len(ring)]
            head, count = head + 1, count - 1
        for col in range(need[i], have[i]):
            r["ring"][tail % len(ring)] = table[i, col]
            tail, count = tail + 1, count + 1
        r["cu"][i] = t
        for k in range(int(new_len[i])):
            pos = int(keep_len[i]) + k
            page = int(r["table"][i, pos // page_len])
            r["slot"][t] = page * page_len + pos % page_len if 0 <= page < n_pages else -1
            r["pos"][t], r["seq"][t] = pos, i
            t += 1
        r["len"][i] = int(keep_len[i]) + int(new_len[i])
    r["cu"][n] = t
    r["free"] = np.array([head % len(ring), count], np.int32)
    return r
