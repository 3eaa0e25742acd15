"""A step's operators without a GPU: the oracle's pins, the frequencies, and every refusal of the entry points of
include/stage_step.h before any device call."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import layer_range_stage_gb300 as L
from layer_range_stage_gb300 import build as lbuild
from oracle import step


@pytest.fixture(scope="module", autouse=True)
def built():
    lbuild.build()


# ------------------------------------------------------------------------------------------- the oracle

def test_e4m3_against_torch_and_exact_rationals():
    torch = pytest.importorskip("torch")
    v = step.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    assert np.array_equal(step.e4m3_codes(v)[~np.isnan(v)], np.arange(256)[~np.isnan(v)])
    rng = np.random.default_rng(0)
    mids = (v[:126] + v[1:127]) / 2                        # every tie
    x = np.concatenate([mids, -mids, rng.uniform(-460, 460, 400), rng.standard_normal(400) * 2.0 ** rng.integers(-12, 5, 400)])
    table = [Fraction(float(a)) for a in v[:127]]
    for xi, c in zip(x, step.e4m3_codes(x)):
        a = min(abs(Fraction(float(xi))), table[-1])
        near = min(range(127), key=lambda i: (abs(table[i] - a), i % 2))
        assert c & 127 == near and bool(c & 128) == bool(np.signbit(xi))


def test_norm_rows_come_back():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 300)).astype(np.float32)
    g = rng.standard_normal(300).astype(np.float32)
    h, y, codes, scales = step.norm_f8(x, x, g, 1e-5)
    assert np.array_equal(h, 2 * x)
    want = 2 * x / np.sqrt((4.0 * x.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-5) * g
    assert np.allclose(y, want, rtol=3e-7, atol=0)
    back = step.e4m3_values()[codes] * np.repeat(scales, 128, 0)[:300].T
    top = np.abs(y).reshape(5, -1)
    assert (np.abs(back - y) <= np.abs(y) * 2.0 ** -4 + top.max() * 2.0 ** -10 / 448 * 1.01).all()
    zero = step.norm_f8(np.zeros((1, 130), np.float32))
    assert (zero[2] == 0).all() and (zero[3] > 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_lengths_and_depends_on_distance_alone(interleaved):
    rng = np.random.default_rng(2)
    f, _ = step.rope_freqs(32, 10000.0)
    q, k = rng.standard_normal((2, 1, 1, 40))
    def score(a, b):
        return (step.rope(q, [a], f, interleaved) * step.rope(k, [b], f, interleaved)).sum()
    assert abs(score(17, 5) - score(100012, 100000)) < 1e-9
    assert np.allclose(np.linalg.norm(step.rope(q, [12345], f, interleaved)), np.linalg.norm(q))
    assert np.array_equal(step.rope(q, [7], f, interleaved)[..., 32:], q[..., 32:])


def test_logprobs_of_a_known_row():
    z = np.log(np.array([[0.5, 0.125, 0.25, 0.125, 0.0]]), where=np.array([[1, 1, 1, 1, 0]], bool), out=np.full((1, 5), -np.inf))
    r = step.logprobs(z, [3], 4)
    assert np.allclose(r["logprob"], math.log(0.125)) and np.allclose(r["entropy"], 1.75 * math.log(2))
    assert r["rank"][0] == 3 and list(r["ids"][0]) == [0, 2, 1, 3]


# ------------------------------------------------------------------------------------------- frequencies

@pytest.mark.parametrize("rot,theta,kind,factor,first,low,high", [
    (128, 10000.0, "plain", 1.0, 1.0, 1.0, 32.0), (64, 500000.0, "linear", 4.0, 1.0, 1.0, 32.0), (80, 10000.0, "base", 2.5, 1.0, 1.0, 32.0),
    (128, 500000.0, "bands", 8.0, 8192.0, 1.0, 4.0), (128, 10000.0, "parts", 16.0, 4096.0, 1.0, 32.0), (2, 10000.0, "parts", 2.0, 64.0, 1.0, 32.0),
    (64, 10000.0, "parts", 40.0, 4.0, 1.0, 32.0), (16, 10000.0, "bands", 2.0, 4.0, 1.0, 4.0)])
def test_frequencies(rot, theta, kind, factor, first, low, high):
    code = {"plain": L.STAGE_ROPE_PLAIN, "linear": L.STAGE_ROPE_LINEAR, "base": L.STAGE_ROPE_BASE, "bands": L.STAGE_ROPE_BANDS, "parts": L.STAGE_ROPE_PARTS}[kind]
    f, s = L.stage_op_rope_freqs(rot, theta, code, factor, first, low, high)
    want, scale = step.rope_freqs(rot, theta, kind, factor, first, low, high)
    # a power, a logarithm and a few operations of 64 bits: far below 2^-44 of a frequency
    assert f.shape == (rot // 2,) and np.allclose(f, want, rtol=2.0 ** -44, atol=0)
    assert abs(s - scale) <= scale * 2.0 ** -24


def test_frequencies_refused():
    ok = dict(rot_dim=64, theta=10000.0, scaling=L.STAGE_ROPE_PARTS, factor=2.0, first_len=4096.0, low=1.0, high=32.0)
    L.stage_op_rope_freqs(**ok)
    for kw in (dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=1026), dict(rot_dim=-2), dict(rot_dim=(1 << 32) + 64), dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf),
               dict(scaling=5), dict(scaling=-1), dict(factor=0.5), dict(factor=math.nan), dict(first_len=0.0), dict(low=0.0), dict(high=1.0), dict(high=math.inf),
               dict(rot_dim=2, scaling=L.STAGE_ROPE_BASE)):
        with pytest.raises(L.StageError):
            L.stage_op_rope_freqs(**{**ok, **kw})


# ------------------------------------------------------------------------------------------- refusals

def test_entry_points_refuse_bad_arguments_before_any_device_call():
    lib, v = L.lib(), ctypes.c_void_p
    buf = ctypes.create_string_buffer(4096 + 64)
    p = v((ctypes.addressof(buf) + 63) // 64 * 64)
    odd, off2, off8 = v(p.value + 1), v(p.value + 2), v(p.value + 8)
    far = (1 << 32) + 1

    def norm(x=p, xt=0, xs=256, r=p, rt=0, rs=256, ro=p, ros=256, g=p, eps=1e-5, n_tok=3, n=256, q=p, qs=256, s=p, ss=3, y=p, ys=256):
        return lib.stage_op_norm_f8(x, xt, xs, r, rt, rs, ro, ros, g, eps, n_tok, n, q, qs, s, ss, y, ys, None)

    def gemm(a=p, as_=256, sa=p, sas=3, w=p, ws=256, sw=p, M=3, N=5, K=250, y=p, yt=0, ys=5, err=None):
        return lib.stage_op_f8_gemm(a, as_, sa, sas, w, ws, sw, M, N, K, y, yt, ys, err, None)

    def rope(q=p, qs=256, hq=2, k=p, ks=128, hk=1, d=128, dt=0, pos=p, n=3, f=p, rot=64, inter=0, scale=1.0, qo=p, qos=256, ko=p, kos=128):
        return lib.stage_op_rope(q, qs, hq, k, ks, hk, d, dt, pos, n, f, rot, inter, scale, qo, qos, ko, kos, None)

    def lp(z=p, dt=0, rs=100, n=3, vocab=100, t=p, l=p, e=p, r=p, top=2, ids=p, best=p):
        return lib.stage_op_logprobs(z, dt, rs, n, vocab, t, l, e, r, top, ids, best, None)

    bad = {
        norm: (dict(x=None), dict(x=off2), dict(x=odd, xt=1), dict(xt=3), dict(xt=-1), dict(xs=255), dict(xs=far), dict(r=None), dict(ro=None), dict(r=off2), dict(rt=1),
               dict(xt=1, rt=2), dict(rs=255), dict(ros=255), dict(ros=far), dict(rs=260), dict(g=off2), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(n_tok=-1),
               dict(n_tok=(1 << 24) + 1), dict(n=0), dict(n=32769, xs=40000), dict(q=None), dict(s=None), dict(q=None, s=None, y=None), dict(qs=255), dict(qs=far), dict(ss=2),
               dict(s=off2), dict(y=off2), dict(ys=255)),
        gemm: (dict(a=None), dict(a=off8), dict(as_=249), dict(as_=255), dict(as_=250), dict(as_=1 << 33), dict(sa=None), dict(sa=off2), dict(sas=2), dict(w=None), dict(w=off8),
               dict(ws=240), dict(ws=257), dict(sw=None), dict(sw=off2), dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=(1 << 20) + 1),
               dict(M=1 << 24, N=1 << 24, sas=1 << 24, ys=1 << 24), dict(y=None), dict(y=off2), dict(yt=5), dict(ys=4), dict(err=off2)),
        rope: (dict(q=None), dict(q=off2), dict(qs=255), dict(qs=far), dict(hq=0), dict(hq=1025), dict(k=None), dict(k=off2), dict(ks=127), dict(hk=-1), dict(hk=1025), dict(d=1),
               dict(d=1026), dict(dt=9), dict(pos=None), dict(pos=off2), dict(n=-1), dict(n=(1 << 24) + 1), dict(f=None), dict(f=v(p.value + 4)), dict(rot=0), dict(rot=63), dict(rot=130),
               dict(scale=math.nan), dict(scale=math.inf), dict(qo=None), dict(qo=off2), dict(qos=255), dict(qos=260), dict(ko=None), dict(kos=260)),
        lp: (dict(z=None), dict(z=off2), dict(dt=4), dict(rs=99), dict(rs=far), dict(n=-1), dict(n=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 19) + 1, rs=1 << 20), dict(t=None),
             dict(t=off2), dict(l=off2), dict(e=odd), dict(r=off2), dict(top=-1), dict(top=33), dict(top=3, vocab=2), dict(ids=off2), dict(best=off2)),
    }
    for fn, cases in bad.items():
        for kw in cases:
            assert fn(**kw) == L.STAGE_E_INVALID, (fn.__name__, kw)
            assert lib.stage_op_last_error().decode()
    none = dict(zip(("x", "r", "ro", "q", "s", "y"), [None] * 6))
    assert norm(n_tok=0, **none) == L.STAGE_OK and gemm(M=0, a=None, y=None) == L.STAGE_OK
    assert rope(n=0, q=None, pos=None) == L.STAGE_OK and lp(n=0, z=None) == L.STAGE_OK
    assert lib.stage_op_f8_debug_stall(17) == L.STAGE_E_INVALID and lib.stage_op_f8_debug_stall(0) == L.STAGE_OK


def test_binding_refuses_host_tensors_shapes_and_types():
    torch = pytest.importorskip("torch")
    x, s, i = torch.zeros(3, 256), torch.zeros(2, 3), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 256, dtype=torch.uint8)
    f = torch.zeros(32, dtype=torch.float64)
    for call in (lambda: L.stage_op_norm_f8(x, q, s), lambda: L.stage_op_f8_gemm(q, s, q, torch.zeros(1, 2), torch.zeros(3, 3)),
                 lambda: L.stage_op_rope(x.view(3, 2, 128), None, i, f), lambda: L.stage_op_logprobs(x, i, torch.zeros(3))):
        with pytest.raises(L.StageError, match="device tensors"):
            call()
    with pytest.raises(L.StageError, match="go together"):
        L.stage_op_norm_f8(x, q)
    with pytest.raises(L.StageError, match="go together"):
        L.stage_op_norm_f8(x, q, s, resid=x)


def test_pairs_that_share_a_k_have_one_tile_each_however_many_sms(tmp_path):
    """The kernel adds a cluster's sums up once: with more tiles than clusters those of all but the last would be lost."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "split.cu"
    src.write_text("""
#include <cstdio>
#include "step.cuh"
int main() {
  int shared = 0;
  for (int sms = 1; sms <= 200; ++sms)
    for (long tiles = 1; tiles <= 300; ++tiles)
      for (int nkb = 1; nkb <= 40; ++nkb) {
        const lrs::BigSplit s = lrs::big_split(tiles, nkb, sms);
        if (s.S < 1 || s.S > 2 || s.clusters < 1 || s.clusters > tiles || (s.S > 1 && s.clusters != tiles)) return printf("%d SMs, %ld tiles: %d, %u\\n", sms, tiles, s.S, s.clusters), 1;
        shared += s.S == 2;
      }
  const lrs::BigSplit all = lrs::big_split(1 << 24, 112, 152);
  return !(shared > 0 && all.S == 1 && all.clusters == 76);
}
""")
    subprocess.run([lbuild.nvcc(), *lbuild.ARCH, "-std=c++17", "-I", os.path.join(root, "layer_range_stage_gb300", "csrc"), "-o", str(tmp_path / "split"), str(src)], check=True, capture_output=True)
    r = subprocess.run([str(tmp_path / "split")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_a_rows_cluster_goes_by_the_sms_there_are(tmp_path):
    """One wave of CTAs where rows are few, whatever the number of SMs, and never more of a row in a CTA than it has room for."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "cluster.cu"
    src.write_text("""
#include <cstdio>
#include "step.cuh"
int main() {
  for (int sms = 1; sms <= 300; ++sms)
    for (int rows = 1; rows <= 400; ++rows)
      for (int chunks = 1; chunks <= (1 << 16) + 1; chunks = chunks < 3 ? chunks + 1 : chunks * 4 / 3 + 1) {
        const int C = lrs::logprobs_cluster(chunks, rows, sms);
        const bool room = (chunks + C - 1) / C <= lrs::kLogprobsMaxChunks;
        const bool half = C > 1 && (chunks + C / 2 - 1) / (C / 2) <= lrs::kLogprobsMaxChunks;   // half of them would have the room
        if (!room || C > lrs::kLogprobsMaxCluster || (half && (long)rows * (C / 2) > sms)) return printf("%d SMs, %d rows of %d chunks: %d\\n", sms, rows, chunks, C), 1;
      }
  return !(lrs::logprobs_cluster(18993, 1, 152) == 8 && lrs::logprobs_cluster(16033, 64, 152) == 4 && lrs::logprobs_cluster(2001, 4099, 152) == 1);
}
""")
    subprocess.run([lbuild.nvcc(), *lbuild.ARCH, "-std=c++17", "-I", os.path.join(root, "layer_range_stage_gb300", "csrc"), "-o", str(tmp_path / "cluster"), str(src)], check=True, capture_output=True)
    r = subprocess.run([str(tmp_path / "cluster")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_late_calls_are_counted_from_none_to_sixteen():
    lib = L.lib()
    for calls in (-1, 17, 1 << 20):
        assert lib.stage_op_f8_debug_late(calls) == L.STAGE_E_INVALID and lib.stage_op_last_error().decode()
    assert lib.stage_op_f8_debug_late(16) == L.STAGE_OK and lib.stage_op_f8_debug_late(0) == L.STAGE_OK
    for calls in (17, 1 << 32, -(1 << 40)):
        with pytest.raises(L.StageError):
            L.stage_op_f8_debug_late(calls)


class Sized:
    """What the binding asks of a device tensor, at sizes that no test allocates: rows side by side."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape

    def get_device(self):
        return 0

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_binding_refuses_sizes_that_a_c_int_would_cut_off(monkeypatch):
    """With 2^32 rows cut to none a call would return and do nothing."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(L.binding, "_launch_on", lambda stream, dev: 0)
    f32, i32, f64, f8 = torch.float32, torch.int32, torch.float64, torch.float8_e4m3fn
    for n in (1 << 32, (1 << 32) + (1 << 40), 1 << 31):
        calls = [
            lambda: L.stage_op_norm_f8(Sized(f32, n, 256), Sized(f8, n, 256), Sized(f32, 2, n)),
            lambda: L.stage_op_norm_f8(Sized(f32, 0, n + 256), y=Sized(f32, 0, n + 256)),
            lambda: L.stage_op_f8_gemm(Sized(f8, n, 256), Sized(f32, 2, n), Sized(f8, 128, 256), Sized(f32, 1, 2), Sized(f32, n, 128)),
            lambda: L.stage_op_f8_gemm(Sized(f8, 0, 256), Sized(f32, 2, 0), Sized(f8, n + 128, 256), Sized(f32, n // 128 + 1, 2), Sized(f32, 0, n + 128)),
            lambda: L.stage_op_f8_gemm(Sized(f8, 0, n + 256), Sized(f32, n // 128 + 2, 0), Sized(f8, 128, n + 256), Sized(f32, 1, n // 128 + 2), Sized(f32, 0, 128)),
            lambda: L.stage_op_rope(Sized(f32, n, 2, 64), None, Sized(i32, n), Sized(f64, 32)),
            lambda: L.stage_op_rope(Sized(f32, 0, n + 2, 64), None, Sized(i32, 0), Sized(f64, 32)),
            lambda: L.stage_op_rope(Sized(f32, 0, 2, 64), Sized(f32, 0, n + 2, 64), Sized(i32, 0), Sized(f64, 32)),
            lambda: L.stage_op_rope(Sized(f32, 0, 2, n + 64), None, Sized(i32, 0), Sized(f64, 32)),
            lambda: L.stage_op_rope(Sized(f32, 0, 2, 64), None, Sized(i32, 0), Sized(f64, n + 32)),
            lambda: L.stage_op_logprobs(Sized(f32, n, 50), entropy=Sized(f32, n)),
            lambda: L.stage_op_logprobs(Sized(f32, 0, n + 50), entropy=Sized(f32, 0)),
            lambda: L.stage_op_logprobs(Sized(f32, 0, 50), top_ids=Sized(i32, 0, n + 3)),
            lambda: L.stage_op_f8_debug_stall(n if n > 1 << 31 else 1 << 33),
        ]
        for i, call in enumerate(calls):
            with pytest.raises(L.StageError) as e:
                call()
            assert e.value.code == L.STAGE_E_INVALID, (n, i)
    # the same calls of ordinary sizes reach the entry points, which do nothing for no rows
    L.stage_op_norm_f8(Sized(f32, 0, 256), Sized(f8, 0, 256), Sized(f32, 2, 0))
    L.stage_op_f8_gemm(Sized(f8, 0, 256), Sized(f32, 2, 0), Sized(f8, 128, 256), Sized(f32, 1, 2), Sized(f32, 0, 128))
    L.stage_op_rope(Sized(f32, 0, 2, 64), Sized(f32, 0, 2, 64), Sized(i32, 0), Sized(f64, 32))
    L.stage_op_logprobs(Sized(f32, 0, 50), top_ids=Sized(i32, 0, 3))


def test_the_product_has_the_registers_that_its_warpgroups_share_out(tmp_path):
    """From a kernel with fewer, the warpgroup that asks for more would wait forever (the launch refuses it)."""
    import os
    import re
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = os.path.join(root, "layer_range_stage_gb300", "csrc", "kernels_f8_gemm.cu")
    r = subprocess.run([lbuild.nvcc(), *lbuild.ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(root, "include"), "-Xptxas", "-v", "-c", src,
                        "-o", str(tmp_path / "x.o")], capture_output=True, text=True, check=True)
    text = open(src).read()
    start, roles, sums = (int(re.search(rf"\b{n} = (\d+)", text).group(1)) for n in ("kRegsStart", "kRegsRoles", "kRegsSums"))
    assert 128 * roles + 256 * sums <= 384 * start
    found = {n: int(v) for n, v in re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", r.stderr, re.S) if "14f8_gemm_kernel" in n}
    assert len(found) == 3 and set(found.values()) == {start}, found
