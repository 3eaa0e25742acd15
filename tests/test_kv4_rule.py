"""Which kernel attention over the paged 4-bit cache runs on, and sizes that no call accepts (no GPU)."""
import pytest

import layer_range_stage_gb300 as L
from layer_range_stage_gb300 import build as lbuild

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    lbuild.build()


def many(n_seqs, n_tok, hq, hkv, max_q, max_len, dtype=torch.float32, d=128):
    return L.stage_op_kv4_attention_many(n_seqs, n_tok, hq, hkv, d, dtype, max_q, max_len)


def test_few_and_many_columns():
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        assert not many(64, 64, 64, 8, 1, 1 << 20, dtype)            # decode, whatever the lengths
        assert not many(16, 80, 32, 8, 5, 1 << 20, dtype)            # 20 columns
        assert many(4, 2048, 32, 8, 512, 512, dtype)                 # prompts
        assert not many(1, 33, 2, 1, 33, 100, dtype)                 # too short to be worth it
        assert many(1, 40, 8, 2, 40, 1 << 28, dtype)
        assert not many(200, 200, 8, 2, 1, 90, dtype)
    assert many(16, 128, 32, 8, 8, 4096, torch.bfloat16) and not many(16, 128, 32, 8, 8, 4096)


def test_the_choice_follows_the_measured_times():
    """16 sequences of 4096 on 8 KV heads: 32 columns take 99 us on the kernel for few at head_dim 128 (tiles: 111, 82, 76) and 64 at 64 (93,
    78, 70); 64 columns 185 and 117."""
    types = (torch.float32, torch.float16, torch.bfloat16)
    assert [many(16, 128, 32, 8, 8, 4096, t) for t in types] == [False, True, True]
    assert [many(16, 128, 32, 8, 8, 4096, t, d=64) for t in types] == [False, False, False]
    assert all(many(16, 256, 32, 8, 16, 4096, t, d) for t in types for d in (64, 128))
    assert not any(many(4, 64, 32, 8, 16, 512, t, d) for t in types[:1] for d in (64, 128))
    assert all(many(4, 256, 32, 8, 64, 512, t, d) for t in types for d in (64, 128))


def test_no_sequence_has_more_tokens_than_the_call():
    assert not many(1, 5, 32, 8, 1 << 20, 1 << 20) and many(1, 500, 32, 8, 1 << 20, 1 << 20)
    assert not many(0, 500, 32, 8, 512, 1 << 20) and not many(4, 0, 32, 8, 512, 1 << 20)


def test_sizes_that_no_call_accepts():
    good = dict(n_seqs=4, n_tok=9, n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=torch.float32, max_q=3, max_len=100)
    assert L.stage_op_kv4_attention_many(**good) is False
    for kw in (dict(n_seqs=-1), dict(n_seqs=65536), dict(n_tok=-1), dict(n_tok=(1 << 24) + 1), dict(n_q_heads=0), dict(n_q_heads=9), dict(n_q_heads=1026),
               dict(n_kv_heads=0), dict(head_dim=96), dict(dtype=torch.float64), dict(max_q=0), dict(max_q=(1 << 20) + 1), dict(max_len=0),
               dict(max_len=(1 << 30) + 1), dict(max_q=(1 << 32) + 3), dict(max_len=(1 << 32) + 100), dict(n_seqs=1 << 32)):
        with pytest.raises(L.StageError) as e:
            L.stage_op_kv4_attention_many(**{**good, **kw})
        assert e.value.code == L.STAGE_E_INVALID, kw


def test_sizes_that_a_c_int_would_cut_off_give_no_bytes():
    assert L.stage_op_kv4_attention_workspace_bytes(4, 8, 2, 64, 3, (1 << 32) + 100) == 0
    assert L.stage_op_kv4_attention_workspace_bytes(4, 8, 2, 64, (1 << 32) + 3, 100) == 0
    assert L.stage_op_kv4_cache_bytes(4, (1 << 32) + 16, 2, 64) == 0 and L.stage_op_kv4_cache_bytes((1 << 64) + 4, 16, 2, 64) == 0


def test_bounds_too_loose_to_look_through_run_on_the_kernel_for_few():
    """2^30 row tiles at the bounds: their places alone would take a tenth of a second to look through."""
    assert many(65535, 1 << 17, 64, 8, 1 << 14, 1 << 16)              # 2^14 * 8 / 128 row tiles * 8 heads * 65535
    assert not many(65535, 1 << 20, 64, 8, 1 << 20, 1 << 16)
    assert not many(65535, 1 << 24, 1024, 8, 1 << 20, 1 << 20, torch.bfloat16)
