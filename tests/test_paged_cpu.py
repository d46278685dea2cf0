"""The paged calls' host-side checks, and the quantiser's reference (no GPU)."""
import ctypes

import numpy as np
import pytest

import paged_ref as ref
import weight_streaming_q4_gb300 as q4
from weight_streaming_q4_gb300 import build

A = 4096    # a 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q4.lib()


def kv(**over):
    d = dict(k_pages=A, v_pages=A, k_scales=A, v_scales=A, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, type=q4.Q4_KV_Q8)
    d.update(over)
    return q4.PagedKV(**d)


def batch(**over):
    d = dict(token_starts=A, kv_lens=A, page_table=A, n_seqs=2, n_tokens=4, table_width=3, max_new=2)
    d.update(over)
    return q4.PagedBatch(**d)


BAD_KV = [dict(k_pages=None), dict(v_pages=None), dict(k_scales=None), dict(v_scales=None), dict(n_pages=0), dict(page_size=8), dict(page_size=48),
          dict(page_size=512), dict(n_kv_heads=0), dict(head_dim=32), dict(head_dim=96), dict(head_dim=320), dict(type=2), dict(type=-1),
          dict(n_pages=1 << 27)]
BAD_BATCH = [dict(token_starts=None), dict(kv_lens=None), dict(page_table=None), dict(n_seqs=-1), dict(n_seqs=65536), dict(n_tokens=-1),
             dict(table_width=0), dict(table_width=1 << 27), dict(max_new=-1)]


def calls(lib, k, b, ld=128, kind=0, row=A):
    ws = q4.q4_attn_paged_workspace_bytes(4, 2, 64)
    return [lib.q4_paged_write(k, b, row, A, kind, ld, None), lib.q4_paged_read(k, b, row, A, kind, ld, None),
            lib.q4_attn_paged(k, b, row, kind, 2 * ld, 4, 0, 0, A, 2 * ld, A, ws, None)]


@pytest.mark.parametrize("over", BAD_KV, ids=str)
def test_cache_checks(lib, over):
    assert calls(lib, kv(**over), batch()) == [q4.Q4_ERR_ARG] * 3


@pytest.mark.parametrize("over", BAD_BATCH, ids=str)
def test_batch_checks(lib, over):
    assert calls(lib, kv(), batch(**over)) == [q4.Q4_ERR_ARG] * 3


def test_positions_of_all_heads_are_counted_in_31_bits(lib):
    widest = (1 << 30) // 16
    assert calls(lib, kv(n_kv_heads=2, page_size=16), batch(table_width=widest)) == [q4.Q4_ERR_ARG] * 3          # 2^31
    assert calls(lib, kv(n_kv_heads=1, page_size=16), batch(table_width=widest + 1), ld=64) == [q4.Q4_ERR_ARG] * 3
    # (taken: the next check, of the rows, refuses)
    assert calls(lib, kv(n_kv_heads=2, page_size=16), batch(table_width=widest - 1), row=A + 8) == [q4.Q4_ERR_ALIGN] * 3


def test_null_structs(lib):
    assert lib.q4_paged_write(None, batch(), A, A, 0, 128, None) == q4.Q4_ERR_ARG
    assert lib.q4_paged_read(kv(), None, A, A, 0, 128, None) == q4.Q4_ERR_ARG


def test_row_checks(lib):
    assert calls(lib, kv(), batch(), row=None) == [q4.Q4_ERR_ARG] * 3
    assert calls(lib, kv(), batch(), kind=2) == [q4.Q4_ERR_ARG] * 3
    assert calls(lib, kv(), batch(), ld=124) == [q4.Q4_ERR_ARG] * 3             # shorter than the row
    assert calls(lib, kv(), batch(), ld=129) [:2] == [q4.Q4_ERR_ALIGN] * 2      # rows not 16-byte aligned
    assert calls(lib, kv(), batch(), row=A + 8) == [q4.Q4_ERR_ALIGN] * 3
    for over in (dict(k_pages=A + 8), dict(v_pages=A + 2), dict(k_scales=A + 8), dict(v_scales=A + 4)):
        assert calls(lib, kv(**over), batch()) == [q4.Q4_ERR_ALIGN] * 3
    for over in (dict(token_starts=A + 2), dict(kv_lens=A + 1), dict(page_table=A + 3)):
        assert calls(lib, kv(), batch(**over)) == [q4.Q4_ERR_ALIGN] * 3


def test_attention_checks(lib):
    ws = q4.q4_attn_paged_workspace_bytes(4, 2, 64)
    assert ws > 0

    def f(n_q=4, window=0, sinks=0, out=A, out_ld=256, w=A, nb=ws, q_ld=256, k=None):
        return lib.q4_attn_paged(k or kv(), batch(), A, 0, q_ld, n_q, window, sinks, out, out_ld, w, nb, None)

    for over in (dict(n_q=3), dict(n_q=1), dict(n_q=0), dict(n_q=130), dict(window=-1), dict(window=4, sinks=-1), dict(sinks=1), dict(out=None),
                 dict(w=None), dict(out_ld=255), dict(q_ld=252), dict(n_q=8)):
        assert f(**over) == q4.Q4_ERR_ARG, over
    assert f(out=A + 8) == q4.Q4_ERR_ALIGN
    assert f(out_ld=260) == q4.Q4_ERR_ALIGN
    assert f(w=A + 8) == q4.Q4_ERR_ALIGN
    assert f(nb=ws - 1) == q4.Q4_ERR_OOM


def test_workspace_sizes(lib):
    assert q4.q4_attn_paged_workspace_bytes(32, 8, 128) % 16 == 0
    for bad in ((0, 1, 64), (3, 2, 64), (65, 1, 64), (4, 2, 96), (4, 0, 64), (4, 2, 320)):
        assert q4.q4_attn_paged_workspace_bytes(*bad) == 0


def test_nothing_to_do_is_not_an_error(lib):
    assert calls(lib, kv(), batch(n_seqs=0, token_starts=None, kv_lens=None, page_table=None)) == [q4.Q4_OK] * 3
    assert calls(lib, kv(), batch(n_tokens=0), row=None) == [q4.Q4_OK] * 3


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(64, dtype=torch.float16)
    with pytest.raises(q4.Q4Error) as e:
        q4.PagedKV.of(t, t, 1, 16, 1, 64)
    assert e.value.status == q4.Q4_ERR_ARG
    with pytest.raises(q4.Q4Error):
        q4.PagedBatch.of(torch.zeros(2, dtype=torch.int32), None, None, 1, 1, 1, 1)


def test_quantiser_reference():
    x = np.zeros((5, 64), np.float32)
    x[0, :32] = np.arange(32) - 16          # |x| <= 16: d = f16(16 / 127)
    x[1, 3] = 1e-9                          # d rounds to zero: everything stands for zero
    x[2, 40] = np.inf
    x[3, 5] = np.nan
    x[4, 7] = 3e38                          # d overflows binary16
    code, d = ref.quantise(x)
    v = ref.values(code, d)
    assert d[0, 0] == np.float16(16 / 127) and abs(int(code[0, 0])) == 127 and not code[0, 32:].any()
    assert np.abs(v[0, :32].astype(np.float64) - x[0, :32]).max() <= 0.5 * float(d[0, 0]) + 2.0 ** -11 * 16
    assert d[1, 0] == 0 and not v[1].any()
    assert np.isnan(v[2, 32:]).all() and not v[2, :32].any()
    assert np.isnan(v[3, :32]).all() and np.isnan(v[4, :32]).all() and not code[4].any()


def test_quantiser_is_the_same_in_32_bits():
    """d and the codes of fp32 divisions are those of exact arithmetic, at values made to sit next to ties."""
    rng = np.random.default_rng(5)
    d = np.abs(rng.normal(size=4000).astype(np.float16)).astype(np.float32)
    n = rng.integers(0, 127, size=4000).astype(np.float32) + np.float32(0.5)
    x = d * n                               # exact: 11 + 8 bits
    for side in (x, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(0))):
        assert np.array_equal(np.rint(side / d), np.rint(side.astype(np.float64) / d.astype(np.float64)))
    h = np.abs(rng.normal(size=4000).astype(np.float16))
    mid = (h.astype(np.float64) + np.nextafter(h, np.float16(np.inf)).astype(np.float64)) / 2
    a = (127 * mid).astype(np.float32)      # exact: 7 + 12 bits
    for side in (a, np.nextafter(a, np.float32(np.inf)), np.nextafter(a, np.float32(0))):
        want = (side.astype(np.float64) / 127.0).astype(np.float16)
        assert np.array_equal((side / np.float32(127)).astype(np.float16), want)
