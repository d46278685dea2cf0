"""What the paged calls' binding refuses of tensors (no GPU: host tensors that are taken for the current device's)."""
import pytest

import weight_streaming_q4_gb300 as q4
from weight_streaming_q4_gb300 import _lib

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def on_device(monkeypatch):
    monkeypatch.setattr(_lib, "_device", lambda: -1)      # (a host tensor's device)


def refused(f, *args, **kw):
    with pytest.raises(q4.Q4Error) as e:
        f(*args, **kw)
    return e.value.status == q4.Q4_ERR_ARG


N_PAGES, PAGE, HEADS, HD = 3, 16, 2, 64
SHAPE = (N_PAGES, HEADS, PAGE, HD)
SIZES = (N_PAGES, PAGE, HEADS, HD)


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


SCALES = SHAPE[:-1] + (HD // 32,)


def test_caches_of_their_type_and_size_are_taken():
    for t in (f16(*SHAPE), f16(*SHAPE).view(torch.int16), f16(N_PAGES + 1, *SHAPE[1:]), f16(N_PAGES * HEADS * PAGE * HD)):
        kv = q4.PagedKV.of(t, t, *SIZES)
        assert kv.k_pages == t.data_ptr() and kv.k_scales is None
    for t in (i8(*SHAPE), i8(*SHAPE).view(torch.uint8)):
        s = f16(*SCALES)
        kv = q4.PagedKV.of(t, t, *SIZES, q4.Q4_KV_Q8, s, s)
        assert kv.v_pages == t.data_ptr() and kv.v_scales == s.data_ptr()
    assert q4.PagedKV.of(4096, 4096, *SIZES).k_pages == 4096


@pytest.mark.parametrize("sizes", [(N_PAGES + 1, PAGE, HEADS, HD), (N_PAGES, 2 * PAGE, HEADS, HD), (N_PAGES, PAGE, HEADS + 1, HD),
                                   (N_PAGES, PAGE, HEADS, 2 * HD)], ids=str)
def test_caches_smaller_than_stated_are_refused(sizes):
    t, big = f16(*SHAPE), f16(2, *SHAPE)
    assert refused(q4.PagedKV.of, t, big, *sizes) and refused(q4.PagedKV.of, big, t, *sizes)
    c, bigc, s, bigs = i8(*SHAPE), i8(2, *SHAPE), f16(*SCALES), f16(2, *SCALES)
    assert refused(q4.PagedKV.of, c, bigc, *sizes, q4.Q4_KV_Q8, bigs, bigs)
    assert refused(q4.PagedKV.of, bigc, bigc, *sizes, q4.Q4_KV_Q8, s, bigs)
    assert refused(q4.PagedKV.of, bigc, bigc, *sizes, q4.Q4_KV_Q8, bigs, s)


def test_caches_of_another_type_are_refused():
    t, c, s = f16(*SHAPE), i8(*SHAPE), f16(*SCALES)
    for bad in (t.bfloat16(), t.float(), c, c.view(torch.uint8)):
        assert refused(q4.PagedKV.of, bad, t, *SIZES) and refused(q4.PagedKV.of, t, bad, *SIZES)
    for bad in (t, t.float()):
        assert refused(q4.PagedKV.of, bad, c, *SIZES, q4.Q4_KV_Q8, s, s) and refused(q4.PagedKV.of, c, bad, *SIZES, q4.Q4_KV_Q8, s, s)
    for bad in (s.float(), s.bfloat16()):
        assert refused(q4.PagedKV.of, c, c, *SIZES, q4.Q4_KV_Q8, bad, s) and refused(q4.PagedKV.of, c, c, *SIZES, q4.Q4_KV_Q8, s, bad)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_batches_of_their_sizes_are_taken():
    for table in (i32(3, 5), i32(4, 5), i32(15)):
        b = q4.PagedBatch.of(i32(4), i32(3), table, 3, 7, 5, 2)
        assert b.page_table == table.data_ptr() and b.n_seqs == 3
    assert q4.PagedBatch.of(i32(2), i32(1), i32(1, 9), 1, 7, 5, 2).table_width == 5       # one row: its first entries
    assert q4.PagedBatch.of(None, None, None, 0, 0, 1, 0).n_seqs == 0
    assert q4.PagedBatch.of(i32(0), i32(0), i32(0, 5), 0, 4, 5, 0).n_seqs == 0


def test_batches_of_other_sizes_or_types_are_refused():
    assert refused(q4.PagedBatch.of, i32(3), i32(3), i32(3, 5), 3, 7, 5, 2)
    assert refused(q4.PagedBatch.of, i32(4), i32(2), i32(3, 5), 3, 7, 5, 2)
    assert refused(q4.PagedBatch.of, i32(4), i32(3), i32(2, 5), 3, 7, 5, 2)
    assert refused(q4.PagedBatch.of, i32(4), i32(3), i32(14), 3, 7, 5, 2)
    assert refused(q4.PagedBatch.of, i32(4), i32(3), i32(3, 6), 3, 7, 5, 2)       # rows 6 apart, read as 5 apart
    for bad in (torch.float32, torch.int64, torch.int16):
        assert refused(q4.PagedBatch.of, i32(4).to(bad), i32(3), i32(3, 5), 3, 7, 5, 2)
        assert refused(q4.PagedBatch.of, i32(4), i32(3).to(bad), i32(3, 5), 3, 7, 5, 2)
        assert refused(q4.PagedBatch.of, i32(4), i32(3), i32(3, 5).to(bad), 3, 7, 5, 2)
    assert refused(q4.PagedBatch.of, i32(4), i32(3), i32(5, 3).T, 3, 7, 5, 2)


class Lib:
    """Stands for the library: notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def q4_status_string(self, st):
        return b"refused"

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or q4.Q4_OK


@pytest.fixture()
def calls(monkeypatch):
    stub = Lib()
    monkeypatch.setattr(_lib, "lib", lambda: stub)
    return stub.calls


ROWS, ROW = 5, HEADS * HD


def write(x, ld, kind=q4.Q4_TYPE_F32, rows=ROWS, other=4096):
    kv = q4.PagedKV.of(4096, 4096, *SIZES)
    b = q4.PagedBatch.of(4096, 4096, 4096, 1, rows, 3, 1)
    q4.q4_paged_write(kv, b, x, other, kind, ld, stream=0)


def test_rows_of_their_layout_are_taken(calls):
    wide = torch.zeros(ROWS, 4 * ROW)
    good = [(wide, 4 * ROW), (wide[:, ROW:], 4 * ROW), (wide[:, 3 * ROW:], 4 * ROW), (torch.zeros(ROWS, HEADS, HD), ROW), (torch.zeros(ROWS * ROW), ROW),
            (torch.zeros(ROWS * HEADS, HD), ROW), (torch.zeros(2 * ROWS, ROW), ROW), (torch.zeros(2 * ROWS, ROW)[ROWS:], ROW), (wide.view(ROWS, 4 * HEADS, HD)[:, HEADS:2 * HEADS], 4 * ROW)]
    for x, ld in good:
        write(x, ld)
    for x in (f16(ROWS, ROW), f16(ROWS, ROW).view(torch.int16)):
        write(x, ROW, q4.Q4_TYPE_F16)
    write(torch.zeros(1, ROW), 4 * ROW, rows=1)
    write(wide[:1, :ROW], ROW, rows=1)
    assert len(calls) == len(good) + 4


def test_rows_of_another_type_or_layout_are_refused(calls):
    x = torch.zeros(ROWS, ROW)
    for bad in (x.half().bfloat16(), x):
        assert refused(write, bad, ROW, q4.Q4_TYPE_F16)
    for bad in (x.half(), x.int(), x.double()):
        assert refused(write, bad, ROW)
    wide = torch.zeros(ROWS, 4 * ROW)
    assert refused(write, torch.zeros(ROW, ROWS).T, ROW)                  # transposed
    assert refused(write, x, ROW, rows=6) and refused(write, x[:, :HD], ROW, rows=6) and refused(write, torch.zeros(ROWS, HD), ROW)      # too few
    assert refused(write, wide[:, :ROW], ROW)                             # rows 4 * ROW apart
    assert refused(write, wide, ROW)
    assert refused(write, torch.zeros(2 * ROWS, ROW)[::2], ROW)
    assert refused(write, torch.zeros(ROW).expand(ROWS, ROW), ROW)        # one row for all
    assert refused(write, torch.zeros(ROWS, 2 * ROW)[:, ::2], 2 * ROW)    # values two apart
    assert refused(write, torch.zeros(ROWS, HD, HEADS).transpose(1, 2), ROW)
    assert refused(write, torch.zeros(2 * ROWS * ROW)[::2], ROW)
    assert refused(write, 4096, ROW, other=x.T)
    kv, b = q4.PagedKV.of(4096, 4096, *SIZES), q4.PagedBatch.of(4096, 4096, 4096, 1, ROWS, 3, 1)
    assert refused(q4.q4_paged_read, kv, b, 4096, x.T, q4.Q4_TYPE_F32, ROW, stream=0)
    assert refused(q4.q4_attn_paged, kv, b, x.T, q4.Q4_TYPE_F32, ROW, HEADS, 0, 0, 4096, ROW, 4096, 1 << 30, stream=0)
    for out in (f16(ROW, ROWS).T, x, x.bfloat16()):
        assert refused(q4.q4_attn_paged, kv, b, x, q4.Q4_TYPE_F32, ROW, HEADS, 0, 0, out, ROW, 4096, 1 << 30, stream=0)
    assert not calls


def test_a_workspace_smaller_than_stated_is_refused(calls):
    kv, b = q4.PagedKV.of(4096, 4096, *SIZES), q4.PagedBatch.of(4096, 4096, 4096, 1, ROWS, 3, 1)

    def attend(ws, n):
        q4.q4_attn_paged(kv, b, torch.zeros(ROWS, ROW), q4.Q4_TYPE_F32, ROW, HEADS, 0, 0, f16(ROWS, ROW), ROW, ws, n, stream=0)

    for ws in (torch.zeros(4095, dtype=torch.uint8), torch.zeros(1023), torch.zeros(0), torch.zeros(64, 128).T):
        assert refused(attend, ws, 4096)
    assert not calls
    for ws in (torch.zeros(4096, dtype=torch.uint8), torch.zeros(1024), 4096):
        attend(ws, 4096)
    assert len(calls) == 3


def test_descriptors_of_another_device_than_the_current_one_are_refused(calls, monkeypatch):
    t = f16(*SHAPE)
    kv, b = q4.PagedKV.of(t, t, *SIZES), q4.PagedBatch.of(i32(2), i32(1), i32(1, 3), 1, ROWS, 3, 1)
    plain = q4.PagedKV.of(4096, 4096, *SIZES), q4.PagedBatch.of(4096, 4096, 4096, 1, ROWS, 3, 1)

    def each(kv, b):
        return [(q4.q4_paged_write, kv, b, 4096, 4096, q4.Q4_TYPE_F32, ROW), (q4.q4_paged_read, kv, b, 4096, 4096, q4.Q4_TYPE_F32, ROW),
                (q4.q4_attn_paged, kv, b, 4096, q4.Q4_TYPE_F32, ROW, HEADS, 0, 0, 4096, ROW, 4096, 1 << 30)]

    for f, *args in each(kv, b) + each(*plain):
        f(*args, stream=0)
    assert len(calls) == 6
    monkeypatch.setattr(_lib, "_device", lambda: 1)
    for f, *args in each(kv, plain[1]) + each(plain[0], b):
        assert refused(f, *args, stream=0)
    for x in (torch.zeros(ROWS, ROW), torch.zeros(ROWS * ROW)):
        assert refused(q4.q4_paged_write, *plain, x, 4096, q4.Q4_TYPE_F32, ROW, stream=0)
    assert refused(q4.q4_attn_paged, *plain, 4096, q4.Q4_TYPE_F32, ROW, HEADS, 0, 0, 4096, ROW, f16(64), 128, stream=0)
    for f, *args in each(*plain):
        f(*args, stream=0)
    assert len(calls) == 9


def test_query_rows_of_a_head_are_counted_in_30_bits():
    """(the library itself: fake addresses, which the next check refuses)"""
    from weight_streaming_q4_gb300 import build
    build.build()
    lib = q4.lib()
    ws = q4.q4_attn_paged_workspace_bytes(64, 1, 64)
    kv = q4.PagedKV(k_pages=4096, v_pages=4096, n_pages=8, page_size=16, n_kv_heads=1, head_dim=64, type=q4.Q4_KV_F16)

    def attend(n_tokens, n_q=64):
        b = q4.PagedBatch(token_starts=4096, kv_lens=4096, page_table=4096, n_seqs=1, n_tokens=n_tokens, table_width=3, max_new=1)
        return lib.q4_attn_paged(kv, b, 4096, 1, 4096, n_q, 0, 0, 4096, 4096, 4096 + 8, ws, None)       # the workspace: not aligned

    assert attend(1 << 24) == q4.Q4_ERR_ALIGN and attend(1 << 30, 1) == q4.Q4_ERR_ALIGN
    for n_tokens, n_q in (((1 << 24) + 1, 64), (1 << 25, 64), (1 << 26, 64), ((1 << 31) - 1, 2), ((1 << 30) + 1, 1)):
        assert attend(n_tokens, n_q) == q4.Q4_ERR_ARG
