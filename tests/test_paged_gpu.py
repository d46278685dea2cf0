"""q4_paged_write, q4_paged_read and q4_attn_paged on the GPU against a plain 64-bit implementation (paged_ref.py)."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import weight_streaming_q4_gb300 as q4
from weight_streaming_q4_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    yield
    assert q4.q4_device_status() == 0, "a kernel wait failed"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Dev:
    """A ref.Cache on the GPU, with its descriptors."""

    def __init__(self, c, max_new=None):
        self.c = c
        self.pages = {n: dev(c.pages[n]) for n in "kv"}
        self.scales = {n: dev(c.scales[n]) if c.q8 else None for n in "kv"}
        self.starts, self.lens, self.table = dev(c.starts), dev(c.lens), dev(c.table)
        self.kv = q4.PagedKV.of(self.pages["k"], self.pages["v"], c.n_pages, c.page, c.n_kv, c.hd,
                                q4.Q4_KV_Q8 if c.q8 else q4.Q4_KV_F16, self.scales["k"], self.scales["v"])
        self.batch = q4.PagedBatch.of(self.starts, self.lens, self.table, len(c.new), c.n_tokens, c.width,
                                      max(c.new + [0]) if max_new is None else max_new)

    def attend(self, q, n_q, window=0, sinks=0, pad=0, stream=None, fill=7.0):
        """Rows pad values apart beyond their own; out starts as `fill`.  Returns the whole buffer as float64."""
        c = self.c
        row = n_q * c.hd
        kind = q4.Q4_TYPE_F32 if q.dtype == np.float32 else q4.Q4_TYPE_F16
        wide = np.full((c.n_tokens, row + pad), np.nan, q.dtype)
        wide[:, :row] = q
        qd = dev(wide)
        out = torch.full((c.n_tokens, row + pad), fill, dtype=torch.float16, device="cuda")
        nb = q4.q4_attn_paged_workspace_bytes(n_q, c.n_kv, c.hd)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        q4.q4_attn_paged(self.kv, self.batch, qd, kind, row + pad, n_q, window, sinks, out, row + pad, ws, nb, stream=stream)
        torch.cuda.synchronize()
        return out.cpu().numpy().astype(np.float64)


def queries(c, n_q, seed, f32, scale=1.5):
    q = (np.random.default_rng(seed).normal(size=(c.n_tokens, n_q * c.hd)) * scale).astype(np.float32)
    return q if f32 else q.astype(np.float16)


def check(got, c, q, n_q, window=0, sinks=0, fill=7.0):
    """Every row of a sequence within the bound, every other row and the padding untouched."""
    row = n_q * c.hd
    want, tol = c.attend(q, n_q, window, sinks)
    mine = np.zeros(c.n_tokens, bool)
    for s in range(len(c.new)):
        mine[c.starts[s]:c.starts[s + 1]] = True
    assert np.all(got[~mine] == fill) and np.all(got[:, row:] == fill)
    a, b, t = got[mine, :row], want[mine], tol[mine]
    same = np.isnan(a) & np.isnan(b) | (a == b)
    with np.errstate(invalid="ignore"):
        err = np.abs(a - b)
        bad = ~(same | (err <= t))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside; worst err/tol {np.nanmax(np.where(bad, err / t, 0)):.3g}"


HEADS = [(32, 8, 128), (8, 8, 64), (16, 1, 256), (12, 4, 192), (64, 8, 128), (10, 2, 64), (7, 1, 128), (64, 1, 64), (3, 3, 256), (33, 1, 128)]


@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("f32", [False, True], ids=["qf16", "qf32"])
@pytest.mark.parametrize("n_q,n_kv,hd", HEADS, ids=lambda v: str(v))
def test_heads(n_q, n_kv, hd, f32, q8):
    """Single tokens and a short chunk beside each other, every head layout and type."""
    c = ref.Cache([1, 9, 1], [70, 150, 1], n_kv, hd, 16, q8, seed=n_q + hd)
    q = queries(c, n_q, 1, f32)
    check(Dev(c).attend(q, n_q), c, q, n_q)
    d = Dev(c, max_new=300)      # another kernel choice, the same results
    check(d.attend(q, n_q), c, q, n_q)


@pytest.mark.parametrize("total", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 5000])
@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
def test_single_token_lengths(total, q8):
    c = ref.Cache([1], [total], 2, 128, 16 if total < 300 else 64, q8, seed=total)
    q = queries(c, 8, 2, True)
    check(Dev(c).attend(q, 8), c, q, 8)


@pytest.mark.parametrize("seqs", [1, 3, 12], ids=["one", "few", "many"])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("f32", [False, True], ids=["qf16", "qf32"])
def test_single_tokens_of_every_type(f32, q8, hd, seqs):
    """One token of one, a few and many sequences: the cluster kernel, and the even split with and without an item per CTA."""
    total = [1 + (997 * (i + 1)) % 1500 for i in range(seqs)]
    c = ref.Cache([1] * seqs, total, 2, hd, 32, q8, seed=hd + seqs)
    q = queries(c, 10, 46, f32)
    check(Dev(c).attend(q, 10), c, q, 10)
    check(Dev(c).attend(q, 10, 100, 3), c, q, 10, 100, 3)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 24, 25, 31, 32, 33, 64])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("f32", [False, True], ids=["qf16", "qf32"])
def test_row_counts(f32, q8, hd, rows):
    """Around every number of query rows that a kernel takes at once, few and many items, as one token and as a draft
    whose last rows see more than its first."""
    for seqs in (1, 6):
        total = [40 + (613 * (i + 1)) % 700 for i in range(seqs)]
        c = ref.Cache([1] * seqs, total, 2, hd, 16, q8, seed=rows + hd)
        q = queries(c, 2 * rows, 47, f32)
        check(Dev(c).attend(q, 2 * rows), c, q, 2 * rows)
        c = ref.Cache([rows] + [1] * (seqs - 1), [rows + 33] + total[1:], 2, hd, 16, q8, seed=rows + hd + 1)
        q = queries(c, 2, 48, f32)
        check(Dev(c).attend(q, 2), c, q, 2)
        check(Dev(c).attend(q, 2, 20, 2), c, q, 2, 20, 2)


@pytest.mark.parametrize("new,total", [(1, 1), (2, 2), (31, 31), (32, 33), (33, 200), (64, 64), (65, 130), (127, 300), (128, 128), (129, 129), (200, 777), (257, 1025)])
@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
def test_chunk_lengths(new, total, q8):
    c = ref.Cache([new], [total], 2, 64, 32, q8, seed=new)
    q = queries(c, 6, 3, False)
    check(Dev(c).attend(q, 6), c, q, 6)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_page_sizes(page, hd):
    c = ref.Cache([1, 70, 3], [page * 2 + 1, page + 70, 2 * page - 1], 2, hd, page, page % 64 == 0, seed=page)
    q = queries(c, 4, 4, page % 128 == 0)
    check(Dev(c).attend(q, 4), c, q, 4)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (16, 4), (100, 0), (100, 37), (130, 300), (700, 4), (100000, 3)])
@pytest.mark.parametrize("new,total", [([1, 1], [900, 40]), ([5, 1], [333, 129]), ([150, 1, 40], [700, 3, 40])], ids=["tokens", "draft", "chunk"])
def test_windows(new, total, window, sinks):
    """Pages that no query sees any more are holes, and hold NaN besides: they are not read."""
    for q8 in (False, True):
        c = ref.Cache(new, total, 2, 128, 16, q8, seed=window, spare=3)
        free = [p for p in range(c.n_pages) if p not in set(c.table.reshape(-1))]
        for s in range(len(new)):
            first = max(0, total[s] - new[s] - window + 1)
            for e in range(c.width):
                if e * 16 >= sinks and (e + 1) * 16 <= first:
                    free.append(c.table[s, e])
                    c.table[s, e] = [-1, c.n_pages, 2 ** 31 - 1, -2 ** 31][e % 4]
        for p in free:
            if not q8:
                c.pages["k"][p], c.pages["v"][p] = np.nan, np.inf
            else:
                c.scales["k"][p], c.scales["v"][p] = np.nan, np.inf
        q = queries(c, 8, 5, not q8)
        check(Dev(c).attend(q, 8, window, sinks), c, q, 8, window, sinks)


def test_holes_are_masked():
    """Pages missing inside what a query sees: their positions are as if not there; a row that sees holes alone gets zeros."""
    c = ref.Cache([1, 40, 2], [200, 150, 30], 2, 64, 16, seed=8)
    c.table[0, 3] = c.table[0, 7] = c.table[1, 0] = c.table[1, 5] = -5
    c.table[2, :] = 10 ** 9
    for f32 in (False, True):
        q = queries(c, 4, 6, f32)
        got = Dev(c).attend(q, 4)
        check(got, c, q, 4)
        assert not got[c.starts[2]:c.starts[3]].any()


def test_rows_outside_every_sequence_are_left():
    """Padding behind the last sequence and before the first, empty sequences, zero lengths, rows at negative positions."""
    c = ref.Cache([0, 3, 0, 4, 1, 0], [5, 3, 0, 40, 1, 9], 2, 64, 16, seed=9, n_tokens=20)
    c.starts = (c.starts + 5).astype(np.int32)
    q = queries(c, 4, 7, True)
    check(Dev(c).attend(q, 4, pad=8), c, q, 4)
    for new, total in (([4], [2]), ([3], [0]), ([300], [10])):
        c = ref.Cache(new, total, 1, 128, 16, seed=10)
        q = queries(c, 2, 8, False)
        got = Dev(c).attend(q, 2)
        check(got, c, q, 2)
        assert not got[:new[0] - total[0]].any()


def test_bad_arrays_stay_in_bounds():
    """Starts and lengths outside their ranges are taken within them: sequences that are sound keep their results."""
    c = ref.Cache([2, 3], [40, 50], 2, 64, 16, seed=11)
    q = queries(c, 4, 9, True)
    c.total[1] = c.width * 16
    wide = np.full((2, c.width), 0, np.int32)
    wide[:, :c.table.shape[1]] = np.maximum(c.table, 0)
    c.table = wide
    d = Dev(c)
    d.lens.copy_(torch.tensor([40, 10 ** 9], dtype=torch.int32))
    check(d.attend(q, 4), c, q, 4)
    d.starts.copy_(torch.tensor([-7, 2, 10 ** 9], dtype=torch.int32))
    check(d.attend(q, 4), c, q, 4)


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("chunk", [1, 5, 150])
def test_masked_nan_and_infinity(hd, chunk):
    """Stale slots, later tokens' keys and values, and values outside the window may be NaN or infinite: a query that does not see
    them is as if they were zero, one that does gets what arithmetic gives."""
    c = ref.Cache([chunk, 1], [chunk + 37, 50], 1, hd, 16, seed=12, n_tokens=chunk + 1)
    n = chunk + 37
    for s, length in ((0, n), (1, 50)):       # slots behind the last position
        p, slot = c.table[s, (length - 1) // 16], length % 16
        if slot:
            for name in "kv":
                c.pages[name][p, :, slot:] = np.array([np.nan, np.inf, -np.inf, 6e4])[np.arange(16 - slot) % 4][None, :, None]
    q = queries(c, 3, 10, False, scale=0.5)
    check(Dev(c).attend(q, 3), c, q, 3)
    if chunk > 1:
        # the last token's value: infinite in one column, NaN in another; its key too in another try
        p, slot = c.table[0, (n - 1) // 16], (n - 1) % 16
        c.pages["v"][p, :, slot, 3], c.pages["v"][p, :, slot, 9] = -np.inf, np.nan
        got = Dev(c).attend(q, 3)
        check(got, c, q, 3)
        assert np.isfinite(got[:chunk - 1]).all() and got[chunk - 1, 3] == -np.inf and np.isnan(got[chunk - 1, 9])
        c.pages["k"][p, :, slot, 1] = np.nan
        got = Dev(c).attend(q, 3)
        assert np.isfinite(got[:chunk - 1]).all() and np.isnan(got[chunk - 1]).all()
    # a value that only the first tokens of the window's edge see
    c = ref.Cache([chunk], [chunk + 300], 1, hd, 16, seed=13)
    t = chunk + 300 - 64 - chunk // 2 - 1
    c.pages["v"][c.table[0, t // 16], :, t % 16, 5] = np.inf
    q = queries(c, 3, 11, True, scale=0.5)
    check(Dev(c).attend(q, 3, window=64, sinks=2), c, q, 3, 64, 2)


@pytest.mark.parametrize("chunk", [1, 140])
def test_extreme_scores(chunk):
    """Scores of thousands, equal scores, and a maximum that keeps rising along the sequence."""
    for kind in range(3):
        c = ref.Cache([chunk], [chunk + 500], 1, 128, 64, seed=14 + kind)
        q = queries(c, 4, 12, kind == 0, scale=(40.0, 0.0, 1.0)[kind])
        if kind == 2:
            for t in range(chunk + 500):
                c.pages["k"][c.table[0, t // 64], :, t % 64] = np.float16(t / 60.0)
            q = np.abs(q)
        check(Dev(c).attend(q, 4), c, q, 4)


def test_small_and_large_values():
    """Values near binary16's ends."""
    for q8 in (False, True):
        c = ref.Cache([1, 130], [300, 400], 1, 64, 16, seed=17)
        c.q8 = q8
        for i, name in enumerate("kv"):
            x = c.pages[name].astype(np.float32) * (1 if i == 0 else 1e-5)
            x[: c.n_pages // 2] *= 1 if i == 0 else 1e9
            if q8:
                c.pages[name], c.scales[name] = ref.quantise(x)
            else:
                c.pages[name] = x.astype(np.float16)
        q = queries(c, 4, 13, True)
        check(Dev(c).attend(q, 4), c, q, 4)


@pytest.mark.parametrize("max_new", [1, 8, 64, 5000])
def test_ragged_batches(max_new):
    rng = np.random.default_rng(18)
    new = [int(rng.integers(0, 40)) for _ in range(20)] + [200, 1]
    total = [n + int(rng.integers(0, 500)) for n in new[:-1]] + [3000]
    c = ref.Cache(new, total, 2, 64, 16, True, seed=19, n_tokens=sum(new) + 3)
    q = queries(c, 8, 14, False)
    check(Dev(c, max_new=max_new).attend(q, 8), c, q, 8)


@pytest.mark.parametrize("new,n_kv", [([40], 2), ([3, 70], 1), ([0, 17, 1], 4)])
def test_more_new_tokens_than_the_caller_knew_of(new, n_kv):
    """max_new chooses the kernel alone: too small a value costs time only (few items: the cluster kernel)."""
    c = ref.Cache(new, [n + 60 for n in new], n_kv, 128, 16, n_kv == 2, seed=42)
    q = queries(c, 4 * n_kv, 43, True)
    for max_new in (0, 1, 3):
        check(Dev(c, max_new=max_new).attend(q, 4 * n_kv), c, q, 4 * n_kv)


def test_windows_as_wide_as_an_int():
    c = ref.Cache([40, 5], [20, 300], 2, 64, 16, seed=44)
    q = queries(c, 4, 45, False)
    for max_new in (1, 100):
        for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (2 ** 30, 7)):
            check(Dev(c, max_new=max_new).attend(q, 4, window, sinks), c, q, 4, window, sinks)


def test_many_sequences():
    """More sequences than a block has threads, most of them empty or short."""
    rng = np.random.default_rng(20)
    new = [int(rng.integers(0, 3)) for _ in range(1300)]
    total = [n + int(rng.integers(0, 30)) for n in new]
    c = ref.Cache(new, total, 1, 64, 16, seed=21)
    q = queries(c, 4, 15, True)
    check(Dev(c).attend(q, 4), c, q, 4)


def test_long_context_is_split_and_joined():
    for q8, hd, chunk in ((False, 128, 1), (True, 128, 3), (False, 64, 130), (True, 256, 1)):
        c = ref.Cache([chunk], [40000], 1, hd, 256, q8, seed=22)
        q = queries(c, 4, 16, True)
        check(Dev(c).attend(q, 4), c, q, 4)


@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("f32", [False, True], ids=["xf16", "xf32"])
@pytest.mark.parametrize("n_kv,hd,page", [(8, 128, 64), (1, 64, 16), (3, 192, 32), (2, 256, 256)])
def test_write_and_read(n_kv, hd, page, f32, q8):
    """Writes touch the new tokens' slots alone, bit for bit the reference; reads give back what the cache stands for."""
    c = ref.Cache([3, 0, 40, 1], [3, 7, 90, page + 1], n_kv, hd, page, q8, seed=23, n_tokens=47)
    rng = np.random.default_rng(24)
    row = n_kv * hd
    x = {n: (rng.normal(size=(47, row + 16)) * np.exp(rng.normal(size=(47, 1)) * 3)).astype(np.float32 if f32 else np.float16) for n in "kv"}
    if q8:
        for a in x.values():
            a[1, :40] = 0
            a[2, 33] = np.inf
            a[4, 2] = np.nan
            a[5, :32] = 1e-9
            a[6, :32] *= 1e-4
            a[7, 1] = 1e30 if f32 else 6e4
    d = Dev(c)
    kind = q4.Q4_TYPE_F32 if f32 else q4.Q4_TYPE_F16
    xs = {n: dev(x[n]) for n in "kv"}
    q4.q4_paged_write(d.kv, d.batch, xs["k"], xs["v"], kind, row + 16)
    back = {n: torch.full((47, row + 16), 5.0, dtype=xs["k"].dtype, device="cuda") for n in "kv"}
    q4.q4_paged_read(d.kv, d.batch, back["k"], back["v"], kind, row + 16)
    torch.cuda.synchronize()
    for n in "kv":
        pages, scales = c.pages[n].copy(), c.scales[n].copy() if q8 else None
        want = np.full((47, row + 16), 5.0)
        for s in range(4):
            for i in range(c.new[s]):
                p, r = c.position(s, i), int(c.starts[s]) + i
                v = x[n][r, :row].astype(np.float32).reshape(n_kv, hd)
                at = (c.table[s, p // page], slice(None), p % page)
                if q8:
                    pages[at], scales[at] = ref.quantise(v)
                    v = ref.values(pages[at], scales[at])
                else:
                    with np.errstate(over="ignore"):
                        pages[at] = v = v.astype(np.float16)
                want[r, :row] = v.reshape(-1)
        assert np.array_equal(d.pages[n].cpu().numpy().view(np.uint8), pages.view(np.uint8))
        if q8:
            got = d.scales[n].cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(scales)) and np.array_equal(got[~np.isnan(got)], scales[~np.isnan(scales)])
        got = back[n].cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_codes_next_to_ties():
    """Values on and beside n + 1/2 steps of every kind of scale, subnormal ones too: the codes are those of exact arithmetic."""
    rng = np.random.default_rng(40)
    n = 4096
    c = ref.Cache([n], [n], 1, 64, 256, True, seed=41)
    d = np.abs(rng.normal(size=(n, 2)) * np.exp2(rng.integers(-26, 8, size=(n, 2)))).astype(np.float16)
    d[:64] = np.arange(1, 129, dtype=np.float64).reshape(64, 2) * 2.0 ** -24       # subnormal scales
    d = np.maximum(d, np.float16(2.0 ** -24)).astype(np.float32)
    q = rng.integers(0, 127, size=(n, 2, 32)).astype(np.float32) + np.float32(0.5)
    x = (d[..., None] * q).astype(np.float32)                                      # exact: 11 + 8 bits
    side = rng.integers(-1, 2, size=x.shape)
    x = np.where(side > 0, np.nextafter(x, np.float32(np.inf)), np.where(side < 0, np.nextafter(x, np.float32(0)), x))
    x *= rng.choice([-1, 1], size=x.shape).astype(np.float32)
    x[:, :, 0] = 127 * d                                                           # the maximum that gives this scale
    x = np.clip(x, -127 * d[..., None], 127 * d[..., None]).reshape(n, 64).astype(np.float32)
    dv = Dev(c)
    xd = dev(x)
    q4.q4_paged_write(dv.kv, dv.batch, xd, xd, q4.Q4_TYPE_F32, 64)
    torch.cuda.synchronize()
    codes, scales = ref.quantise(x)
    at = (c.table[0, np.arange(n) // 256], 0, np.arange(n) % 256)
    assert np.array_equal(dv.scales["k"].cpu().numpy()[at], scales)
    assert np.array_equal(dv.pages["k"].cpu().numpy()[at], codes)


def test_write_and_read_skip_holes_and_negative_positions():
    c = ref.Cache([4, 2], [2, 40], 2, 64, 16, seed=25, n_tokens=7)
    c.table[1, 2] = c.n_pages
    d = Dev(c)
    x = torch.randn((7, 128), device="cuda")
    before = {n: d.pages[n].clone() for n in "kv"}
    q4.q4_paged_write(d.kv, d.batch, x, x, q4.Q4_TYPE_F32, 128)
    back = torch.full((2, 7, 128), 3.0, device="cuda")
    q4.q4_paged_read(d.kv, d.batch, back[0], back[1], q4.Q4_TYPE_F32, 128)
    torch.cuda.synchronize()
    assert torch.equal(back[0, 2:4], x[2:4].half().float()) and not back[0, :2].any() and not back[0, 4:6].any()
    assert (back[:, 6] == 3.0).all()
    for n in "kv":      # two rows written, nothing else
        changed = (d.pages[n] != before[n]).any(-1).any(1).sum()
        assert int(changed) == 2


def test_write_attend_read_as_a_server_does():
    """Prompts in chunks, then tokens: every step's write and attention, against the reference's cache; then a page pool read into the
    contiguous bucket, where the one-sequence attention gives the same as the paged one."""
    n_q, n_kv, hd, page = 8, 2, 128, 16
    row = n_kv * hd
    rng = np.random.default_rng(26)
    total = np.zeros(3, int)
    c = ref.Cache([0, 0, 0], [300, 300, 300], n_kv, hd, page, False, seed=27)
    for new in ([100, 1, 0], [60, 40, 3], [1, 1, 1], [1, 1, 1], [2, 0, 5]):
        total = total + new
        c.new, c.total = list(new), [int(t) for t in total]
        c.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        c.lens = total.astype(np.int32)
        c.n_tokens = int(sum(new)) + 1
        d = Dev(c)
        wide = (n_q + 2 * n_kv) * hd
        x = rng.normal(size=(c.n_tokens, wide)).astype(np.float32)
        xd = dev(x)
        q4.q4_paged_write(d.kv, d.batch, xd[:, n_q * hd:], xd[:, n_q * hd + row:], q4.Q4_TYPE_F32, wide)
        out = torch.full((c.n_tokens, n_q * hd), 7.0, dtype=torch.float16, device="cuda")
        nb = q4.q4_attn_paged_workspace_bytes(n_q, n_kv, hd)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        q4.q4_attn_paged(d.kv, d.batch, xd, q4.Q4_TYPE_F32, wide, n_q, 0, 0, out, n_q * hd, ws, nb)
        torch.cuda.synchronize()
        for name in "kv":
            c.pages[name] = d.pages[name].cpu().numpy()
        for s in range(3):
            for i in range(new[s]):
                p, r = c.position(s, i), int(c.starts[s]) + i
                got = c.pages["k"][c.table[s, p // page], :, p % page]
                assert np.array_equal(got.reshape(-1), x[r, n_q * hd:n_q * hd + row].astype(np.float16))
        q = x[:, :n_q * hd]
        check(out.cpu().numpy().astype(np.float64), c, q, n_q)
    # sequence 0 into a bucket of 512 positions
    n = int(total[0])
    bucket = torch.zeros((2, 512, row), dtype=torch.float16, device="cuda")
    one = q4.PagedBatch.of(dev(np.array([0, n], np.int32)), d.lens, d.table, 1, 512, c.width, n)
    q4.q4_paged_read(d.kv, one, bucket[0], bucket[1], q4.Q4_TYPE_F16, row)
    q1 = rng.normal(size=(1, n_q * hd)).astype(np.float32)
    out = torch.empty(n_q * hd, dtype=torch.float16, device="cuda")
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    wb = q4.q4_attn_workspace_bytes(n_q, n_kv, hd, 512)
    q4.q4_attn_decode(dev(q1), bucket[0], bucket[1], ctx, 512, n_q, n_kv, hd, out, torch.zeros(wb, dtype=torch.uint8, device="cuda"), wb)
    torch.cuda.synchronize()
    k, _ = c.stored("k", 0, n)
    assert np.array_equal(bucket[0, :n].cpu().numpy().astype(np.float64).reshape(n, n_kv, hd).transpose(1, 0, 2), k)
    assert not bucket[:, n:].any()
    c.new, c.total, c.starts, c.lens, c.n_tokens = [1], [n], np.array([0, 1], np.int32), np.array([n], np.int32), 1
    want, tol = c.attend(q1, n_q)
    assert np.all(np.abs(out.cpu().numpy().astype(np.float64) - want[0]) <= tol[0])
    check(Dev(c).attend(q1, n_q), c, q1, n_q)


@pytest.mark.parametrize("chunk", [1, 150])
def test_one_graph_serves_every_content_of_the_batch(chunk):
    """Captured once, replayed after lengths, starts and table changed; two graphs share a workspace, one after the other."""
    n_q, n_kv, hd = 8, 2, 128
    big = ref.Cache([chunk, chunk], [900, 700], n_kv, hd, 16, True, seed=28, n_tokens=2 * chunk + 2)
    d = Dev(big)
    q = queries(big, n_q, 17, True)
    qd = dev(q)
    out = torch.full((2, big.n_tokens, n_q * hd), 7.0, dtype=torch.float16, device="cuda")
    nb = q4.q4_attn_paged_workspace_bytes(n_q, n_kv, hd)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    graphs = []
    for i, window in enumerate((0, 50)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            q4.q4_attn_paged(d.kv, d.batch, qd, q4.Q4_TYPE_F32, n_q * hd, n_q, window, 0, out[i], n_q * hd, ws, nb, stream=s)
            s.synchronize()
            with torch.cuda.graph(g, stream=s):
                q4.q4_attn_paged(d.kv, d.batch, qd, q4.Q4_TYPE_F32, n_q * hd, n_q, window, 0, out[i], n_q * hd, ws, nb, stream=s)
        graphs.append(g)
    for new, total in (([1, chunk], [1, 700]), ([chunk, 0], [chunk, 50]), ([chunk, chunk], [900, 651])):
        big.new, big.total = new, total
        big.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        d.starts.copy_(dev(big.starts))
        d.lens.copy_(torch.tensor(total, dtype=torch.int32))
        big.table = big.table[::-1].copy() if total[1] < 700 and total[0] < 700 else big.table
        d.table.copy_(dev(big.table))
        out.fill_(7.0)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, window in enumerate((0, 50)):
            check(out[i].cpu().numpy().astype(np.float64), big, q, n_q, window)


def test_calls_on_two_streams_at_once():
    """Calls with workspaces of their own do not disturb one another, and each equals the call alone, bit for bit."""
    n_q, n_kv, hd = 8, 2, 128
    work = []
    for i, chunk in enumerate((1, 150, 4, 300)):
        c = ref.Cache([chunk, 2], [2000 + i, 500], n_kv, hd, 16, i % 2 == 0, seed=29 + i)
        d = Dev(c)
        qd = dev(queries(c, n_q, 18 + i, True))
        nb = q4.q4_attn_paged_workspace_bytes(n_q, n_kv, hd)
        work.append([c, d, qd, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb, torch.cuda.Stream()])

    def go(c, d, qd, ws, nb, s):
        out = torch.zeros((c.n_tokens, n_q * hd), dtype=torch.float16, device="cuda")
        torch.cuda.current_stream().synchronize()
        q4.q4_attn_paged(d.kv, d.batch, qd, q4.Q4_TYPE_F32, n_q * hd, n_q, 0, 0, out, n_q * hd, ws, nb, stream=s)
        return out

    alone = []
    for w in work:
        alone.append(go(*w))
        torch.cuda.synchronize()
    for _ in range(5):
        outs = [go(*w) for w in work]
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 values: pages at its far end, for the write, the read and the attention."""
    n_kv, hd, page = 2, 256, 256
    n_pages = (1 << 31) // (n_kv * hd * page) + 64      # 2^31 values and more, 4.3 GB per pool
    kp = torch.zeros((n_pages, n_kv, page, hd), dtype=torch.float16, device="cuda")
    vp = torch.zeros((n_pages, n_kv, page, hd), dtype=torch.float16, device="cuda")
    for new, total in ((300, 700), (1, 700)):
        c = ref.Cache([new], [total], n_kv, hd, page, seed=33)
        small = c.n_pages
        for p in range(small):
            kp[n_pages - small + p] = dev(c.pages["k"][p])
            vp[n_pages - small + p] = dev(c.pages["v"][p])
        far = np.where(c.table >= 0, c.table + n_pages - small, -1).astype(np.int32)
        kv = q4.PagedKV.of(kp, vp, n_pages, page, n_kv, hd)
        b = q4.PagedBatch.of(dev(c.starts), dev(c.lens), dev(far), 1, c.n_tokens, c.width, new)
        x = torch.randn((c.n_tokens, n_kv * hd), device="cuda")
        q4.q4_paged_write(kv, b, x, x, q4.Q4_TYPE_F32, n_kv * hd)
        back = torch.zeros((2, c.n_tokens, n_kv * hd), device="cuda")
        q4.q4_paged_read(kv, b, back[0], back[1], q4.Q4_TYPE_F32, n_kv * hd)
        torch.cuda.synchronize()
        assert torch.equal(back[0], x.half().float()) and torch.equal(back[1], x.half().float())
        for p in range(small):
            c.pages["k"][p] = kp[n_pages - small + p].cpu().numpy()
            c.pages["v"][p] = vp[n_pages - small + p].cpu().numpy()
        q = queries(c, 4, 34, True)
        qd = dev(q)
        out = torch.full((c.n_tokens, 4 * hd), 7.0, dtype=torch.float16, device="cuda")
        nb = q4.q4_attn_paged_workspace_bytes(4, n_kv, hd)
        q4.q4_attn_paged(kv, b, qd, q4.Q4_TYPE_F32, 4 * hd, 4, 0, 0, out, 4 * hd, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
        torch.cuda.synchronize()
        check(out.cpu().numpy().astype(np.float64), c, q, 4)


def test_binding_refuses_wrong_tensors():
    c = ref.Cache([1], [5], 1, 64, 16, seed=35)
    d = Dev(c)
    x = torch.zeros((1, 64), device="cuda")
    for bad in (x.cpu(), x.half(), x[:, :32].clone()):
        with pytest.raises(q4.Q4Error) as e:
            q4.q4_paged_write(d.kv, d.batch, bad, x, q4.Q4_TYPE_F32, 64)
        assert e.value.status == q4.Q4_ERR_ARG
    with pytest.raises(q4.Q4Error):
        q4.PagedKV.of(d.pages["k"].transpose(0, 1).expand(1, -1, -1, -1)[..., ::2], d.pages["v"], 1, 16, 1, 64)
    with pytest.raises(q4.Q4Error):
        q4.PagedBatch.of(d.starts.long(), d.lens, d.table, 1, 1, 1, 1)
