"""q4_attn_paged where values are not finite or numbers are far from one, against paged_ref.py in 64 bits."""
import numpy as np
import pytest

import paged_ref as ref
import weight_streaming_q4_gb300 as q4
from test_paged_gpu import Dev, check, queries
from weight_streaming_q4_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    yield
    assert q4.q4_device_status() == 0, "a kernel wait failed"


def put(c, s, t, kind, name="v", block=1):
    """Block `block` of every head of sequence s's position t: NaN throughout, or infinities of both signs."""
    p, slot, at = c.table[s, t // c.page], t % c.page, slice(32 * block, 32 * block + 32)
    sign = np.where(np.arange(32) % 2, 1, -1)
    if not c.q8:
        c.pages[name][p, :, slot, at] = np.nan if kind == "nan" else sign * np.inf
    else:
        c.scales[name][p, :, slot, block] = np.nan if kind == "nan" else 6e4
        c.pages[name][p, :, slot, at] = 0 if kind == "nan" else 100 * sign      # f16(100 * 6e4) is infinite


def both_kernels(c, q, n_q, window=0, sinks=0):
    """The kernel of few rows and that of many: which one runs must not show.  (An infinite bound takes any number, so
    what is not finite has to be the same besides.)"""
    want, _ = c.attend(q, n_q, window, sinks)
    odd = ~np.isfinite(want)
    odd[:c.starts[0]] = odd[c.starts[-1]:] = False      # rows of no sequence
    for max_new in (1, 300):
        got = Dev(c, max_new=max_new).attend(q, n_q, window, sinks)
        check(got, c, q, n_q, window, sinks)
        assert np.array_equal(got[:, :n_q * c.hd][odd], want[odd], equal_nan=True)


@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("chunk", [1, 5, 150])
def test_a_hole_beside_a_value_that_all_rows_see(chunk, hd, q8, kind):
    """A page missing from a key tile that every row sees whole, and a value in it that is not finite."""
    c = ref.Cache([chunk, 1], [chunk + 300, 40], 1, hd, 16, q8, seed=hd + chunk, n_tokens=chunk + 1)
    c.table[0, 3] = -1
    put(c, 0, 2, kind)
    put(c, 0, 70, kind, block=0)
    q = queries(c, 3, 50, False, scale=0.5)
    want, _ = c.attend(q, 3)
    assert not np.isfinite(want[:chunk, :64]).any() and np.isfinite(want[chunk:]).all()
    both_kernels(c, q, 3)


@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("chunk", [1, 5, 150])
def test_values_that_some_rows_see(chunk, hd, q8, kind):
    """Of blocks that are not finite, every row gets what those it sees make of it: at the causal edge, at a window's, among the
    sinks, and in no row's sight (stale slots, positions between the sinks and the window)."""
    total = chunk + 300
    c = ref.Cache([chunk, 1], [total, 50], 1, hd, 16, q8, seed=hd + chunk + 1, n_tokens=chunk + 1)
    for t in range(total, -(-total // 16) * 16):       # slots behind the last position
        put(c, 0, t, kind)
        put(c, 0, t, kind, name="k", block=0)
    put(c, 0, total - 1, kind)                         # the last token alone
    put(c, 0, total - 1 - chunk // 2, kind, block=0)   # half of the tokens
    q = queries(c, 3, 51, True, scale=0.5)
    both_kernels(c, q, 3)
    if chunk > 1:
        put(c, 0, total - 1, "nan", name="k")          # a score: the last token's row
        got = Dev(c).attend(q, 3)
        assert np.isnan(got[chunk - 1]).all() and np.isfinite(got[:chunk - 1 - chunk // 2]).all()
    c = ref.Cache([chunk], [total], 1, hd, 16, q8, seed=hd + chunk + 2)
    put(c, 0, 1, kind)                                 # a sink
    put(c, 0, 40, kind)                                # between sinks and window
    put(c, 0, total - 64 - chunk // 2 - 1, kind, block=0)    # only the first tokens' windows reach it
    both_kernels(c, queries(c, 3, 52, False, scale=0.5), 3, 64, 3)
    put(c, 0, 1, "nan", block=0)
    both_kernels(c, queries(c, 3, 53, False, scale=0.5), 3, 64, 1)


@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
def test_many_items_that_some_rows_see_infinities_in(q8):
    """Long runs of items of few rows between items of two query tiles, each with values that are not finite for its last token."""
    new = [40 if s % 11 == 0 else 1 + s % 2 for s in range(1500)]
    c = ref.Cache(new, [n + s % 60 for s, n in enumerate(new)], 2, 64, 16, q8, seed=60)
    for s, n in enumerate(c.total):
        if s % 3:
            put(c, s, n - 1, "nan" if s % 2 else "inf", block=s % 2)
    q = queries(c, 16, 54, False, scale=0.5)
    both_kernels(c, q, 16)


@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("rows", [4, 12, 20, 28, 160])
def test_small_fp32_queries_against_large_keys(rows, hd, q8):
    """Queries whose last bits lie far below binary16's smallest number, against keys near its largest: 22 bits of a query count
    whatever its size.  Heads of one item are of sizes from 1 down to fp32's subnormal numbers, and zero."""
    c = ref.Cache([rows // 2, 1], [rows // 2 + 200, 90], 1, hd, 16, seed=hd + rows, n_tokens=rows // 2 + 1)
    half = np.where(np.arange(hd) < hd // 2, 1, -1)
    k = 6e4 * half * c.rng.choice([-1, 1], size=(c.n_pages, 1, 16, 1)) * np.exp2(-c.rng.integers(0, 3, size=(c.n_pages, 1, 16, 1)))
    if q8:
        c.q8 = True
        v = c.pages["v"].astype(np.float32)
        (c.pages["k"], c.scales["k"]), (c.pages["v"], c.scales["v"]) = ref.quantise(k.astype(np.float32)), ref.quantise(v)
    else:
        c.pages["k"] = k.astype(np.float16)
    # 2^-12 and 0.49 or 0.51 steps of binary16's smallest number: errors of one sign along a key, were the rest rounded to such steps
    one = 2.0 ** -12 + np.where(half > 0, 0.49, 0.51) * 2.0 ** -24
    size = np.exp2(-(np.arange(c.n_tokens * 2) % 7) * (np.arange(c.n_tokens * 2) % 3)).reshape(c.n_tokens, 2, 1)
    size[1::5, 1], size[2::5, 0], size[3::5, 1], size[4::5, 0] = 2.0 ** 12, 0.0, 2.0 ** -130, 2.0 ** 20
    q = (one * size).astype(np.float32).reshape(c.n_tokens, 2 * hd)
    check(Dev(c).attend(q, 2), c, q, 2)
    both_kernels(c, q, 2)


@pytest.mark.parametrize("chunk", [1, 40])
def test_values_that_are_not_finite_under_scores_of_minus_infinity(chunk):
    """0 times an infinity is no number, however the positions are shared out: most of a long sequence's scores are -infinity, so whole
    parts of it have no other, and some values there are infinite or NaN."""
    c = ref.Cache([chunk], [40000], 1, 128, 256, seed=61)
    far = c.table[0, :117]                             # positions 0 .. 29951
    c.pages["k"][far, :, :, 0] = -np.inf
    for i, kind in enumerate(("nan", "inf")):
        put(c, 0, 100 + 9000 * i, kind, block=i)
    q = queries(c, 8, 55, False, scale=0.5)
    q.reshape(chunk, 8, 128)[:, :, 0] = 0.25
    with np.errstate(invalid="ignore"):
        want, _ = c.attend(q, 8)
    odd = np.isnan(want)
    assert odd.reshape(chunk, 8, 128)[:, :, :64].all() and np.isfinite(want[~odd]).all()
    for max_new in (1, 300):
        got = Dev(c, max_new=max_new).attend(q, 8)
        check(got, c, q, 8)
        assert np.array_equal(~np.isfinite(got), odd)


@pytest.mark.parametrize("q8", [False, True], ids=["f16", "q8"])
def test_stale_slots_cost_nothing(q8):
    """What lies behind the sequences' last positions, NaN here, is not searched for: a call takes as long as with numbers there (it
    took 2 to 3 times as long; the bound is half way)."""
    import torch
    c = ref.Cache([1] * 64, [2000 + 61 * s + s % 2 for s in range(64)], 4, 128, 64, q8, seed=62)
    q = queries(c, 32, 56, True)
    times = []
    for stale in (False, True):
        if stale:
            for s, n in enumerate(c.total):
                for t in range(n, -(-n // 64) * 64):
                    for block in range(4):
                        put(c, s, t, "nan", block=block)
        d = Dev(c)
        qd, out = torch.from_numpy(q).cuda(), torch.empty((64, 32 * 128), dtype=torch.float16, device="cuda")
        nb = q4.q4_attn_paged_workspace_bytes(32, 4, 128)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        best = 1e9
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                q4.q4_attn_paged(d.kv, d.batch, qd, q4.Q4_TYPE_F32, 32 * 128, 32, 0, 0, out, 32 * 128, ws, nb)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
        check(out.cpu().numpy().astype(np.float64), c, q, 32)
    assert times[1] < 1.5 * times[0], times
