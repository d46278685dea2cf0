"""Products, norms and rotations of a prompt's layer where tiles, rings, lengths and values meet their ends, on the GPU, against plain 64-bit forms."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import prompt_ref as ref
from exact_circle import circle
import weight_streaming_q4_gb300 as q4

pytestmark = pytest.mark.gpu

F16, F32 = q4.Q4_TYPE_F16, q4.Q4_TYPE_F32


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def settled():
    torch.cuda.synchronize()
    assert q4.q4_device_status() == 0, "a kernel's wait ran out"


def activated(t, off, gelu):
    """(the activation of t in 64 bits, how far it may be): as in prompt_ref, GELU by the 64-bit complementary error function."""
    a = 0.5 * t * torch.erfc(torch.from_numpy(-t / math.sqrt(2))).numpy() if gelu else t
    return a, ref.SLOPE * off + 2.0 ** -20 * np.abs(a) + 2.0 ** -22 * np.abs(t)


# Two and more tiles for each of 76 pairs of CTAs, and rows so short that the operand ring holds more than the steps of the tiles whose
# sums have a place: the warps that fill it are done while the products of the tile before the last one still wait for an epilogue.
SHORT = [(300, 28672, 512), (150, 49152, 512), (550, 16384, 288), (280, 28672, 256), (150, 25000, 256), (12, 128256, 256), (64, 128256, 256)]


@pytest.mark.parametrize("slow", [False, True], ids=["plain", "slow_epilogue"])
@pytest.mark.parametrize("rows,n,k", SHORT)
def test_short_rows_and_many_tiles(rows, n, k, slow):
    rng = np.random.default_rng(rows + n + k)
    blocks = ref.q4_bytes(n, k, n)
    w, x = ref.weights(blocks), rng.normal(size=(rows, k)).astype(np.float16)
    bias = rng.normal(size=n).astype(np.float32) if slow else None
    res = dev(rng.normal(size=(rows, n)).astype(np.float32)) if slow else None
    ep = q4.Epilogue.of(n, rows, q4.Q4_ACT_GELU, 0.5, dev(bias), res, F32) if slow else None
    wd, xd = dev(blocks), dev(x)
    ys = [torch.zeros((rows, n), dtype=torch.float16, device="cuda") for _ in range(5)]
    for y in ys:
        q4.q4_gemm(wd, xd, k, n, k, rows, ep, y, n)
    settled()
    t, off = ref.product(w, x.astype(np.float64), bias)
    if slow:
        a, off = activated(t, off, True)
        t = 0.5 * a + ref.host(res)
        off = 0.5 * off + 2.0 ** -23 * (np.abs(a) + np.abs(t) + np.abs(ref.host(res)))
    ref.assert_near(ref.host(ys[0]), t, ref.rounded(t, off), f"{rows} x {n} x {k}")
    for y in ys[1:]:
        assert torch.equal(y, ys[0])


@pytest.mark.parametrize("gelu", [False, True], ids=["none", "gelu"])
@pytest.mark.parametrize("rows,n,k", [(80, 49152, 256), (70, 50001, 224)])
def test_short_rows_and_many_tiles_of_two_matrices(rows, n, k, gelu):
    rng = np.random.default_rng(rows + n + k)
    blocks = [ref.q4_bytes(n, k, n + i) for i in range(2)]
    x = rng.normal(size=(rows, k)).astype(np.float16)
    bias = [rng.normal(size=n).astype(np.float32) for _ in range(2)]
    ep = q4.GatedEpilogue.of(n, q4.Q4_ACT_GELU if gelu else q4.Q4_ACT_NONE, *map(dev, bias))
    wd, xd = [dev(b) for b in blocks], dev(x)
    ys = [torch.zeros((rows, n), dtype=torch.float16, device="cuda") for _ in range(5)]
    for y in ys:
        q4.q4_gemm_gated(*wd, xd, k, n, k, rows, ep, y, n)
    settled()
    (g, dg), (u, du) = (ref.product(ref.weights(b), x.astype(np.float64), v) for b, v in zip(blocks, bias))
    a, da = activated(g, dg, gelu)
    want = a * u
    ref.assert_near(ref.host(ys[0]), want, ref.rounded(want, np.abs(a) * du + da * np.abs(u) + da * du + 2.0 ** -23 * np.abs(want)), f"{rows} x {n} x {k}")
    for y in ys[1:]:
        assert torch.equal(y, ys[0])


@pytest.mark.parametrize("k", [256, 512, 768, 1280, 1792, 2304, 2560])
@pytest.mark.parametrize("rows,n", [(9, 20000), (70, 20000), (130, 20000), (250, 20000), (250, 300)])
def test_rings_that_end_in_any_place(rows, n, k):
    """Steps of k that fill the rings once, in part or several times, over the same buffers again and again: what one launch leaves open the next would meet."""
    rng = np.random.default_rng(rows + n + k)
    blocks = [dev(ref.q4_bytes(n, k, n + i)) for i in range(2)]
    w = [torch.from_numpy(ref.weights(ref.q4_bytes(n, k, n + i))).cuda().float() for i in range(2)]
    x = dev(rng.normal(size=(rows, k)).astype(np.float16))
    first = None
    for _ in range(8):
        y = torch.zeros((2, rows, n), dtype=torch.float16, device="cuda")
        q4.q4_gemm(blocks[0], x, k, n, k, rows, None, y[0], n)
        q4.q4_gemm_gated(*blocks, x, k, n, k, rows, q4.GatedEpilogue.of(n, q4.Q4_ACT_NONE), y[1], n)
        first = y if first is None else first
        assert torch.equal(y, first)
    settled()
    t = [x.double() @ v.double().T for v in w]
    s = [k * 2.0 ** -23 * (x.double().abs() @ v.double().abs().T) for v in w]
    for got, want, off in ((first[0], t[0], s[0]), (first[1], t[0] * t[1], t[0].abs() * s[1] + s[0] * t[1].abs() + s[0] * s[1] + 2.0 ** -23 * (t[0] * t[1]).abs())):
        assert torch.all((got.double() - want).abs() <= off + 2.0 ** -11 * (want.abs() + off) + 2.0 ** -25)


@pytest.mark.parametrize("kind", [F16, F32])
@pytest.mark.parametrize("rows,n,k", [(20, 33, 256), (100, 20001, 320), (250, 20031, 256), (40, 289, 8192), (200, 1055, 4096), (256, 14337, 1024), (65, 31, 96)])
def test_warps_whose_last_rows_of_w_are_not_there(rows, n, k, kind):
    """A residual, and a matrix whose last warp has rows of W in some lanes only, in the first, middle, last and shared tiles of a pair."""
    rng = np.random.default_rng(rows + n + k)
    blocks = ref.q4_bytes(n, k, n)
    x = dev(rng.normal(size=(rows, k)).astype(np.float16))
    res = dev(rng.normal(size=(rows, n))).to(torch.float32 if kind == F32 else torch.float16)
    y = torch.full((rows + 1, n), 7.0, dtype=torch.float16, device="cuda")
    q4.q4_gemm(dev(blocks), x, k, n, k, rows, q4.Epilogue.of(n, rows, residual=res, residual_type=kind), y, n)
    settled()
    ref.assert_near(ref.host(y[:rows]), *ref.gemm(ref.weights(blocks), ref.host(x), residual=ref.host(res)))
    assert torch.all(y[rows:] == 7)


@pytest.mark.parametrize("halves", [True, False])
def test_far_positions_against_exact_angles(halves):
    """Cosines and sines of angles reduced in exact arithmetic: within 2^-22 whatever the position and the frequency."""
    freqs = [1.0, 0.794, 2.0, 3.7, 30.0, 100.0, -3.0, 0.25, 1e-4, 12345.678, -1e9, 2.0 ** 60]
    places = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 123456789, 100003, 1, 0, -77]
    two_pi, pairs = circle(), len(freqs)
    turns = np.array([[float(Fraction(f) * p / two_pi % 1) for f in freqs] for p in places])
    x = torch.zeros((len(places), 2 * pairs), device="cuda")
    first = np.arange(pairs) if halves else 2 * np.arange(pairs)
    second = first + (pairs if halves else 1)
    x[:, dev(first)] = 1                          # (1, 0) turns into (cos, sin)
    y = torch.zeros_like(x)
    rot = q4.Rope.of(2 * pairs, freqs, None, q4.Q4_ROPE_HALVES if halves else q4.Q4_ROPE_ADJACENT)
    at = q4.RopePlaces.of(dev(np.array(places, dtype=np.int32)), 1, len(places))
    q4.q4_rope(rot, at, 1, x, F32, 2 * pairs, y, F32, 2 * pairs)
    settled()
    got = ref.host(y)
    ref.assert_near(got[:, first], np.cos(2 * math.pi * turns), 2.0 ** -22, "cosines")
    ref.assert_near(got[:, second], np.sin(2 * math.pi * turns), 2.0 ** -22, "sines")


@pytest.mark.parametrize("rows,k", [(1, 2 ** 30 + 4096), (9, 2 ** 30 + 4096), (2, 2 ** 30 + 4096 + 32), (1, 2 ** 31 - 32)])
def test_rows_of_a_billion_values(rows, k):
    """One row of W whose bytes, and whose x's, are no longer counted in 31 bits; x is zero but for some runs of it."""
    gen = torch.Generator(device="cuda").manual_seed(k % 1000 + rows)
    w = torch.randint(0, 256, (k // 32, 18), generator=gen, dtype=torch.uint8, device="cuda")
    w[:, 1] = (w[:, 1] & 0x83) | 0x24              # scales of both signs, 2^-6 to 2^-5
    x = torch.zeros((rows, k), dtype=torch.float16, device="cuda")
    runs = [0, 4096, 2 ** 29 - 64, 2 ** 30 - 64, 2 ** 30 + 2048, k - 2048, k - 96]
    runs = [(a, min(a + 2048, k)) for a in runs]
    for a, b in runs:
        x[:, a:b] = torch.randn((rows, b - a), generator=gen, device="cuda").half()
    there = torch.cat([torch.arange(a // 32, b // 32) for a, b in runs]).unique()
    ws = ref.weights(w[there.cuda()].cpu().numpy()[None])                 # [1][values there]
    xs = ref.host(x.view(rows, -1, 32)[:, there.cuda()].reshape(rows, -1))
    y, z = (torch.zeros((rows, 1), dtype=torch.float16, device="cuda") for _ in range(2))
    q4.q4_gemm(w, x, k, 1, k, rows, None, y, 1)
    q4.q4_gemm_gated(w, w, x, k, 1, k, rows, q4.GatedEpilogue.of(1, q4.Q4_ACT_NONE), z, 1)
    settled()
    # (sums of zeros are exact: prompt_ref's bound with the number of values that are there for k)
    t, off = ref.product(ws, xs)
    ref.assert_near(ref.host(y), t, ref.rounded(t, off), "product")
    ref.assert_near(ref.host(z), t * t, ref.rounded(t * t, 2 * np.abs(t) * off + off * off + 2.0 ** -23 * t * t), "gated product")


# The size of a relative error of an activation, in 2^-23, beside its rounding to binary16, for an argument t that is exact.
#   gelu       t / sqrt 2 is off by 2^-23 of itself, which (t^2 + 2) times over is erfc's error; erfcf itself 4, three products 3
#   silu       __expf 2 + 1.173 |t|, half as much again for the sum and the quotient's own 2, a product
#   gelu_tanh  the exponent z is off by 2^-21 of itself (five roundings), which is e^z's error |z| times over; the rest as for silu
TAILS = dict(gelu=lambda t: t * t + 9, silu=lambda t: 1.173 * np.abs(t) + 9,
             gelu_tanh=lambda t: (4 + 1.173) * np.abs(math.sqrt(8 / math.pi) * (t + 0.044715 * t ** 3)) + 9)


@pytest.mark.parametrize("name", list(TAILS))
@pytest.mark.parametrize("rows", [8, 40])
def test_the_tails_of_activations_keep_their_digits(rows, name):
    """Small values of an activation, multiplied by a large second product or scale: what is left of them is right relative to itself."""
    n, k = 37, 32
    d = np.linspace(0.25, 1.0, n).astype(np.float16)
    blocks = [np.full((n, 1, 18), 0x88, dtype=np.uint8) for _ in range(2)]
    for b, scale, at in ((blocks[0], d, 0), (blocks[1], np.full(n, 1000, dtype=np.float16), 1)):
        b[:, 0, :2] = scale[:, None].view(np.uint8)
        b[:, 0, 2 + at] = 0x89                    # one weight of 1, the others 0
    x = np.zeros((rows, k), dtype=np.float16)
    x[:, 0], x[:, 1] = np.linspace(-12, 9, rows), np.linspace(1000, 60000, rows)
    g = x[:, :1].astype(np.float64) * d.astype(np.float64)
    u = x[:, 1:2].astype(np.float64) * 1000
    a = {"gelu": lambda t: 0.5 * t * torch.erfc(torch.from_numpy(-t / math.sqrt(2))).numpy(), "silu": lambda t: t / (1 + np.exp(-t)),
         "gelu_tanh": lambda t: t / (1 + np.exp(-math.sqrt(8 / math.pi) * (t + 0.044715 * t ** 3)))}[name](g)
    y = torch.zeros((2, rows, n), dtype=torch.float16, device="cuda")
    act = dict(gelu=q4.Q4_ACT_GELU, silu=q4.Q4_ACT_SILU, gelu_tanh=q4.Q4_ACT_GELU_TANH)[name]
    q4.q4_gemm_gated(*map(dev, blocks), dev(x), k, n, k, rows, q4.GatedEpilogue.of(n, act), y[0], n)
    q4.q4_gemm(dev(blocks[0]), dev(x), k, n, k, rows, q4.Epilogue.of(n, rows, act, 2.0 ** 20), y[1], n)
    settled()
    for got, want in ((y[0], a * u), (y[1], a * 2.0 ** 20)):
        there = np.abs(want) < 65000              # (beyond that binary16 has only infinity)
        off = np.abs(want) * (2.0 ** -11 + 2.0 ** -23 * TAILS[name](g)) + 2.0 ** -25
        ref.assert_near(ref.host(got)[there], want[there], off[there], name)


@pytest.mark.parametrize("rows", [2, 8, 9, 40, 300])
def test_a_row_depends_on_its_own_inputs_and_the_number_of_rows(rows):
    """Other values in the other rows leave a row's bits as they were; other numbers of rows its values within the bound (the sums' order may be another)."""
    n, k, rng = 700, 4096, np.random.default_rng(rows)
    blocks = ref.q4_bytes(n, k, 3)
    w, x = dev(blocks), dev(rng.normal(size=(2, rows, k)).astype(np.float16))
    x[1, rows // 2] = x[0, rows // 2]
    y, z = (torch.zeros((2, rows, n), dtype=torch.float16, device="cuda") for _ in range(2))
    wide = dev(rng.normal(size=(2, 200 * (rows > 8) + rows, 5001)).astype(np.float16))        # more and fewer rows than SMs
    wide[1, rows // 2] = wide[0, rows // 2]
    v = torch.zeros_like(wide)
    for i in range(2):
        q4.q4_gemm(w, x[i], k, n, k, rows, None, y[i], n)
        q4.q4_gemm_gated(w, w, x[i], k, n, k, rows, None, z[i], n)
        q4.q4_block_norm(q4.BlockNorm.of(5001), wide.size(1), wide[i], F16, 5001, None, F16, 5001, None, F16, 5001, v[i], F16, 5001)
    one = torch.zeros((3, n), dtype=torch.float16, device="cuda")
    q4.q4_gemm(w, x[0, rows // 2:], k, n, k, 1, None, one, n)
    settled()
    for got in (y, z, v):
        assert torch.equal(got[0, rows // 2], got[1, rows // 2])
    want, off = ref.gemm(ref.weights(blocks), ref.host(x[0, rows // 2:rows // 2 + 1]))
    for got in (one[0], y[0, rows // 2]):
        ref.assert_near(ref.host(got)[None], want, off)
    assert torch.all(one[1:] == 0)


@pytest.mark.parametrize("n", [64, 300, 4096, 5001, 8200, 20001])
@pytest.mark.parametrize("kind", [q4.Q4_NORM_RMS, q4.Q4_NORM_LAYER])
@pytest.mark.parametrize("typ", [F16, F32])
def test_norms_of_infinities_and_nan_in_every_place(n, kind, typ):
    """Every value of a row with something that is not finite: NaN, or of a root mean square with an infinity 0 times the weight and the bias."""
    rows, rng = 6, np.random.default_rng(n)
    x = dev(rng.normal(size=(rows, n))).to(torch.float16 if typ == F16 else torch.float32)
    x[1, 5], x[2, n - 1], x[4, 9], x[4, 30] = math.nan, math.inf, -math.inf, math.inf
    clean = ref.host(x)[[0, 3, 5]]
    weight, bias, post = rng.normal(size=n).astype(np.float32), rng.integers(-4, 5, size=n).astype(np.float32), rng.integers(-4, 5, size=n).astype(np.float32)
    res = dev(rng.integers(-8, 9, size=(rows, n)).astype(np.float32))
    t, z = (torch.zeros((rows, n), device="cuda") for _ in range(2))
    # one norm, then one around the block that has a clean residual and a scale of 2
    q4.q4_block_norm(q4.BlockNorm.of(n, kind, weight=dev(weight), bias=dev(bias)), rows, x, typ, n, None, F32, n, None, F32, n, z, F32, n)
    q4.q4_block_norm(q4.BlockNorm.of(n, kind, post_bias=dev(post), scale=2.0), rows, x, typ, n, res, F32, n, t, F32, n, None, F32, n)
    settled()
    gone = {1: list(range(n)), 2: [n - 1], 4: [9, 30]} if kind == q4.Q4_NORM_RMS else {r: list(range(n)) for r in (1, 2, 4)}
    for r, places in gone.items():
        for got, rest in ((z[r], bias), (t[r], ref.host(res[r]) + 2 * post)):
            want = rest.astype(np.float64)
            want[places] = math.nan
            np.testing.assert_array_equal(ref.host(got), want)
    name, eps = "rms" if kind == q4.Q4_NORM_RMS else "layer", float(np.float32(1e-5))
    v, off = ref.block_norm(clean, None, name, eps, weight=weight, bias=bias)[1]
    ref.assert_near(ref.host(z)[[0, 3, 5]], v, off + 2.0 ** -23 * np.abs(v))
    v, off = ref.block_norm(clean, ref.host(res)[[0, 3, 5]], name, eps, post=True, post_bias=post, scale=2.0)[0]
    ref.assert_near(ref.host(t)[[0, 3, 5]], v, off + 2.0 ** -23 * np.abs(v))
