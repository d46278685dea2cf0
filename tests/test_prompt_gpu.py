"""The operators of a prompt's layer beside its attention, on the GPU, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import prompt_ref as ref
import weight_streaming_q4_gb300 as q4

pytestmark = pytest.mark.gpu

F16, F32 = q4.Q4_TYPE_F16, q4.Q4_TYPE_F32
TORCH = {F16: torch.float16, F32: torch.float32}
ACT = dict(none=q4.Q4_ACT_NONE, relu=q4.Q4_ACT_RELU, silu=q4.Q4_ACT_SILU, gelu=q4.Q4_ACT_GELU, gelu_tanh=q4.Q4_ACT_GELU_TANH)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def rows_of(rng, rows, n, kind=F16, ld=None, fill=math.nan, scale=1.0):
    """(buffer with a strip of `fill` beside every row, its values in 64 bits)"""
    buf = torch.full((rows, ld or n), fill, dtype=TORCH[kind], device="cuda")
    buf[:, :n] = dev(rng.normal(size=(rows, n)) * scale).to(TORCH[kind])
    return buf, ref.host(buf[:, :n])


def settled():
    torch.cuda.synchronize()
    assert q4.q4_device_status() == 0, "a kernel's wait ran out"


# ------------------------------------------------------------------ products

ODD = [(1, 1, 32), (1, 64, 256), (2, 5, 64), (3, 130, 96), (7, 128, 512), (16, 127, 288), (17, 129, 768), (31, 255, 1024), (33, 256, 2048),
       (64, 257, 256), (65, 300, 1056), (100, 512, 4096), (128, 33, 14336), (129, 1000, 544), (200, 384, 1280), (255, 640, 256), (256, 513, 800),
       (257, 260, 2304), (300, 1030, 512), (520, 700, 320), (1000, 257, 128), (1500, 5200, 96), (2100, 4100, 512), (37, 4099, 4128), (1, 4096, 4096), (4, 6144, 4096),
       # few tiles and a long k, shared by up to 8 pairs
       (40, 300, 8192), (33, 1024, 8192), (200, 1000, 4096), (17, 256, 11008), (60, 520, 8224), (96, 1500, 4352), (12, 100, 28672),
       (5, 300, 11008), (8, 1030, 8224), (1, 1024, 4096), (3, 2000, 6176), (7, 40, 28672), (2, 5000, 4128), (1, 100, 3200), (6, 2500, 2304),
       # more tiles than run at once, by the rows of x that a tile takes
       (30, 20000, 288), (64, 20000, 256), (100, 20000, 256), (150, 500, 320), (190, 700, 512), (384, 10300, 256), (8, 12000, 256), (9, 5000, 96)]


@pytest.mark.parametrize("rows,n,k", ODD)
def test_gemm(rows, n, k):
    rng = np.random.default_rng(rows * 1000 + n + k)
    blocks = ref.q4_bytes(n, k, n + k)
    w, x_ld, y_ld = ref.weights(blocks), k + 8 * (rows % 3), n + rows % 4
    xb, x = rows_of(rng, rows, k, F16, x_ld)
    name = ref.ACTS[(rows + n) % 5]
    bias = rng.normal(size=n).astype(np.float32) if n % 2 else None
    kind = F32 if rows % 2 else F16
    scale = [1.0, 0.25, -1.5][k // 32 % 3]
    rb, r = rows_of(rng, rows, n, kind, n + 3) if rows % 5 else (None, None)
    ep = q4.Epilogue.of(n, rows, ACT[name], scale, None if bias is None else dev(bias), rb, kind, n + 3)
    y = torch.full((rows + 2, y_ld), 7.0, dtype=torch.float16, device="cuda")
    q4.q4_gemm(dev(blocks), xb, x_ld, n, k, rows, ep, y, y_ld)
    settled()
    want, off = ref.gemm(w, x, bias, name, scale, r)
    ref.assert_near(ref.host(y[:rows, :n]), want, off, f"{rows} x {n} x {k} {name}")
    assert torch.all(y[rows:] == 7) and torch.all(y[:, n:] == 7), "memory behind the rows or values was written"


@pytest.mark.parametrize("rows,n,k", ODD)
def test_gated(rows, n, k):
    rng = np.random.default_rng(rows * 999 + n + k)
    blocks = [ref.q4_bytes(n, k, n + k + i) for i in range(2)]
    x_ld, y_ld = k + 8 * (n % 3), n + k // 32 % 4
    xb, x = rows_of(rng, rows, k, F16, x_ld)
    name = ref.ACTS[(rows + n + 1) % 5]
    biases = [rng.normal(size=n).astype(np.float32) if (n >> i) % 2 else None for i in range(2)]
    ep = q4.GatedEpilogue.of(n, ACT[name], *[None if b is None else dev(b) for b in biases])
    y = torch.full((rows + 2, y_ld), 7.0, dtype=torch.float16, device="cuda")
    q4.q4_gemm_gated(*map(dev, blocks), xb, x_ld, n, k, rows, ep, y, y_ld)
    settled()
    want, off = ref.gated(*map(ref.weights, blocks), x, *biases, name)
    ref.assert_near(ref.host(y[:rows, :n]), want, off, f"{rows} x {n} x {k} {name}")
    assert torch.all(y[rows:] == 7) and torch.all(y[:, n:] == 7), "memory behind the rows or values was written"


@pytest.mark.parametrize("rows,n,k", [(5, 70, 256), (40, 300, 288), (300, 200, 512)])
def test_defaults_and_flat_buffers(rows, n, k):
    rng = np.random.default_rng(4)
    blocks, (xb, x) = ref.q4_bytes(n, k, 1), rows_of(rng, rows, k)
    y = torch.zeros(rows * n, dtype=torch.float16, device="cuda")
    q4.q4_gemm(dev(blocks).view(-1), xb.view(-1), k, n, k, rows, None, y, n)
    settled()
    w = ref.weights(blocks)
    ref.assert_near(ref.host(y.view(rows, n)), *ref.gemm(w, x))
    q4.q4_gemm_gated(dev(blocks), dev(blocks), xb, k, n, k, rows, None, y, n)
    settled()
    ref.assert_near(ref.host(y.view(rows, n)), *ref.gated(w, w, x))
    y.fill_(3)
    q4.q4_gemm(dev(blocks), xb, k, n, k, 0, None, y, n)
    settled()
    assert torch.all(y == 3)


@pytest.mark.parametrize("rows", [1, 8, 9, 150])
@pytest.mark.parametrize("k", [32, 96, 160, 224, 256, 288, 480])
@pytest.mark.parametrize("n", [16, 31, 64, 65, 129, 257])
def test_matrices_that_end_inside_a_copy(rows, n, k):
    """Narrow matrices at the end of a buffer: a copy of 256 or 1024 columns spans rows, and the last ones would leave the matrix."""
    rng = np.random.default_rng(n + k)
    blocks, (xb, x) = [ref.q4_bytes(n, k, k + i) for i in range(2)], rows_of(rng, rows, k)
    behind = []
    for b in blocks:
        buf = torch.full((1 << 16 | b.size,), 255, dtype=torch.uint8, device="cuda")
        behind.append(buf[buf.numel() - b.size & ~15:][:b.size])
        behind[-1].copy_(dev(b).view(-1))
    w = [ref.weights(b) for b in blocks]
    y = torch.zeros((rows, n), dtype=torch.float16, device="cuda")
    q4.q4_gemm(behind[0], xb, k, n, k, rows, None, y, n)
    settled()
    ref.assert_near(ref.host(y), *ref.gemm(w[0], x))
    q4.q4_gemm_gated(*behind, xb, k, n, k, rows, None, y, n)
    settled()
    ref.assert_near(ref.host(y), *ref.gated(*w, x))


def test_a_chained_product_waits_for_the_product_before_it():
    """A chained matrix-vector product whose x a many-row product has just written."""
    n, k, rng = 4096, 4096, np.random.default_rng(5)
    blocks = [dev(ref.q4_bytes(n, k, i)) for i in range(2)]
    x = rows_of(rng, 64, k)[0]
    for _ in range(4):
        y, z = torch.zeros((64, n), dtype=torch.float16, device="cuda"), torch.zeros((2, n), device="cuda")
        q4.q4_gemv(blocks[1], x[0], z[1], n, k, 1)
        q4.q4_gemm(blocks[0], x, k, n, k, 64, None, y, n)
        q4.q4_gemv(blocks[1], y[63], z[0], n, k, 1, chain=True)
        torch.cuda.synchronize()
        q4.q4_gemv(blocks[1], y[63], z[1], n, k, 1)
        settled()
        assert torch.equal(z[0], z[1])


@pytest.mark.parametrize("rows", [1, 20, 300])
@pytest.mark.parametrize("k", [256, 288, 4096])
def test_residual_may_be_the_output(rows, k):
    n, rng = 190, np.random.default_rng(rows + k)
    blocks, (xb, x) = ref.q4_bytes(n, k, 2), rows_of(rng, rows, k)
    y, r = rows_of(rng, rows, n, F16, n + 1, 5.0)
    q4.q4_gemm(dev(blocks), xb, k, n, k, rows, q4.Epilogue.of(n, rows, residual=y, residual_ld=n + 1), y, n + 1)
    settled()
    ref.assert_near(ref.host(y[:, :n]), *ref.gemm(ref.weights(blocks), x, residual=r))


@pytest.mark.parametrize("rows", [3, 18, 140])
@pytest.mark.parametrize("k", [512, 352])
def test_what_is_not_finite_stays_in_its_row_and_column(rows, k):
    """A row of x, and a scale of W, that are not finite spoil that row, and that column, of y alone."""
    n, rng = 150, np.random.default_rng(rows + k)
    blocks = ref.q4_bytes(n, k, 3)
    d = blocks[..., :2].copy().view(np.float16)
    d[7, 1], d[n - 1, k // 32 - 1] = np.nan, np.inf
    blocks[..., :2] = d.view(np.uint8)
    xb, x = rows_of(rng, rows, k, F16, k + 8)
    xb[1, k - 1], xb[rows - 1, 3] = math.nan, math.inf
    y = torch.zeros((rows, n), dtype=torch.float16, device="cuda")
    for two in (False, True):
        y.fill_(9)
        if two:
            q4.q4_gemm_gated(dev(blocks), dev(blocks), xb, k + 8, n, k, rows, None, y, n)
        else:
            q4.q4_gemm(dev(blocks), xb, k + 8, n, k, rows, None, y, n)
        settled()
        got, w = ref.host(y), ref.weights(blocks)
        good_r, good_n = [r for r in range(rows) if r not in (1, rows - 1)], [i for i in range(n) if i not in (7, n - 1)]
        assert not np.isfinite(got[[1, rows - 1]]).any() and not np.isfinite(got[:, [7, n - 1]]).any()
        want, off = ref.gated(w[good_n], w[good_n], x[good_r]) if two else ref.gemm(w[good_n], x[good_r])
        ref.assert_near(got[np.ix_(good_r, good_n)], want, off)


@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("k", [256, 64])
def test_scales_at_the_ends_of_binary16(rows, k):
    """Zero, subnormal, negative and the largest scales: a weight is the binary16 value, zero times anything finite is zero."""
    n, rng = 12, np.random.default_rng(k)
    s = np.array([0.0, 6e-8, -6e-8, 3e-6, 6.2e-5, -6.2e-5, 1e-3, 0.3, -1.7, 300.0, 8188.0, -8188.0], dtype=np.float16)
    blocks = ref.q4_bytes(n, k, 5, s[:, None])
    x = np.zeros((rows, k))
    x[:, ::7] = rng.normal(size=x[:, ::7].shape) * 2.0 ** -6
    x = x.astype(np.float16).astype(np.float64)
    y = torch.zeros((rows, n), dtype=torch.float16, device="cuda")
    q4.q4_gemm(dev(blocks), dev(x, torch.float16), k, n, k, rows, None, y, n)
    settled()
    w = ref.weights(blocks)
    assert np.isfinite(w).all()
    ref.assert_near(ref.host(y), *ref.gemm(w, x))
    blocks[..., 2:] = 0x88       # codes of 8: exactly zero, whatever the scale
    q4.q4_gemm(dev(blocks), dev(x, torch.float16), k, n, k, rows, None, y, n)
    settled()
    assert torch.all(y == 0)


@pytest.mark.parametrize("rows,n,k", [(1, 4096, 4096), (24, 512, 2048), (300, 1030, 544), (513, 600, 1024)])
def test_products_repeat_their_bits_on_other_streams_and_in_graphs(rows, n, k):
    rng = np.random.default_rng(9)
    blocks = [dev(ref.q4_bytes(n, k, i)) for i in range(2)]
    xb, _ = rows_of(rng, rows, k)
    other = rows_of(rng, rows, k)[0]
    ep = q4.Epilogue.of(n, rows, q4.Q4_ACT_GELU, 0.5, dev(rng.normal(size=n).astype(np.float32)))

    def outs(x):
        y = torch.zeros((2, rows, n), dtype=torch.float16, device="cuda")
        q4.q4_gemm(blocks[0], x, k, n, k, rows, ep, y[0], n)
        q4.q4_gemm_gated(*blocks, x, k, n, k, rows, None, y[1], n)
        return y

    first, second = outs(xb), outs(other)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, s in enumerate(streams * 2):      # two at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append((i % 2, outs(other if i % 2 else xb)))
    torch.cuda.synchronize()
    for which, y in got:
        assert torch.equal(y, second if which else first)
    x = xb.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = outs(x)
    for which, src in ((1, other), (0, xb)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, second if which else first)
    settled()


def test_rows_beyond_31_bits():
    """Rows so far apart that their offsets pass 2^31 values."""
    rows, n, k, ld = 36, 96, 256, (1 << 26) + 8
    rng = np.random.default_rng(2)
    blocks = ref.q4_bytes(n, k, 6)
    xb = torch.empty(rows * ld, dtype=torch.float16, device="cuda").view(rows, ld)
    y = torch.empty(rows * ld, dtype=torch.float16, device="cuda").view(rows, ld)
    xb[:, :k] = dev(rng.normal(size=(rows, k))).half()
    x = ref.host(xb[:, :k])
    q4.q4_gemm(dev(blocks), xb, ld, n, k, rows, None, y, ld)
    settled()
    ref.assert_near(ref.host(y[:, :n]), *ref.gemm(ref.weights(blocks), x))
    norms = q4.BlockNorm.of(n)
    q4.q4_block_norm(norms, rows, xb, F16, ld, None, F16, n, None, F16, n, y, F16, ld)
    settled()
    z, off = ref.block_norm(x[:, :n], None)[1]
    ref.assert_near(ref.host(y[:, :n]), z, ref.rounded(z, off))
    freqs = [1.0, 0.1, 0.01, 0.001]
    places = np.arange(rows)[None] * 1000
    q4.q4_rope(q4.Rope.of(8, freqs), q4.RopePlaces.of(dev(places.astype(np.int32)), 1, rows), n // 8, xb, F16, ld, y, F16, ld)
    settled()
    want, off = ref.rope(x[:, :n], places, freqs, [0] * 4, 8, True)
    ref.assert_near(ref.host(y[:, :n]), want, ref.rounded(want, off))


# ------------------------------------------------------------------ norms

WIDTHS = [1, 7, 8, 33, 64, 255, 500, 512, 1000, 1024, 2048, 4096, 5120, 8184, 8192, 8200, 10007, 16384, 16392, 28672, 32768]


def check_norm(rows, n, kind, i, pads):
    """One call against the formula; i picks types, gates and vectors, pads are what lies beside the rows of block, residual, t and z."""
    rng = np.random.default_rng(n)
    post, gate_rows = i % 2 == 0, [0, 2, 1, rows, None][i % 5]
    b_ld, r_ld, t_ld, z_ld = (n + pad for pad in pads)
    bt, rt, tt, zt = (F32 if i >> j & 1 else F16 for j in range(4))
    vec = lambda: rng.normal(size=n).astype(np.float32)     # noqa: E731
    block, b = rows_of(rng, rows, n, bt, b_ld, scale=3.0)
    res, r = rows_of(rng, rows, n, rt, r_ld) if i % 4 else (None, None)
    weight, bias, pw, pb = vec(), vec() if i % 3 else None, vec() if post and i % 4 else None, vec() if post and i % 3 else None
    gates = None if gate_rows is None else rng.normal(size=(-(-rows // gate_rows) if gate_rows else 1, n)).astype(np.float32)
    gate = None if gates is None else gates[np.arange(rows) // gate_rows] if gate_rows else gates
    d = lambda v: None if v is None else dev(v)     # noqa: E731
    norms = q4.BlockNorm.of(n, q4.Q4_NORM_LAYER if kind == "layer" else q4.Q4_NORM_RMS, 1e-5, d(weight), d(bias), d(pw), d(pb), 0.5, d(gates), n, gate_rows or 0, post)
    t = torch.full((rows + 1, t_ld), 7.0, dtype=TORCH[tt], device="cuda")
    z = torch.full((rows + 1, z_ld), 7.0, dtype=TORCH[zt], device="cuda")
    q4.q4_block_norm(norms, rows, block, bt, b_ld, res, rt, r_ld, t, tt, t_ld, z, zt, z_ld)
    settled()
    want = ref.block_norm(b, r, kind, float(np.float32(1e-5)), post, pw, pb, 0.5, gate, weight, bias)
    for got, typ, (v, off) in ((t, tt, want[0]), (z, zt, want[1])):
        ref.assert_near(ref.host(got[:rows, :n]), v, ref.rounded(v, off) if typ == F16 else off + 2.0 ** -23 * np.abs(v), f"{n} {kind}")
        assert torch.all(got[rows:] == 7) and torch.all(got[:, n:] == 7), "memory behind the rows or values was written"


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_block_norm(n, kind):
    i = WIDTHS.index(n) + (kind == "layer") * 7
    check_norm(5, n, kind, i, (i % 3, i % 2, 2, 4))


@pytest.mark.parametrize("n", [n for n in WIDTHS if n % 8 == 0])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_block_norm_of_whole_pieces(n, kind):
    i = WIDTHS.index(n) + (kind == "layer") * 7
    check_norm(5, n, kind, i + 1, (0, 8, 16, 0))


@pytest.mark.parametrize("rows,n", [(6000, 24), (3000, 136), (700, 1024), (640, 4096), (500, 8192), (470, 8200), (310, 16384), (320, 16392), (310, 32768),
                                    (6000, 17), (3000, 33), (700, 1125), (500, 4095), (330, 4097), (152, 5935), (330, 5935), (310, 8193), (310, 16385)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("turn", range(3))
def test_more_rows_than_run_at_once(rows, n, kind, turn):
    check_norm(rows, n, kind, n + 5 * turn + (kind == "layer") + turn // 2, (8, 0, 0, 16) if n % 8 == 0 else (0, turn, 1, 0))


@pytest.mark.parametrize("n", [72, 4096])
def test_norms_in_place_and_with_buffers_left_out(n):
    rows, rng = 70, np.random.default_rng(n)
    (block, b), (res, r) = rows_of(rng, rows, n), rows_of(rng, rows, n, F32)
    (_, t_off), (z, z_off) = want = ref.block_norm(b, r, eps=float(np.float32(1e-5)))
    norms = q4.BlockNorm.of(n)
    q4.q4_block_norm(norms, rows, block, F16, n, res, F32, n, res, F32, n, block, F16, n)      # t into the residual, z into the block
    settled()
    ref.assert_near(ref.host(res), want[0][0], t_off + 2.0 ** -23 * np.abs(want[0][0]))
    ref.assert_near(ref.host(block), z, ref.rounded(z, z_off))
    x, v = rows_of(rng, rows, n, F32)
    out = torch.zeros((rows, n), dtype=torch.float32, device="cuda")
    q4.q4_block_norm(norms, rows, None, F16, n, x, F32, n, None, F16, n, out, F32, n)          # the residual's norm alone
    settled()
    z, off = ref.block_norm(None, v, eps=float(np.float32(1e-5)))[1]
    ref.assert_near(ref.host(out), z, off + 2.0 ** -23 * np.abs(z))
    q4.q4_block_norm(norms, rows, x, F32, n, None, F16, n, out, F32, n, None, F16, n)          # t alone: a copy
    settled()
    assert torch.equal(out, x)
    q4.q4_block_norm(norms, 0, x, F32, n, None, F16, n, out, F32, n, None, F16, n)


def test_norms_of_rows_that_are_zero_or_not_finite():
    n, rows = 300, 6
    x = torch.ones((rows, n), device="cuda")
    x[0], x[2, 5], x[3, 7], x[5] = 0, math.nan, math.inf, 2.0 ** 56
    z = torch.zeros((rows, n), device="cuda")
    q4.q4_block_norm(q4.BlockNorm.of(n), rows, x, F32, n, None, F32, n, None, F32, n, z, F32, n)
    settled()
    assert torch.all(z[0] == 0) and not torch.isfinite(z[2, 5]) and not torch.isfinite(z[3, 7])
    assert torch.allclose(z[1], torch.full((n,), 1 / math.sqrt(1 + 1e-5), device="cuda")) and torch.allclose(z[5], torch.ones(n, device="cuda"))
    assert torch.equal(z[1], z[4])


# ------------------------------------------------------------------ rotary positions

HEADS = [(1, 2, 2), (3, 6, 4), (3, 7, 4), (65, 9, 2), (5, 64, 64), (40, 128, 128), (8, 80, 40), (2, 80, 38), (3, 192, 96), (2, 256, 256), (7, 100, 10), (1, 1024, 256)]


@pytest.mark.parametrize("heads,head_dim,rot", HEADS)
@pytest.mark.parametrize("halves", [True, False])
def test_rope(heads, head_dim, rot, halves):
    i = HEADS.index((heads, head_dim, rot)) + 10 * halves
    rng, pairs, axes = np.random.default_rng(i), rot // 2, 1 + i % 4
    freqs = [10000.0 ** (-j / pairs) for j in range(pairs)]
    axis = [(j * 7) % axes for j in range(pairs)]
    xt, yt = F32 if i & 1 else F16, F32 if i & 2 else F16
    rot_ = q4.Rope.of(head_dim, freqs, axis, q4.Q4_ROPE_HALVES if halves else q4.Q4_ROPE_ADJACENT)
    for rows in (1, 9, 200):
        n = heads * head_dim
        places = rng.integers(-1000, 2 ** (10 + i), size=(axes, rows + 2))
        x, v = rows_of(rng, rows, n, xt, n + 8 * (i % 3))
        y = torch.full((rows + 1, n + i % 5), 7.0, dtype=TORCH[yt], device="cuda")
        at = q4.RopePlaces.of(dev(places.astype(np.int32)), axes, rows, rows + 2)
        for inverse in (False, True):
            q4.q4_rope(rot_, at, heads, x, xt, x.shape[1], y, yt, y.shape[1], inverse)
            settled()
            want, off = ref.rope(v, places[:, :rows], freqs, axis, head_dim, halves, inverse)
            ref.assert_near(ref.host(y[:rows, :n]), want, ref.rounded(want, off) if yt == F16 else off, f"{rows} rows")
            assert torch.all(y[rows:] == 7) and torch.all(y[:, n:] == 7), "memory behind the rows or values was written"


def test_rope_in_place_and_back():
    rng, heads, hd, rows = np.random.default_rng(1), 10, 64, 33
    freqs = [10000.0 ** (-j / 32) for j in range(32)]
    x, v = rows_of(rng, rows, heads * hd, F32)
    at = q4.RopePlaces.of(dev(rng.integers(0, 10 ** 6, size=(1, rows)).astype(np.int32)), 1, rows)
    rot = q4.Rope.of(hd, freqs)
    q4.q4_rope(rot, at, heads, x, F32, heads * hd, x, F32, heads * hd)
    moved = ref.host(x)
    q4.q4_rope(rot, at, heads, x, F32, heads * hd, x, F32, heads * hd, inverse=True)
    settled()
    # (there and back with the same cosine and sine: their squares add up to 1 within 2^-20)
    assert np.abs(moved - v).max() > 0.5 and np.abs(ref.host(x) - v).max() < 2.0 ** -19 * np.abs(v).max()


def test_rope_far_positions_and_frequencies_beyond_a_turn():
    """The largest positions of an int, and angles of many turns per position."""
    freqs = [1.0, 100.0, -3.0, 2 * math.pi * 0.25]
    places = np.array([[2 ** 31 - 1, -2 ** 31, 0, 1, 123456789]])
    rng, rows = np.random.default_rng(3), 5
    x, v = rows_of(rng, rows, 8, F32)
    y = torch.zeros_like(x)
    q4.q4_rope(q4.Rope.of(8, freqs), q4.RopePlaces.of(dev(places.astype(np.int32)), 1, rows), 1, x, F32, 8, y, F32, 8)
    settled()
    ref.assert_near(ref.host(y), *ref.rope(v, places, freqs, [0] * 4, 8, True))


@pytest.mark.parametrize("heads,hd", [(1, 8), (1, 16), (3, 8)])
@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("rows", [1, 2500])
def test_rope_of_the_smallest_heads(heads, hd, halves, rows):
    """Rows of one or a few 16-byte pieces, where a share of the rows' pieces rounds to none."""
    rng, pairs = np.random.default_rng(heads * hd), hd // 2
    freqs = [10000.0 ** (-j / pairs) for j in range(pairs)]
    places = rng.integers(0, 100000, size=(1, rows))
    x, v = rows_of(rng, rows, heads * hd, F16)
    y = torch.full((rows + 1, heads * hd), 7.0, dtype=torch.float16, device="cuda")
    rot = q4.Rope.of(hd, freqs, None, q4.Q4_ROPE_HALVES if halves else q4.Q4_ROPE_ADJACENT)
    q4.q4_rope(rot, q4.RopePlaces.of(dev(places.astype(np.int32)), 1, rows), heads, x, F16, heads * hd, y, F16, heads * hd)
    settled()
    want, off = ref.rope(v, places, freqs, [0] * pairs, hd, halves)
    ref.assert_near(ref.host(y[:rows]), want, ref.rounded(want, off))
    assert torch.all(y[rows:] == 7), "memory behind the rows was written"


@pytest.mark.parametrize("new", [[1], [3, 0, 5], [1] * 40, [0, 0, 2], [100, 1, 1, 300]])
def test_rope_at_a_batchs_positions(new):
    rng, heads, hd = np.random.default_rng(len(new)), 6, 128
    freqs = [10000.0 ** (-j / 64) for j in range(64)]
    starts = np.concatenate([[0], np.cumsum(new)]) + 1          # the first row belongs to no sequence
    lens = np.array(new) + rng.integers(0, 5000, size=len(new))
    lens[-1] = new[-1] - 1                                       # a row before position 0
    rows = int(starts[-1]) + 3                                   # nor do the last ones
    x, v = rows_of(rng, rows, heads * hd, F32, heads * hd + 256)
    y = torch.full((rows, heads * hd), 7.0, dtype=torch.float16, device="cuda")
    at = q4.RopePlaces.of_batch(dev(starts.astype(np.int32)), dev(lens.astype(np.int32)), len(new), rows)
    q4.q4_rope(q4.Rope.of(hd, freqs), at, heads, x, F32, heads * hd + 256, y, F16, heads * hd)
    settled()
    places = np.concatenate([np.arange(length - n, length) for n, length in zip(new, lens)])[None]
    a, b = int(starts[0]), int(starts[-1])
    want, off = ref.rope(v[a:b], places, freqs, [0] * 64, hd, True)
    ref.assert_near(ref.host(y[a:b]), want, ref.rounded(want, off))
    assert torch.all(y[:a] == 7) and torch.all(y[b:] == 7), "rows of no sequence were written"


def test_norms_and_rope_in_a_graph():
    rng, rows, heads, hd = np.random.default_rng(8), 21, 4, 64
    n = heads * hd
    x, _ = rows_of(rng, rows, n, F32)
    places = torch.zeros((1, rows), dtype=torch.int32, device="cuda")
    rot, at, norms = q4.Rope.of(hd, [0.5 ** j for j in range(32)]), q4.RopePlaces.of(places, 1, rows), q4.BlockNorm.of(n)
    z, y = torch.zeros((rows, n), device="cuda"), torch.zeros((rows, n), device="cuda")

    def both():
        q4.q4_block_norm(norms, rows, x, F32, n, None, F32, n, None, F32, n, z, F32, n)
        q4.q4_rope(rot, at, heads, z, F32, n, y, F32, n)

    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for step in (3, 70000):
        x.copy_(dev(rng.normal(size=(rows, n))).float())
        places.copy_(torch.arange(rows, device="cuda")[None] * step)
        g.replay()
        settled()
        zw, off = ref.block_norm(ref.host(x), None, eps=float(np.float32(1e-5)))[1]
        ref.assert_near(ref.host(z), zw, off + 2.0 ** -23 * np.abs(zw))
        ref.assert_near(ref.host(y), *ref.rope(ref.host(z), ref.host(places), [0.5 ** j for j in range(32)], [0] * 32, hd, True))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("new,ctx", [([1], [70]), ([5, 1, 37], [0, 64, 20]), ([150], [33])])
def test_a_layer_over_the_paged_cache(new, ctx):
    """A ragged step through a whole layer: every operator against its plain form of what the one before it left."""
    rng, hidden, heads, kv_heads, hd, ffn, page = np.random.default_rng(sum(new)), 256, 4, 2, 64, 672, 16
    rows, lens = sum(new), [a + b for a, b in zip(new, ctx)]
    qkv = (heads + 2 * kv_heads) * hd
    width = max(-(-n // page) for n in lens)
    shapes = dict(qkv=(qkv, hidden), o=(hidden, heads * hd), gate=(ffn, hidden), up=(ffn, hidden), down=(hidden, ffn))
    blocks = {m: ref.q4_bytes(n, k, i) for i, (m, (n, k)) in enumerate(shapes.items())}
    w, wd = {m: ref.weights(b) for m, b in blocks.items()}, {m: dev(b) for m, b in blocks.items()}
    table = rng.permutation(len(new) * width).astype(np.int32).reshape(len(new), width)
    starts, lens_d, table_d = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), dev(np.array(lens, dtype=np.int32)), dev(table)
    pages = [dev(rng.normal(size=(table.size, kv_heads, page, hd))).half() for _ in range(2)]
    kv = q4.PagedKV.of(*pages, table.size, page, kv_heads, hd)
    batch = q4.PagedBatch.of(starts, lens_d, table_d, len(new), rows, width, max(new))
    freqs = [10000.0 ** (-j / 32) for j in range(32)]
    rot, at = q4.Rope.of(hd, freqs), q4.RopePlaces.of_batch(starts, lens_d, len(new), rows)
    weight = [rng.normal(size=hidden).astype(np.float32) for _ in range(2)]
    norms = [q4.BlockNorm.of(hidden, weight=dev(v)) for v in weight]
    eps = float(np.float32(1e-5))

    def buffer(n, kind=torch.float16):
        return torch.zeros((rows, n), dtype=kind, device="cuda")

    stream, z, r, a, o, act, t2 = buffer(hidden, torch.float32), buffer(hidden), buffer(qkv), buffer(heads * hd), buffer(hidden), buffer(ffn), buffer(hidden)
    stream.copy_(dev(rng.normal(size=(rows, hidden))).float())
    s0 = ref.host(stream)
    ws_bytes = q4.q4_attn_paged_workspace_bytes(heads, kv_heads, hd)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    ep = q4.Epilogue.of(hidden, rows, residual=o)

    def layer():
        q4.q4_block_norm(norms[0], rows, None, F16, hidden, stream, F32, hidden, None, F16, hidden, z, F16, hidden)
        q4.q4_gemm(wd["qkv"], z, hidden, qkv, hidden, rows, None, r, qkv)
        q4.q4_rope(rot, at, heads + kv_heads, r, F16, qkv, r, F16, qkv)
        k = r.data_ptr() + 2 * heads * hd
        q4.q4_paged_write(kv, batch, k, k + 2 * kv_heads * hd, F16, qkv)
        q4.q4_attn_paged(kv, batch, r, F16, qkv, heads, 0, 0, a, heads * hd, ws, ws_bytes)
        q4.q4_gemm(wd["o"], a, heads * hd, hidden, heads * hd, rows, None, o, hidden)
        q4.q4_block_norm(norms[1], rows, o, F16, hidden, stream, F32, hidden, stream, F32, hidden, z, F16, hidden)
        q4.q4_gemm_gated(wd["gate"], wd["up"], z, hidden, ffn, hidden, rows, None, act, ffn)
        q4.q4_gemm(wd["down"], act, ffn, hidden, ffn, rows, ep, t2, hidden)

    layer()
    settled()
    first = [t.clone() for t in (r, a, o, stream, z, act, t2)]
    # the first norm and the product's rows, turned (z and r have been overwritten since: they are made again, apart)
    z0, r0 = buffer(hidden), buffer(qkv)
    q4.q4_block_norm(norms[0], rows, None, F16, hidden, dev(s0, torch.float32), F32, hidden, None, F16, hidden, z0, F16, hidden)
    q4.q4_gemm(wd["qkv"], z0, hidden, qkv, hidden, rows, None, r0, qkv)
    settled()
    v, off = ref.block_norm(None, s0, eps=eps, weight=weight[0])[1]
    ref.assert_near(ref.host(z0), v, ref.rounded(v, off), "first norm")
    ref.assert_near(ref.host(r0), *ref.gemm(w["qkv"], ref.host(z0)), "q | k | v")
    places = np.concatenate([np.arange(n - m, n) for m, n in zip(new, lens)])[None]
    n_turn = (heads + kv_heads) * hd
    v, off = ref.rope(ref.host(r0)[:, :n_turn], places, freqs, [0] * 32, hd, True)
    ref.assert_near(ref.host(r)[:, :n_turn], v, ref.rounded(v, off), "turned")
    assert torch.equal(r[:, n_turn:], r0[:, n_turn:])
    # attention over the pages, the new tokens' keys and values among them
    kh, vh = (ref.host(p) for p in pages)
    for s, (m, n) in enumerate(zip(new, lens)):
        rr = slice(int(starts[s]), int(starts[s + 1]))
        keys, values = (np.stack([h[table[s, p // page], :, p % page] for p in range(n)]) for h in (kh, vh))
        np.testing.assert_array_equal(keys[n - m:].reshape(m, -1), ref.host(r)[rr, heads * hd:n_turn])
        np.testing.assert_array_equal(values[n - m:].reshape(m, -1), ref.host(r)[rr, n_turn:])
        q = ref.host(r)[rr, :heads * hd].reshape(m, heads, hd)
        for h in range(heads):
            kk, vv = keys[:, h // 2], values[:, h // 2]
            sc = q[:, h] @ kk.T / 8 + np.where(np.arange(n)[None] <= np.arange(n - m, n)[:, None], 0.0, -np.inf)
            p = np.exp(sc - sc.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            big = (np.abs(q[:, h]) @ np.abs(kk).T / 8).max(1, keepdims=True)
            off = (2.0 ** -10 + 2.0 ** -19 * big) * (p @ np.abs(vv)) + n * 2.0 ** -25 * np.abs(vv).max() + 2.0 ** -24
            ref.assert_near(ref.host(a)[rr, h * hd:(h + 1) * hd], p @ vv, off, "attention")
    ref.assert_near(ref.host(o), *ref.gemm(w["o"], ref.host(a)), "o")
    (t, t_off), (v, off) = ref.block_norm(ref.host(o), s0, eps=eps, weight=weight[1])
    ref.assert_near(ref.host(stream), t, t_off + 2.0 ** -23 * np.abs(t), "residual stream")
    ref.assert_near(ref.host(z), v, ref.rounded(v, off), "second norm")
    ref.assert_near(ref.host(act), *ref.gated(w["gate"], w["up"], ref.host(z)), "gated product")
    ref.assert_near(ref.host(t2), *ref.gemm(w["down"], ref.host(act), residual=ref.host(o)), "down")
    # the same step from a graph
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for t in (r, a, o, z, act, t2):
        t.zero_()
    stream.copy_(dev(s0, torch.float32))
    g.replay()
    settled()
    for got, before in zip((r, a, o, stream, z, act, t2), first):
        assert torch.equal(got, before)
