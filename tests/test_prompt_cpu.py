"""The host-side checks of the operators of a prompt's layer, and what their binding refuses of tensors (no GPU)."""
import ctypes
import math

import pytest

import weight_streaming_q4_gb300 as q4
from weight_streaming_q4_gb300 import _lib, build

torch = pytest.importorskip("torch")

A = 4096    # a 16-byte aligned fake address; never dereferenced
F16, F32 = q4.Q4_TYPE_F16, q4.Q4_TYPE_F32
ARG, ALIGN, OK = q4.Q4_ERR_ARG, q4.Q4_ERR_ALIGN, q4.Q4_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q4.lib()


def gemm(lib, **over):
    d = dict(w=A, w_up=A, x=A, x_ld=64, n=8, k=64, rows=2, bias=None, act=0, residual=None, residual_type=F16, residual_ld=8, y=A, y_ld=8)
    d.update(over)
    ep = q4.Epilogue(d["bias"], d["act"], 1.0, d["residual"], d["residual_type"], d["residual_ld"])
    gep = q4.GatedEpilogue(d["bias"], d["bias"], d["act"])
    one = lib.q4_gemm(d["w"], d["x"], d["x_ld"], d["n"], d["k"], d["rows"], ep, d["y"], d["y_ld"], None)
    two = lib.q4_gemm_gated(d["w"], d["w_up"], d["x"], d["x_ld"], d["n"], d["k"], d["rows"], gep, d["y"], d["y_ld"], None)
    return one, two


@pytest.mark.parametrize("over", [dict(w=None), dict(x=None), dict(y=None), dict(n=0), dict(n=-1), dict(k=0), dict(k=48), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(x_ld=56),
                                  dict(y_ld=7), dict(act=5), dict(act=-1), dict(n=1 << 20, k=(1 << 14) - 32, x_ld=1 << 14, y_ld=1 << 20), dict(x_ld=(1 << 31) + 8),
                                  dict(y_ld=(1 << 31) + 1), dict(n=(1 << 30) + 1, y_ld=1 << 31, residual_ld=1 << 31)], ids=str)
def test_product_arguments(lib, over):
    assert gemm(lib, **over) == (ARG, ARG)


@pytest.mark.parametrize("over", [dict(w=A + 8), dict(x=A + 2), dict(x=A + 8), dict(x_ld=68), dict(y=A + 1), dict(bias=A + 2)], ids=str)
def test_product_alignment(lib, over):
    assert gemm(lib, **over) == (ALIGN, ALIGN)


def test_products_own_arguments(lib):
    assert gemm(lib, w_up=None)[1] == ARG and gemm(lib, w_up=A + 4)[1] == ALIGN
    assert gemm(lib, residual=A, residual_type=2)[0] == ARG and gemm(lib, residual=A, residual_ld=7)[0] == ARG
    assert gemm(lib, residual=A + 2, residual_type=F32)[0] == ALIGN and gemm(lib, residual=A + 1)[0] == ALIGN
    # no row: nothing to do, the rows are not looked at
    assert gemm(lib, rows=0, x=None, y=None) == (OK, OK)


def test_products_onto_their_inputs(lib):
    far = dict(w=2 * A, w_up=3 * A, x=4 * A, y=A)
    assert gemm(lib, **{**far, "x": A}) == (ARG, ARG) and gemm(lib, **{**far, "w": A}) == (ARG, ARG) and gemm(lib, **{**far, "w_up": A})[1] == ARG
    # the residual may be y, in y's rows
    assert gemm(lib, **far, residual=A, residual_type=F32)[0] == ARG and gemm(lib, **far, residual=A, residual_ld=9)[0] == ARG
    assert gemm(lib, **far, rows=1, residual=A, residual_type=F32)[0] == ARG


def norm(lib, kind=0, eps=1e-5, gate=None, gate_ld=8, gate_rows=0, weight=None, rows=2, n=8, block=A, residual=None, t=None, z=A, types=(F16,) * 4, ld=8):
    p = q4.BlockNorm(kind, eps, 0, None, None, 1.0, gate, gate_ld, gate_rows, weight, None)
    return lib.q4_block_norm(p, rows, n, block, types[0], ld, residual, types[1], ld, t, types[2], ld, z, types[3], ld, None)


@pytest.mark.parametrize("over", [dict(kind=2), dict(kind=-1), dict(eps=-1.0), dict(eps=math.nan), dict(n=0), dict(n=32769, ld=32769), dict(rows=-1), dict(rows=(1 << 24) + 1),
                                  dict(block=None), dict(z=None), dict(ld=7), dict(types=(2, F16, F16, F16)), dict(types=(F16, F16, F16, -1)),
                                  dict(residual=A, types=(F16, 3, F16, F16)), dict(t=A, types=(F16, F16, 4, F16)), dict(gate=A, gate_rows=-1),
                                  dict(gate=A, gate_rows=1, gate_ld=7)], ids=str)
def test_norm_arguments(lib, over):
    assert norm(lib, **over) == ARG


@pytest.mark.parametrize("over", [dict(block=A + 1), dict(residual=A + 2, types=(F16, F32, F16, F16)), dict(t=A + 1), dict(z=A + 2, types=(F16, F16, F16, F32)),
                                  dict(gate=A + 1), dict(weight=A + 2)], ids=str)
def test_norm_alignment(lib, over):
    assert norm(lib, **over) == ALIGN
    assert lib.q4_block_norm(None, 1, 8, A, F16, 8, None, F16, 8, None, F16, 8, A, F16, 8, None) == ARG
    assert norm(lib, rows=0, block=None, z=None) == OK


def test_norms_onto_their_inputs(lib):
    assert norm(lib, block=A, t=2 * A, z=2 * A) == ARG
    for over in (dict(block=A, z=A, types=(F16, F16, F16, F32)), dict(block=A, z=2 * A, t=A, types=(F32, F16, F16, F16)),
                 dict(block=A, residual=2 * A, z=2 * A, types=(F16, F32, F16, F16)), dict(block=A, residual=2 * A, t=2 * A, z=3 * A, types=(F16, F16, F32, F16))):
        assert norm(lib, **over) == ARG
    p = q4.BlockNorm(0, 1e-5, 0, None, None, 1.0, None, 0, 0, None, None)
    assert lib.q4_block_norm(p, 2, 8, A, F16, 8, None, F16, 8, None, F16, 8, A, F16, 16, None) == ARG


def test_rotations(lib):
    r = q4.Rope.of(128, [1.0, 0.25, 2 * math.pi], [0, 2, 1], q4.Q4_ROPE_ADJACENT)
    assert (r.head_dim, r.rot_dim, r.style, r.n_axes) == (128, 6, q4.Q4_ROPE_ADJACENT, 3) and list(r.axis[:3]) == [0, 2, 1]
    for got, f in zip(r.turn, (1.0, 0.25)):
        assert abs(got / 2 ** 64 - f / (2 * math.pi)) < 2.0 ** -50
    assert min(r.turn[2], 2 ** 64 - r.turn[2]) < 2 ** 12              # a whole turn
    back = q4.Rope.of(8, [-1e-6]).turn[0]                             # (its bits are kept although it wraps)
    assert abs((back - 2 ** 64) / 2 ** 64 + 1e-6 / (2 * math.pi)) < 2.0 ** -64 + 1e-6 * 2.0 ** -50
    for bad in (dict(head_dim=4, freqs=[1.0] * 3), dict(head_dim=1, freqs=[1.0]), dict(head_dim=1026, freqs=[1.0]), dict(head_dim=512, freqs=[1.0] * 129),
                dict(head_dim=8, freqs=[]), dict(head_dim=8, freqs=[math.inf]), dict(head_dim=8, freqs=[math.nan]), dict(head_dim=8, freqs=[1.0], axes=[4]),
                dict(head_dim=8, freqs=[1.0], axes=[-1]), dict(head_dim=8, freqs=[1.0], style=2), dict(head_dim=8, freqs=[1.0], axes=[0, 0])):
        with pytest.raises(q4.Q4Error):
            q4.Rope.of(**bad)
    assert lib.q4_rotation_init(None, 8, 2, (ctypes.c_double * 1)(1.0), None, 0) == ARG
    assert lib.q4_rotation_init(q4.Rope(), 8, 2, None, None, 0) == ARG


def rope(lib, rot=None, heads=2, x=A, x_type=F16, x_ld=16, y=2 * A, y_type=F16, y_ld=16, **places):
    d = dict(positions=A, ld=3, n_axes=1, token_starts=None, kv_lens=None, n_seqs=0, n_tokens=3)
    d.update(places)
    return lib.q4_rope(rot or q4.Rope.of(8, [1.0]), q4.RopePlaces(**d), 0, heads, x, x_type, x_ld, y, y_type, y_ld, None)


BATCH = dict(positions=None, token_starts=A, kv_lens=A, n_seqs=2)


@pytest.mark.parametrize("over", [dict(heads=0), dict(heads=65537), dict(n_tokens=-1), dict(n_tokens=(1 << 24) + 1, ld=1 << 25), dict(ld=2), dict(n_axes=0), dict(x=None), dict(y=None),
                                  dict(x_ld=15), dict(y_ld=15), dict(x_type=2), dict(y_type=2), dict(y=A, y_type=F32), dict(y=A, y_ld=24),
                                  dict(BATCH, n_seqs=-1), dict(BATCH, n_seqs=65536), dict(BATCH, token_starts=None), dict(BATCH, kv_lens=None)], ids=str)
def test_rope_arguments(lib, over):
    assert rope(lib, **over) == ARG


def test_rope_alignment_and_calls_of_nothing(lib):
    for over in (dict(positions=A + 2), dict(x=A + 1), dict(y=A + 2, y_type=F32), dict(BATCH, token_starts=A + 1), dict(BATCH, kv_lens=A + 2)):
        assert rope(lib, **over) == ALIGN
    assert rope(lib, n_tokens=0, x=None) == OK and rope(lib, **dict(BATCH, n_seqs=0)) == OK
    assert lib.q4_rope(None, q4.RopePlaces(), 0, 1, A, F16, 8, A, F16, 8, None) == ARG
    assert lib.q4_rope(q4.Rope.of(8, [1.0]), None, 0, 1, A, F16, 8, A, F16, 8, None) == ARG
    # an axis that the places have not, in a rotation that was written by hand too
    two = q4.Rope.of(8, [1.0, 0.5], [0, 1])
    assert rope(lib, rot=two) == ARG
    two.n_axes = 1
    assert rope(lib, rot=two) == ARG
    for field, value in (("head_dim", 0), ("rot_dim", 3), ("rot_dim", 16), ("rot_dim", 512), ("style", 7)):
        bad = q4.Rope.of(8, [1.0])
        setattr(bad, field, value)
        assert rope(lib, rot=bad) == ARG


# ------------------------------------------------------------------ the binding (host tensors that are taken for the current device's)

@pytest.fixture
def on_device(monkeypatch):
    monkeypatch.setattr(_lib, "_device", lambda: -1)


def refused(f, *args, **kw):
    with pytest.raises(q4.Q4Error) as e:
        f(*args, **kw)
    return e.value.status == ARG


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def test_epilogues_of_tensors(lib, on_device):
    e = q4.Epilogue.of(8, 3, bias=f32(8), residual=f16(3, 8))
    assert e.residual_ld == 8 and e.residual == e._keep[1].data_ptr()
    for bad in (dict(bias=f32(7)), dict(bias=f16(8)), dict(bias=f32(16)[::2]), dict(residual=f16(2, 8)), dict(residual=f32(3, 8)), dict(residual=f16(3, 9)),
                dict(residual=f16(3, 8), residual_type=F32), dict(residual=f16(3, 8), residual_ld=16)):
        assert refused(q4.Epilogue.of, 8, 3, **bad)
    assert refused(q4.GatedEpilogue.of, 8, q4.Q4_ACT_SILU, f32(7)) and refused(q4.GatedEpilogue.of, 8, q4.Q4_ACT_SILU, None, f16(8))


def test_products_of_tensors(lib, on_device):
    n, k, rows = 8, 64, 3
    good = dict(w=torch.zeros((n, k // 32, 18), dtype=torch.uint8), x=f16(rows, k), x_ld=k, n=n, k=k, rows=rows, ep=None, y=f16(rows, n), y_ld=n)
    bad = [dict(w=good["w"][1:]), dict(w=f16(n, k)), dict(w=good["w"].repeat(1, 2, 1)[:, ::2]), dict(x=f16(2, k)), dict(x=f32(rows, k)), dict(x=f16(rows, 2 * k)),
           dict(x=f16(k, rows).T), dict(y=f16(2, n)), dict(y=f32(rows, n)), dict(y=f16(rows, 2 * n)), dict(ep=q4.Epilogue.of(n + 1, rows, bias=f32(n + 1))),
           dict(ep=q4.Epilogue.of(n, rows - 1, residual=f16(rows - 1, n)))]
    for b in bad:
        assert refused(q4.q4_gemm, **{**good, **b}), b.keys()
    two = {("w_gate" if key == "w" else key): v for key, v in good.items()}
    assert refused(q4.q4_gemm_gated, w_up=good["w"][1:], **two) and refused(q4.q4_gemm_gated, w_up=good["w"], **{**two, "w_gate": good["w"][1:]})
    assert refused(q4.q4_gemm_gated, w_up=good["w"], **{**two, "ep": q4.GatedEpilogue.of(n + 8)})


def test_norms_of_tensors(lib, on_device):
    assert q4.BlockNorm.of(8, post_weight=f32(8)).post and not q4.BlockNorm.of(8).post
    for bad in (dict(weight=f32(7)), dict(bias=f16(8)), dict(post_weight=f32(4)), dict(post_bias=f32(7)), dict(gate=f32(7)), dict(gate=f16(2, 8), gate_rows=1)):
        assert refused(q4.BlockNorm.of, 8, **bad)
    p = q4.BlockNorm.of(8, gate=f32(2, 8), gate_rows=3)
    rows = [f16(7, 8), F16, 8, None, F16, 8, None, F16, 8, f16(7, 8), F16, 8]
    assert refused(q4.q4_block_norm, p, 7, *rows)                     # gates for six rows
    for i, bad in ((0, f16(6, 8)), (0, f32(7, 8)), (3, f16(6, 8)), (6, f16(7, 9)), (9, f32(7, 8))):
        assert refused(q4.q4_block_norm, q4.BlockNorm.of(8), 7, *rows[:i], bad, *rows[i + 1:])
    assert refused(q4.q4_block_norm, q4.BlockNorm.of(8), 7, *rows, n=9)


def test_places_of_tensors(lib, on_device):
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)     # noqa: E731
    assert q4.RopePlaces.of(i32(12), 3, 4).ld == 4
    for bad in ((i32(11), 3, 4), (torch.zeros(12, dtype=torch.int64), 3, 4), (i32(24)[::2], 3, 4), (i32(12), 3, 4, 5)):
        assert refused(q4.RopePlaces.of, *bad)
    assert refused(q4.RopePlaces.of_batch, i32(2), i32(2), 2, 4) and refused(q4.RopePlaces.of_batch, i32(3), i32(1), 2, 4)
    at = q4.RopePlaces.of(i32(4), 1, 4)
    rot = q4.Rope.of(8, [1.0])
    for x, y in ((f16(3, 16), f16(4, 16)), (f16(4, 16), f16(4, 15)), (f32(4, 16), f16(4, 16)), (f16(4, 16), f32(4, 16))):
        assert refused(q4.q4_rope, rot, at, 2, x, F16, 16, y, F16, 16)


def test_descriptors_of_another_device(lib, on_device, monkeypatch):
    ep, norms, at = q4.Epilogue.of(8, 3, bias=f32(8)), q4.BlockNorm.of(8, weight=f32(8)), q4.RopePlaces.of(torch.zeros(4, dtype=torch.int32), 1, 4)
    monkeypatch.setattr(_lib, "_device", lambda: 1)
    assert refused(q4.q4_gemm, A, A, 64, 8, 64, 3, ep, A, 8) and refused(q4.q4_block_norm, norms, 3, A, F16, 8, None, F16, 8, None, F16, 8, A, F16, 8)
    assert refused(q4.q4_rope, q4.Rope.of(8, [1.0]), at, 1, A, F16, 8, 2 * A, F16, 8)
