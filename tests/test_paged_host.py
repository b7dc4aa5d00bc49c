"""Host side of the paged cache (no GPU): the rotation's frequencies, and
the refusals of every entry point before it touches the device."""
import ctypes as C

import numpy as np
import pytest

import diffusion_transformer_denoiser_qi21_gb300 as q
from diffusion_transformer_denoiser_qi21_gb300 import _binding as B
from tests import pagedcheck as P


def _turns(r):
    return np.array([int(t) for t in r.turns[:r.rot_dim // 2]], dtype=object)


@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("kw", [dict(scaling="plain"), dict(scaling="linear", factor=4.0),
                                dict(scaling="base", factor=8.0), dict(scaling="ramp", factor=8.0, orig_len=8192.0),
                                dict(scaling="ramp", factor=32.0, orig_len=40.0),
                                dict(scaling="band", factor=8.0, orig_len=8192.0)])
def test_frequencies(rot, kw):
    if rot == 2 and kw["scaling"] == "base":
        pytest.skip("one pair: there is no slowest pair to stretch to")
    r = q.rope(128, rot, **kw)
    want = P.frequencies(rot, **kw)
    got = np.array([float(t) for t in _turns(r) * 1]) * 2.0 ** -64 * 2 * np.pi
    # f64 evaluations of one formula: a few ulp of pow, log and the mixing
    np.testing.assert_allclose(got, want, rtol=1e-13, atol=0)
    scale = 0.1 * np.log(kw.get("factor", 1.0)) + 1 if kw["scaling"] == "ramp" else 1.0
    assert r.out_scale == np.float32(scale)
    assert (r.head_dim, r.rot_dim, r.naxes) == (128, rot, 1)


def test_three_axes_follow_the_layout():
    r = q.rope(128, axes=(16, 56, 56))
    assert r.naxes == 3
    assert list(r.axis[:64]) == [0] * 8 + [1] * 28 + [2] * 28
    got = np.array([float(t) for t in _turns(r)]) * 2.0 ** -64 * 2 * np.pi
    np.testing.assert_allclose(got, np.concatenate([P.frequencies(w) for w in (16, 56, 56)]), rtol=1e-13)


def test_out_scale_given():
    assert q.rope(64, scaling="ramp", factor=4.0, orig_len=100.0, out_scale=0.5).out_scale == 0.5
    assert q.rope(64, out_scale=-2.0).out_scale == -2.0


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=127), -3), (dict(head_dim=0), -3), (dict(head_dim=258), -3),
    (dict(head_dim=64, rot_dim=66), -3), (dict(head_dim=64, rot_dim=7), -3), (dict(head_dim=64, rot_dim=0), -3),
    (dict(head_dim=128, axes=(16, 56, 58)), -3), (dict(head_dim=128, axes=(15, 57, 56)), -3),
    (dict(head_dim=128, axes=(-2, 74, 56)), -3),
    (dict(head_dim=64, base=1.0), -1), (dict(head_dim=64, base=float("nan")), -1),
    (dict(head_dim=64, scaling="linear", factor=0.5), -1), (dict(head_dim=64, factor=float("inf")), -1),
    (dict(head_dim=64, scaling="ramp", factor=2.0), -1),  # no orig_len
    (dict(head_dim=64, scaling="band", factor=2.0, orig_len=100.0, fast_turns=1.0, slow_turns=1.0), -1),
    (dict(head_dim=64, scaling="band", factor=2.0, orig_len=100.0, slow_turns=-1.0), -1),
    (dict(head_dim=64, out_scale=float("nan")), -1),
])
def test_rope_refusals(kw, code):
    with pytest.raises(q.Qi21Error) as e:
        q.rope(**kw)
    assert e.value.code == code


def test_rope_names():
    with pytest.raises(ValueError):
        q.rope(64, layout="pairs")
    with pytest.raises(ValueError):
        q.rope(64, scaling="other")
    with pytest.raises(ValueError):
        q.rope(128, axes=(64, 64))


def test_op_rope_refuses_before_the_device():
    lib = q.load()
    r = q.rope(64)
    call = lambda r=C.byref(r), elem=2, rows=4, heads=2, x=16, ldx=128, out=4096, ldo=128, pos=8, grad=0: \
        lib.qi21_op_rope(r, elem, rows, heads, x, ldx, out, ldo, pos, grad, None)  # noqa: E731
    assert call(rows=0, x=None, out=None, pos=None) == 0
    assert call(r=None) == -1
    assert call(elem=0) == -1 and call(elem=5) == -1
    assert call(grad=2) == -1
    assert call(rows=-1) == -2 and call(heads=0) == -2 and call(heads=2000) == -2
    assert call(ldx=127) == -2 and call(ldo=127) == -2
    assert call(x=None) == -1 and call(out=None) == -1 and call(pos=None) == -1
    assert call(x=17) == -1 and call(elem=4, x=18) == -1 and call(pos=12) == -1
    assert call(x=4096, ldx=256) == -1  # in place with another stride
    bad = q.rope(64)
    bad.axis[3] = 1
    assert call(r=C.byref(bad)) == -1
    bad = q.rope(64)
    bad.rot_dim = 66
    assert call(r=C.byref(bad)) == -3


def _paged(**kw):
    c = B.Paged()
    for k, v in dict(pool=256, dtype=1, npages=10, page_rows=16, kv_heads=2, head_dim=128, nseq=3, table=256,
                     table_stride=4, lens=256, cu=256, prefix_pages=256, prefix_len=20).items():
        setattr(c, k, kw.get(k, v))
    return c


BAD = [(dict(dtype=2), -1), (dict(head_dim=96), -3), (dict(head_dim=256), -3), (dict(kv_heads=0), -3),
       (dict(page_rows=0), -3), (dict(page_rows=24), -3), (dict(page_rows=8), -3), (dict(npages=-1), -2), (dict(npages=0), -2),
       (dict(npages=1 << 28), -2), (dict(nseq=-1), -2), (dict(table_stride=-1), -2), (dict(prefix_len=-1), -2),
       (dict(lens=None), -1), (dict(cu=None), -1), (dict(table=None), -1), (dict(pool=None), -1),
       (dict(prefix_pages=None), -1), (dict(pool=264), -1)]


@pytest.mark.parametrize("kw,code", BAD)
def test_paged_descriptor_refusals(kw, code):
    lib = q.load()
    c = C.byref(_paged(**kw))
    assert lib.qi21_op_kv_append(c, 4, 256, 256, 256, 256, None, None, None) == code
    assert lib.qi21_op_attention_paged(c, 4, 4, 256, 512, 256, 512, 1, None, 0.1, 256, 1 << 40, None) == code
    if not any(kw.get(k, 1) is None or k == "pool" for k in kw):
        assert lib.qi21_attention_paged_bytes(c, 4, 4) == 0


def test_append_refusals():
    lib = q.load()
    c = _paged()
    call = lambda kv=C.byref(c), rows=4, k=256, ldk=256, v=256, ldv=256, rope=None, pos=None: \
        lib.qi21_op_kv_append(kv, rows, k, ldk, v, ldv, rope, pos, None)  # noqa: E731
    assert call(rows=0, k=None, v=None) == 0
    assert call(kv=C.byref(_paged(nseq=0, table=None, lens=None, cu=None))) == 0
    assert call(kv=None) == -1 and call(rows=-2) == -2 and call(ldk=255) == -2 and call(ldv=100) == -2
    assert call(k=None) == -1 and call(v=None) == -1 and call(k=257) == -1
    assert call(rope=C.byref(q.rope(64))) == -2             # another head width
    assert call(rope=C.byref(q.rope(128, axes=(16, 56, 56)))) == -1  # three axes without positions
    assert call(rope=C.byref(q.rope(128)), pos=4) == -1     # positions out of line


def test_attention_refusals():
    lib = q.load()
    c = _paged()
    call = lambda kv=C.byref(c), rows=4, heads=4, qq=256, ldq=512, out=256, ldo=512, vis=None, scale=0.1, ws=256, \
        n=1 << 40: lib.qi21_op_attention_paged(kv, rows, heads, qq, ldq, out, ldo, 1, vis, scale, ws, n, None)  # noqa: E731,E501
    assert call(rows=0, qq=None, out=None, ws=None, n=0) == 0
    assert call(kv=None) == -1 and call(rows=-1) == -2 and call(rows=(1 << 24) + 1) == -2
    assert call(heads=3) == -2 and call(heads=0) == -2 and call(heads=2048) == -2
    assert call(ldq=511) == -2 and call(ldq=516) == -2 and call(ldo=504) == -2
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == -1
    assert call(qq=None) == -1 and call(out=None) == -1 and call(qq=264) == -1 and call(out=258) == -1
    assert call(vis=6) == -1
    need = lib.qi21_attention_paged_bytes(C.byref(c), 4, 4)
    assert need > 0
    assert call(ws=None) == -8 and call(ws=128) == -8 and call(n=need - 1) == -8
    assert b"workspace" in lib.qi21_last_error()


def test_workspace_covers_fewer_rows():
    lib = q.load()
    for kw in (dict(), dict(prefix_len=1 << 20, table_stride=1 << 16), dict(head_dim=64, prefix_len=0)):
        c = C.byref(_paged(**kw))
        sizes = [lib.qi21_attention_paged_bytes(c, n, 8) for n in (0, 1, 2, 7, 16, 17, 100, 1000, 1025, 5000)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_limits_of_lengths_and_scale():
    lib = q.load()
    c = C.byref(_paged(prefix_len=1 << 30))  # with the own rows 2^31 keys
    assert lib.qi21_op_attention_paged(c, 4, 4, 256, 512, 256, 512, 1, None, 0.1, 256, 1 << 40, None) == -2
    c = C.byref(_paged())
    assert lib.qi21_op_attention_paged(c, 4, 4, 256, 512, 256, 512, 1, None, 2e38, 256, 1 << 40, None) == -1
