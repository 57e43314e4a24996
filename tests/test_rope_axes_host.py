"""The argument checks of svdq_qk_norm_rope and svdq_rope_axes_tables (no kernel runs here), and the
oracle's rotation against the single-axis one."""

import ctypes

import numpy as np
import pytest
import torch

import bit_diffusion_transformer_act_b200 as P
from oracle import qkv_epilogue, rope_axes

L = P.LIB


def _at(mb, off=0):
    return ctypes.c_void_p((mb << 20) + off)


def _axes(dims, thetas=None):
    n = len(dims)
    return n, (ctypes.c_int32 * n)(*dims), (ctypes.c_double * n)(*(thetas or [10000.0] * n))


def _rope(q=_at(1), qs=(768, 128), nq=2, k=_at(1, 512), ks=(768, 128), nk=2, M=4, D=128, wq=_at(64), wk=_at(65),
          eps=1e-6, pos=_at(66), P_=4, dims=(16, 56, 56), thetas=None, pairing=0, oq=_at(70), oqs=(256, 128), ok=_at(80),
          oks=(256, 128)):
    n, d, t = _axes(dims, thetas)
    return L.svdq_qk_norm_rope(q, qs[0], qs[1], nq, k, ks[0], ks[1], nk, M, D, wq, wk, eps, pos, 0, P_, n, d, t,
                               pairing, oq, oqs[0], oqs[1], ok, oks[0], oks[1], None)


def _tables(pos=_at(1), P_=4, dims=(16, 56, 56), thetas=None, M=4, D=128, cos=_at(2), sin=_at(3)):
    n, d, t = _axes(dims, thetas)
    return L.svdq_rope_axes_tables(pos, 0, P_, n, d, t, M, D, cos, sin, None)


OK = 4                                                 # past the checks: no device here

needs_no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


@needs_no_device
def test_valid_calls_reach_the_device():
    assert _rope() == OK
    assert _rope(wq=None, wk=None, eps=float("nan")) == OK
    assert _rope(q=None, nq=0, oq=None) == OK
    assert _rope(k=None, nk=0, ok=None) == OK
    # in place on the packed projection; head-major outputs
    assert _rope(oq=_at(1), oqs=(768, 128), ok=_at(1, 512), oks=(768, 128)) == OK
    assert _rope(oqs=(128, 512), oks=(128, 512)) == OK
    # into the thirds of another packed buffer
    assert _rope(oq=_at(70), oqs=(768, 128), ok=_at(70, 512), oks=(768, 128)) == OK
    assert _tables() == OK
    assert _tables(pos=_at(1, 4)) == OK                 # a slice of a longer list of positions
    assert _rope(pos=_at(66, 12)) == OK


def test_empty_calls():
    assert _rope(M=0, q=None, k=None, oq=None, ok=None, pos=None) == 0
    assert _rope(q=None, nq=0, k=None, nk=0, oq=None, ok=None) == 0
    assert _tables(M=0, pos=None, cos=None, sin=None) == 0


def test_refusals_of_both():
    for call in (_rope, _tables):
        assert call(M=-1) == 1
        assert call(D=0) == 1
        assert call(D=264) == 2
        assert call(dims=(16, 56, 0)) == 1
        assert call(dims=(16, 57, 55)) == 2
        assert call(dims=(16, 56, 64)) == 2            # past the head
        assert call(dims=(2, 4, 4)) == 2               # 10 rotated columns
        assert call(dims=(8,) * 9) == 2
        assert call(thetas=[10000.0, 0.0, 1.0]) == 1
        assert call(thetas=[10000.0, float("inf"), 1.0]) == 1
        assert call(thetas=[10000.0, float("nan"), 1.0]) == 1
        assert call(P_=3) == 1
        assert call(P_=0) == 1
        assert call(pos=None) == 1
        assert call(pos=_at(1, 2)) == 1
    assert _tables(cos=None) == 1
    assert _tables(sin=_at(1, 8)) == 1
    assert _tables(D=127, dims=(16, 56, 48)) == 2


def test_refusals_of_the_rotation():
    assert _rope(nq=-1) == 1
    assert _rope(pairing=2) == 1
    assert _rope(eps=-1.0) == 1
    assert _rope(eps=float("nan")) == 1
    assert _rope(D=124, dims=(16, 56, 48)) == 2
    assert _rope(wq=_at(1, 8)) == 1
    for name in ("q", "k", "oq", "ok"):
        assert _rope(**{name: None}) == 1
        assert _rope(**{name: _at(30, 8)}) == 1
    assert _rope(qs=(764, 128)) == 1                   # rows that are not 16-byte aligned
    assert _rope(qs=(-768, 128)) == 1
    assert _rope(oqs=(128, 128)) == 1                  # outputs whose heads fall on other rows
    assert _rope(oqs=(256, 64)) == 1
    assert _rope(oqs=(0, 128)) == 1
    # outputs on an input or on one another
    assert _rope(oq=_at(1), oqs=(256, 128)) == 1       # q's place with other strides
    assert _rope(oq=_at(1, 512), oqs=(768, 128)) == 1  # k's place
    assert _rope(oq=_at(1, 256), oqs=(768, 128)) == 1  # half of each
    assert _rope(ok=_at(70)) == 1
    assert _rope(ok=_at(1), oks=(768, 128)) == 1


def test_python_wrappers_refuse_before_the_call():
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    pos = torch.zeros((4, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        P.svdq_qk_norm_rope(q, None, None, None, 0.0, pos, [16, 56, 56], 10000.0)
    with pytest.raises(ValueError, match="int32 or float32"):
        P.svdq_rope_axes_tables(pos.long(), [16, 56, 56], 10000.0, 128)
    with pytest.raises(ValueError, match="q or k"):
        P.svdq_qk_norm_rope(None, None, None, None, 0.0, pos, [16, 56, 56], 10000.0)
    with pytest.raises(ValueError, match="int32 or float32"):
        P.svdq_rope_axes_tables(pos[:, :2], [16, 56], 10000.0, 128)


def test_oracle_is_the_single_axis_oracle_on_one_axis():
    r = np.random.default_rng(0)
    x, w = r.standard_normal((6, 2, 16)), r.standard_normal(16)
    ang = rope_axes.angles(np.arange(6)[:, None], [16], [100.0])
    assert np.allclose(ang[3], 3 * 100.0 ** (-np.arange(8) / 8))
    got = rope_axes.rotate(rope_axes.norm(x, w, 1e-6), ang, half=False)
    assert np.allclose(got, qkv_epilogue.rope(qkv_epilogue.rmsnorm_heads(x, w, 1e-6), np.cos(ang), np.sin(ang)))
    # halves: the same rotation after sorting even before odd columns
    order = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    assert np.allclose(rope_axes.rotate(x[..., order], ang, half=True), rope_axes.rotate(x, ang, half=False)[..., order])


def _elements(base, strides, heads, M, D):
    at = base + strides[0] * np.arange(M)[:, None] + strides[1] * np.arange(heads)
    return set((at[..., None] + np.arange(D)).ravel().tolist())


@needs_no_device
def test_heads_of_q_and_k_side_by_side_in_place():
    """[M, heads, 3, D]: the rows of q and k interlace, which was refused although no element is shared."""
    s = (2 * 384, 384)
    assert _rope(q=_at(1), qs=s, k=_at(1, 256), ks=s, oq=_at(1), oqs=s, ok=_at(1, 256), oks=s) == OK
    one = (5 * 128, 2 * 128)                           # one k head between two of q's
    assert _rope(q=_at(1), qs=one, k=_at(1, 256), ks=(640, 8), nk=1, oq=_at(1), oqs=one, ok=_at(1, 256), oks=(640, 8)) == OK
    assert _rope(q=_at(1), qs=one, k=_at(1, 512), ks=(640, 8), nk=1, oq=_at(1), oqs=one, ok=_at(1, 512), oks=(640, 8)) == 1
    assert _rope(q=_at(1), qs=s, k=_at(1, 240), ks=s, oq=_at(1), oqs=s, ok=_at(1, 240), oks=s) == 1


@needs_no_device
@pytest.mark.parametrize("seed", range(6))
def test_overlaps_of_equal_strides_are_found_exactly(seed):
    r = np.random.default_rng(seed)
    answers = []
    for _ in range(400):
        M, nq, nk, D = int(r.integers(1, 5)), int(r.integers(1, 5)), int(r.integers(1, 5)), 8 * int(r.integers(1, 4))
        head = D + 8 * int(r.integers(0, 6))
        row = (max(nq, nk) - 1) * head + D + 8 * int(r.integers(0, 8))
        if r.random() < 0.3:                           # head-major
            row, head = D + 8 * int(r.integers(0, 4)), 0
            head = (M - 1) * row + D + 8 * int(r.integers(0, 4))
        q0 = 1 << 19
        k0 = q0 + 8 * int(r.integers(-40, 40))
        apart = not _elements(q0, (row, head), nq, M, D) & _elements(k0, (row, head), nk, M, D)
        q, k = ctypes.c_void_p(2 * q0), ctypes.c_void_p(2 * k0)
        st = _rope(q=q, qs=(row, head), nq=nq, k=k, ks=(row, head), nk=nk, M=M, D=D, P_=M, dims=(8,), oq=q,
                   oqs=(row, head), ok=k, oks=(row, head))
        if not apart:
            assert st == 1
        answers.append((apart, st == OK))
    wrong = [a for a in answers if a[0] != a[1]]
    assert not wrong, len(wrong)
    assert len(set(answers)) == 2
