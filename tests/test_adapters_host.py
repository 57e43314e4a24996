"""The adapters' host side: what a packed plan holds, and the argument checks of svdq_lora_plan_pack and
svdq_lora_add (no kernel runs here)."""

import ctypes

import numpy as np
import pytest
import torch

import bit_diffusion_transformer_act_b200 as P

L = P.LIB
FAKE = ctypes.c_void_p(1 << 20)


def _decode(plan):
    """(tiles, copy tiles, groups) of a plan packed for the CPU, following the layout in lora_plan.h."""
    w = plan.words.view(torch.int32).numpy()
    s = plan.struct
    assert bytes(w[:2].tobytes()) == b"SVDQLORA"
    assert list(w[2:10]) == [s.M, s.requests, s.slots, s.adapters, s.tiles, s.copy_tiles, s.groups, s.copy_groups]
    tw, gw = (4 + 2 * s.slots + 3) // 4 * 4, 28 + 16 * s.slots
    nt, ng = s.tiles + s.copy_tiles, s.groups + s.copy_groups
    tiles = w[16:16 + tw * nt].reshape(-1, tw)
    groups = w[16 + tw * nt:16 + tw * nt + gw * ng].reshape(-1, gw)
    assert (16 + tw * nt + gw * ng) * 4 == s.bytes == plan.words.numel()
    return tiles[:s.tiles], tiles[s.tiles:], groups[:s.groups], groups[s.groups:]


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("slots", [1, 3, 8])
def test_a_plan_covers_every_row_once(seed, slots):
    r = np.random.default_rng(seed)
    n = int(r.integers(0, 40))
    lens = r.choice([0, 1, 1, 2, 15, 16, 17, 33, 127, 128, 129, 300], size=n)
    off = int(r.integers(0, 5)) + np.concatenate([[0], np.cumsum(lens)])
    M = int(off[-1] + r.integers(0, 140))
    ids = r.integers(-1, 3, size=(n, slots))
    w = r.standard_normal((n, slots)).astype(np.float32)
    plan = P.LoraPlan(off, ids, w, M, 3, device="cpu")
    tiles, copies, groups, copy_groups = _decode(plan)
    owner = np.full(M, -1)
    for s in range(n):
        owner[off[s]:off[s + 1]] = s
    seen = np.zeros(M, int)
    for t in tiles:
        row, rows, s = t[:3]
        assert 1 <= rows <= 128 and (owner[row:row + rows] == s).all() and (ids[s] >= 0).any()
        assert np.array_equal(t[4:4 + slots], ids[s]) and np.array_equal(t[4 + slots:4 + 2 * slots].view(np.float32), w[s])
        seen[row:row + rows] += 1
    untouched = [m for m in range(M) if owner[m] < 0 or (ids[owner[m]] < 0).all()]
    for t in copies:
        row, rows, s = t[:3]
        assert 1 <= rows <= 128 and s == -1 and (t[4:4 + slots] == -1).all()
        assert set(range(row, row + rows)) <= set(untouched)
        seen[row:row + rows] += 1
    for g in groups:
        assert 1 <= g[0] <= 16
        for i in range(g[0]):
            s = owner[g[12 + i]]
            assert np.array_equal(g[4:4 + slots], ids[s]) and (ids[s] >= 0).any()
            assert np.array_equal(g[28 + i * slots:28 + (i + 1) * slots].view(np.float32), w[s])
            seen[g[12 + i]] += 1
    for g in copy_groups:
        assert 1 <= g[0] <= 16 and (g[4:12] == -1).all()
        assert set(g[12:12 + g[0]]) <= set(untouched)
        seen[g[12:12 + g[0]]] += 1
    assert (seen == 1).all()


def test_rows_of_requests_with_the_same_adapters_share_groups():
    plan = P.LoraPlan(list(range(65)), np.arange(64) % 4, np.ones(64), 64, 4, device="cpu")
    assert plan.struct.groups == 4 and plan.struct.tiles == 0
    groups = _decode(plan)[2]
    assert [list(g[12:28]) for g in groups] == [list(range(a, 64, 4)) for a in range(4)]


def _pack(off, ids, w, slots=1, M=10, adapters=2, room=None):
    n = len(off) - 1
    off, ids, w = np.array(off, np.int32), np.array(ids, np.int32), np.array(w, np.float32)
    room = int(L.svdq_lora_plan_bytes(M, n, slots)) if room is None else room
    out = np.zeros(max(room, 16), np.uint8)
    s = P.ops.LoraPlanStruct()
    return L.svdq_lora_plan_pack(off.ctypes.data, ids.ctypes.data, w.ctypes.data, n, slots, M, adapters,
                                 out.ctypes.data, room, ctypes.byref(s)), s


def test_plan_refusals():
    assert _pack([0, 4, 10], [0, 1], [1, 1])[0] == 0
    assert _pack([0, 4, 3], [0, 1], [1, 1])[0] == 1                   # decreasing
    assert _pack([-1, 4, 5], [0, 1], [1, 1])[0] == 1                  # before the first row
    assert _pack([0, 4, 11], [0, 1], [1, 1])[0] == 1                  # past the last
    assert _pack([0, 4, 10], [0, 2], [1, 1])[0] == 1                  # no such adapter
    assert _pack([0, 4, 10], [0, -2], [1, 1])[0] == 1
    assert _pack([0, 4, 10], [0, 1], [1, np.inf])[0] == 1
    assert _pack([0, 4, 10], [0, 1], [np.nan, 1])[0] == 1
    assert _pack([0, 4, 10], [0, 1], [1, 1], room=32)[0] == 1         # short buffer
    assert _pack([0, 4, 10], [0, 1], [1, 1], adapters=-1)[0] == 1
    assert L.svdq_lora_plan_bytes(-1, 1, 1) == 0
    assert L.svdq_lora_plan_bytes(1, -1, 1) == 0
    assert L.svdq_lora_plan_bytes(1, 1, 0) == 0
    assert L.svdq_lora_plan_bytes(1, 1, 9) == 0
    assert L.svdq_lora_plan_bytes(0, 0, 1) > 0
    with pytest.raises(ValueError, match="row_offsets"):
        P.LoraPlan([0, 1], [0, 1], [1, 1], 4, 2, device="cpu")
    with pytest.raises(ValueError, match="32-bit"):
        P.LoraPlan(np.array([0, 2 ** 32 + 1]), [0], [1.0], 4, 2, device="cpu")
    with pytest.raises(P.SvdqError):
        P.LoraPlan([0, 5], [0], [1.0], 4, 2, device="cpu")


def _add(s, X=FAKE, ldx=64, Yin=FAKE, ldyin=128, A=FAKE, B=FAKE, dev=FAKE, pbytes=None, M=10, N=128, K=64, rank=16,
         ws=FAKE, wsb=1 << 30, Y=FAKE, ldy=128):
    return L.svdq_lora_add(X, ldx, Yin, ldyin, A, B, ctypes.byref(s) if s else None, dev,
                           s.bytes if pbytes is None and s else pbytes or 0, M, N, K, rank, ws, wsb, Y, ldy, None)


def test_lora_add_refusals():
    s = _pack([0, 4, 10], [0, 1], [1, 1])[1]
    far = ctypes.c_void_p(1 << 24)                                    # X away from Y
    assert _add(None) == 1
    assert _add(s, X=far, M=11) == 1                                  # another batch's plan
    assert _add(s, X=far, M=-1) == 1
    assert _add(s, X=far, N=0) == 1
    assert _add(s, X=far, N=96) == 2
    assert _add(s, X=far, K=96) == 2
    assert _add(s, X=far, rank=24) == 2
    assert _add(s, X=far, rank=144) == 2
    for name in ("X", "Yin", "A", "B", "dev", "ws", "Y"):
        kw = {"X": far}
        kw[name] = None
        assert _add(s, **kw) == 1, name
        kw[name] = ctypes.c_void_p((1 << 24) + 8)
        assert _add(s, **kw) == 1, name                               # misaligned
    assert _add(s, X=far, ldx=56) == 1                                # rows that overlap
    assert _add(s, X=far, ldx=68) == 1                                # rows that are not 16-byte aligned
    assert _add(s, X=far, ldyin=120) == 1
    assert _add(s, X=far, ldy=132) == 1
    assert _add(s, X=far, pbytes=s.bytes - 4) == 1
    # X inside Y's rows; Y that overlaps Yin without being it
    assert _add(s, X=FAKE) == 1
    assert _add(s, X=far, Y=ctypes.c_void_p((1 << 20) + 256)) == 1
    assert _add(s, X=far, ldy=256) == 1
    broken = P.ops.LoraPlanStruct(*[getattr(s, n) for n, _ in s._fields_])
    broken.groups += 1
    assert _add(broken, X=far) == 1
    two = _pack([0, 4, 10], [[0, 1], [1, 0]], [[1, 1], [1, 1]], slots=2)[1]
    assert _add(two, X=far, rank=80) == 2                             # slots * rank
    empty = _pack([0], [], [], M=0)[1]
    assert _add(empty, X=None, Yin=None, Y=None, A=None, B=None, dev=None, ws=None, wsb=0, M=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device_report_a_cuda_error():
    s = _pack([0, 4, 10], [0, 1], [1, 1])[1]
    far = ctypes.c_void_p(1 << 24)
    assert _add(s, X=far) == 4
    # a column window into another window of the same rows does not overlap it
    assert _add(s, X=far, ldyin=256, ldy=256, Y=ctypes.c_void_p((1 << 20) + 256)) == 4


def test_a_batch_without_requests():
    plan = P.LoraPlan([0], [], [], 5, 3, device="cpu")
    assert (plan.requests, plan.slots, plan.struct.tiles, plan.struct.groups) == (0, 1, 0, 0)
    assert plan.sizes()[:4] == P.LoraPlan([0], np.zeros((0, 1), np.int32), np.zeros((0, 1)), 5, 3, device="cpu").sizes()[:4]
    with pytest.raises(ValueError, match="row_offsets"):
        P.LoraPlan([0, 4], [0], [1.0, 1.0], 4, 2, device="cpu")


def test_python_wrapper_refuses_before_the_call():
    plan = P.LoraPlan([0, 4], [0], [1.0], 4, 2, device="cpu")
    bf = torch.bfloat16
    x, y = torch.zeros((4, 64), dtype=bf), torch.zeros((4, 128), dtype=bf)
    a, b = torch.zeros((2, 16, 64), dtype=bf), torch.zeros((2, 128, 16), dtype=bf)
    with pytest.raises(ValueError, match="CUDA tensor"):
        P.svdq_lora_add(x, y, a, b, plan)
    with pytest.raises(ValueError, match="the plan is for 4 rows"):
        P.svdq_lora_add(x[:3], y[:3], a, b, plan)
    with pytest.raises(ValueError, match="2 adapters"):
        P.svdq_lora_add(x, y, a[:1], b[:1], plan)
    with pytest.raises(ValueError, match="bfloat16"):
        P.svdq_lora_add(x.float(), y, a, b, plan)
    with pytest.raises(ValueError, match="contiguous"):
        P.svdq_lora_add(torch.zeros((64, 4), dtype=bf).t(), y, a, b, plan)
    with pytest.raises(ValueError, match="LoraPlan"):
        P.svdq_lora_add(x, y, a, b, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_a_single_row_is_in_place_whatever_its_strides():
    s = _pack([0, 1], [0], [1], M=1)[1]
    assert _add(s, X=ctypes.c_void_p(1 << 24), M=1, ldy=256) == 4


def test_pools_whose_rows_pass_32_bits_are_refused():
    far = ctypes.c_void_p(1 << 24)
    s = _pack([0, 4, 10], [0, 1], [1, 1], adapters=1 << 24)[1]
    assert _add(s, X=far, rank=128, N=64, ldyin=64, ldy=64) == 2        # rows of A
    assert _add(s, X=far, N=128) == 2                                   # rows of B
