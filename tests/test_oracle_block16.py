"""The operators around the linears of an attention block, without a GPU: the
oracles against the formulas, and what the library and its wrappers refuse."""
import ctypes
import math

import numpy as np
import pytest
import torch

import w4a4_rank_corrected_smooth_amd as S
from oracle import rotary

INV, SHAPE, NODEV, WS = 1, 2, 3, 5
FAKE = 1 << 20            # an aligned address that no refused call reads
I64 = ctypes.c_int64


# ------------------------------------------------------------------ rotary
def test_rotary_oracle_is_a_rotation():
    """Each pair as a complex number times e^{i angle}; scores depend on differences of positions only."""
    r = np.random.default_rng(1)
    freq, axis = rotary.ladder([4, 6], 100.0, True)
    assert np.allclose(freq, [1, 0.1, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)]) and axis.tolist() == [0, 0, 1, 1, 1]
    x, pos = r.standard_normal((3, 2, 12)), r.integers(0, 9, (3, 2))
    for inter in (True, False):
        y = rotary.turn(x, pos, freq, axis, inter)
        j = np.arange(5)
        i0, i1 = (2 * j, 2 * j + 1) if inter else (j, j + 5)
        z = (x[..., i0] + 1j * x[..., i1]) * np.exp(1j * pos[:, axis] * freq)[:, None]
        assert np.allclose(y[..., i0], z.real) and np.allclose(y[..., i1], z.imag) and np.array_equal(y[..., 10:], x[..., 10:])
    q, k = r.standard_normal((2, 1, 1, 12))
    a = (rotary.turn(q, [[5, 2]], freq, axis, True) * rotary.turn(k, [[3, 1]], freq, axis, True)).sum()
    b = (rotary.turn(q, [[105, 22]], freq, axis, True) * rotary.turn(k, [[103, 21]], freq, axis, True)).sum()
    assert math.isclose(a, b, rel_tol=1e-12, abs_tol=1e-12)


@pytest.mark.parametrize("per_axis", [True, False])
def test_rotary_plan_holds_the_ladder(per_axis):
    widths = [16, 56, 40]
    plan = S.RotaryPlan(128, widths, theta=500.0, interleaved=False, per_axis=per_axis)
    freq, axis = rotary.ladder(widths, 500.0, per_axis)
    assert plan.pairs == 56 and plan.axes == 3 and plan._c.interleaved == 0
    assert np.allclose(plan._c.freq[:56], freq, rtol=1e-15, atol=0) and list(plan._c.axis[:56]) == axis.tolist()
    again = S.RotaryPlan.from_tables(128, freq, axis, interleaved=False)
    assert list(again._c.freq) == pytest.approx(list(plan._c.freq), rel=1e-15) and bytes(again._c.axis) == bytes(plan._c.axis)


def test_rotary_plan_refusals():
    for bad in ((12, [4]), (264, [8]), (0, [2]), (64, []), (64, [3]), (64, [0]), (64, [-2]), (64, [40, 26]), (64, [2] * 9)):
        with pytest.raises(S.SvdqError):
            S.RotaryPlan(*bad)
    for theta in (0.0, -1.0, math.inf, math.nan, 1e-320):
        with pytest.raises(S.SvdqError):
            S.RotaryPlan(64, [64], theta=theta)
    with pytest.raises(ValueError, match="32-bit"):
        S.RotaryPlan(64 + (1 << 32), [64])
    for bad in (dict(freq=[1.0] * 33, axis=[0] * 33), dict(freq=[1.0], axis=[0, 0]), dict(freq=[], axis=[]),
                dict(freq=[math.nan], axis=[0]), dict(freq=[1.0], axis=[8]), dict(freq=[1.0], axis=[-1])):
        with pytest.raises(ValueError):
            S.RotaryPlan.from_tables(64, **bad)
    assert S._lib.svdq_rotary_plan(64, None, 1, 1e4, 1, 1, ctypes.byref(S.RotaryStruct())) == INV


def test_rotary_argument_errors():
    plan = S.RotaryPlan(64, [32, 32])

    def go(p=plan._c, q=FAKE, qs=(128, 64), qh=2, qo=FAKE, qos=(128, 64), k=FAKE, kh=2, ko=FAKE, dt=S.BF16, pos=FAKE, T=4):
        return S._lib.svdq_rotary_apply(ctypes.byref(p) if p else None, q, *qs, qh, qo, *qos, k, 128, 64, kh, ko, 128, 64,
                                        dt, pos, 0, T, None)
    assert go(p=None) == INV and go(q=0) == INV and go(qo=0) == INV and go(k=0) == INV and go(ko=0) == INV and go(pos=0) == INV
    assert go(q=FAKE + 8) == INV and go(qo=FAKE + 2) == INV and go(pos=FAKE + 2) == INV and go(qs=(129, 64)) == INV
    assert go(qs=(128, -64)) == INV and go(qos=(128, 4)) == INV and go(dt=S.FP32) == INV
    assert go(T=-1) == SHAPE and go(qh=-1) == SHAPE and go(kh=65535) == SHAPE and go(T=1 << 30) == SHAPE
    assert go(T=0, q=0, pos=0) == 0 and go(qh=0, kh=0, q=0, k=0) == 0
    for field, value in (("head_dim", 60), ("head_dim", 512), ("pairs", 0), ("pairs", 33), ("axes", 0), ("axes", 9)):
        p = S.RotaryStruct.from_buffer_copy(plan._c)
        setattr(p, field, value)
        assert go(p=p) == SHAPE, field
    p = S.RotaryStruct.from_buffer_copy(plan._c)
    p.axis[3] = 2
    assert go(p=p) == INV
    p = S.RotaryStruct.from_buffer_copy(plan._c)
    p.freq[31] = math.inf
    assert go(p=p) == INV
    if not torch.cuda.is_available():
        assert go() == NODEV


def test_rotary_wrapper_checks():
    plan = S.RotaryPlan(64, [32, 32])
    q, pos = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, dtype=torch.int32)
    for bad in (dict(q=q[..., :32]), dict(q=q.float()), dict(k=q[:4]), dict(k=q.half()), dict(k=q[..., ::2]), dict(positions=pos[:4]),
                dict(positions=pos[:, :1]), dict(positions=pos.long()), dict(positions=pos.t().contiguous().t()),
                dict(q_out=q[:, :2]), dict(q_out=q.half()), dict(k_out=q), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            S.rotary_apply(**{**dict(plan=plan, q=q, k=None, positions=pos), **bad})
    with pytest.raises(TypeError):
        S.rotary_apply(plan, [1], None, pos)
    with pytest.raises(TypeError):
        S.rotary_apply(plan, q, [1], pos)
    with pytest.raises(ValueError, match="not on cpu"):
        S.rotary_apply(plan, q, q, pos)
    big = torch.empty((1 << 32) + 1, 1, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="32-bit"):
        S.rotary_apply(plan, big, None, torch.empty((1 << 32) + 1, 2, dtype=torch.int32, device="meta"))


# --------------------------------------------------------- cross attention
def test_cross_oracle_is_a_softmax():
    from oracle import cross
    r = np.random.default_rng(2)
    q, k, v = r.standard_normal((2, 3, 4, 8)), r.standard_normal((2, 5, 2, 8)), r.standard_normal((2, 5, 2, 8))
    seen = np.array([[1, 0, 1, 1, 0], [0, 0, 0, 0, 0]], bool)
    out, mean, size = cross.attend(q, k, v, seen, 0.5)
    for i in range(3):
        for h in range(4):
            e = [math.exp(0.5 * (q[0, i, h] * k[0, t, h // 2]).sum()) for t in (0, 2, 3)]
            want = sum(x * v[0, t, h // 2] for x, t in zip(e, (0, 2, 3))) / sum(e)
            assert np.allclose(out[0, i, h], want) and (mean[0, i, h] >= abs(want) - 1e-12).all()
            assert size[0, i, h, 0] == pytest.approx(max(0.5 * np.abs(q[0, i, h] * k[0, t, h // 2]).sum() for t in (0, 2, 3)))
    assert not out[1].any()


def test_cross_workspace_and_shapes():
    f = S._lib.svdq_cross_attention_workspace_bytes
    assert f(1, 4096, 512, 16, 16, 128, 0) >= 1 and f(2, 4096, 300, 16, 16, 72, 1) >= 4 * 2 * 300
    assert f(8, 1, 1500, 20, 20, 64, 0) > 0 and f(0, 0, 0, 1, 1, 8, 0) >= 1
    for bad in ((-1, 1, 1, 1, 1, 64), (65537, 1, 1, 1, 1, 64), (1, -1, 1, 1, 1, 64), (1, 1, -1, 1, 1, 64), (1, 1, (1 << 30) + 1, 1, 1, 64),
                (1, 1, 1, 0, 1, 64), (1, 1, 1, 1, 0, 64), (1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 0), (1, 1, 1, 1, 1, 60),
                (1, 1, 1, 1, 1, 264), (2, 1 << 27, 1, 2, 1, 64), (65536, 1, 1, 17, 17, 64), (1, 2 ** 31 - 1, 1, 2 ** 31 - 1, 1, 64)):
        assert f(*bad, 0) == 0, bad


def test_cross_argument_errors():
    need = S._lib.svdq_cross_attention_workspace_bytes(2, 4, 50, 4, 2, 64, 1)
    row = dict(q=(FAKE, 1024, 256, 64), k=(FAKE, 8192, 128, 64), v=(FAKE, 8192, 128, 64))

    def go(dt=S.BF16, B=2, Lq=4, Lk=50, Hq=4, Hkv=2, D=64, lens=None, mask=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=need, **kw):
        r = {**row, **kw}
        return S._lib.svdq_cross_attention(*r["q"], *r["k"], *r["v"], dt, B, Lq, Lk, Hq, Hkv, D, lens, mask, scale, out, ws, n, None)
    for name in "qkv":
        p, b, t, h = row[name]
        assert go(**{name: (0, b, t, h)}) == INV and go(**{name: (p + 8, b, t, h)}) == INV
        for bad in ((p, b + 4, t, h), (p, b, -t, h), (p, b, t, 4)):
            assert go(**{name: bad}) == INV
    assert go(k=(FAKE, 0, 1 << 24, 64)) == SHAPE and go(v=(FAKE, 0, 1 << 24, 64)) == SHAPE
    assert go(dt=S.FP32) == INV and go(out=0) == INV and go(out=FAKE + 2) == INV and go(ws=0) == INV and go(ws=FAKE + 8) == INV
    assert go(lens=FAKE + 2) == INV and go(n=need - 1) == WS and go(D=68) == SHAPE and go(Hq=3) == SHAPE and go(B=-1) == SHAPE
    for scale in (math.inf, -math.inf, math.nan, 2.0 ** 127):
        assert go(scale=scale) == INV
    assert go(B=0, q=(0, 0, 0, 0)) == 0 and go(Lq=0, out=0) == 0
    if not torch.cuda.is_available():
        assert go() == NODEV and go(Lk=0, k=(0, 0, 0, 0), v=(0, 0, 0, 0)) == NODEV


def test_cross_wrapper_checks():
    bf = torch.bfloat16
    q, k = torch.zeros(2, 3, 4, 64, dtype=bf), torch.zeros(2, 7, 2, 64, dtype=bf)
    lens, mask = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 7, dtype=torch.bool)
    good = dict(q=q, k=k, v=k)
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=k.half()), dict(k=k[:1]), dict(v=k[:, :6]), dict(k=k[..., :32]),
                dict(q=q[0]), dict(key_lens=lens.long()), dict(key_lens=lens[:1]), dict(mask=mask.byte()), dict(mask=mask[:, :6]),
                dict(mask=mask.t().contiguous().t()), dict(out=q.half()), dict(out=q[:, :2]), dict(workspace=torch.zeros(9)),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(v=k.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            S.cross_attention(**{**good, **bad})
    for bad in (dict(q=1), dict(k=None), dict(v=[1]), dict(mask=[1]), dict(key_lens=[1, 2])):
        with pytest.raises(TypeError):
            S.cross_attention(**{**good, **bad})
    with pytest.raises(S.SvdqError):
        S.cross_attention(q[:, :, :3], k, k)               # 3 heads over 2
    with pytest.raises(ValueError, match="not on cpu"):
        S.cross_attention(q, k, k)
    big = torch.empty(1, (1 << 32) + 1, 1, 64, dtype=bf, device="meta")
    with pytest.raises(ValueError, match="32-bit"):
        S.cross_attention(big, big[:, :1], big[:, :1])
    with pytest.raises(ValueError, match="32-bit"):
        S.cross_attention(big[:, :1], big, big)
    with pytest.raises(ValueError, match="32-bit"):
        S.cross_attention_workspace(big[:, :1], big)
