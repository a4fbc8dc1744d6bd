"""Rotary positions on the GPU against the float64 oracle.

Tolerance of a value y = a cos - b sin (or a sin + b cos): its rounding to the
16-bit type, eps / 2 |y| (2^-25 at least for float16's subnormals), and the float32
steps before it: a sine or cosine is off by at most 2^-23 (its argument's rounding
2^-24 pi / 4, the series' steps below 2^-24 of 1, the series' rest 2^-28), a product and the
sum round three times by 2^-24; together below 2^-21 (|a| + |b|)."""
import numpy as np
import pytest
import torch

from oracle import rotary as O
from tests.conftest import announce

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def S():
    import w4a4_rank_corrected_smooth_amd as lib
    lib.device_check()
    return lib


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(r, shape, dtype):
    x = r.standard_normal(shape)
    x[..., ::29] *= 9.0
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def near(got, x, positions, freq, axis, interleaved):
    x = f64(x)
    want = O.turn(x, positions, freq, axis, interleaved)
    n = len(freq)
    i, j = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    size = np.zeros_like(want)
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    eps = torch.finfo(got.dtype).eps
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    off = np.abs(f64(got) - want)
    assert (off <= eps / 2 * np.abs(want) * (1 + 2.0 ** -10) + tiny + 2.0 ** -21 * size).all(), off.max()
    assert np.array_equal(f64(got)[..., 2 * n:], x[..., 2 * n:])


CASES = [  # T, Hq, Hk, D, widths, per_axis, interleaved, far
    (1, 1, 1, 8, [2], True, True, 0),
    (1, 32, 8, 128, [32, 48, 48], False, False, 10 ** 6),
    (5, 3, 1, 64, [64], True, False, 2 ** 31 - 200),
    (67, 24, 24, 128, [16, 56, 56], True, True, 100),
    (129, 2, 2, 128, [44, 42, 42], True, True, 5000),
    (33, 4, 2, 72, [24, 24, 24], True, False, 50),          # halves of 36: pieces of four
    (31, 2, 1, 80, [20], False, False, 50),                 # halves of 10: single channels, 60 stay
    (17, 5, 0, 256, [64, 192], False, True, 1000),
    (9, 2, 2, 256, [30], True, True, 10),                   # a piece of which only a part turns
    (300, 1, 1, 96, [2, 2, 2, 2, 2, 2, 2, 2], False, False, 3),
    (2, 700, 300, 16, [8], True, False, 9),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,Hq,Hk,D,widths,per_axis,interleaved,far", CASES)
def test_rotary_against_the_oracle(S, T, Hq, Hk, D, widths, per_axis, interleaved, far, dtype):
    announce(f"rotary T={T} Hq={Hq} Hk={Hk} D={D} {widths} per_axis={per_axis} interleaved={interleaved} {dtype}")
    r = np.random.default_rng(T * D + Hq)
    pos = r.integers(-far, far + 1, (T, len(widths)))
    freq, axis = O.ladder(widths, 10000.0, per_axis)
    plan = S.RotaryPlan(D, widths, interleaved=interleaved, per_axis=per_axis)
    q = rows(r, (T, Hq, D), dtype)
    k = rows(r, (T, Hk, D), dtype) if Hk else None
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    qo, ko = S.rotary_apply(plan, q, k, p)
    near(qo, q, pos, freq, axis, interleaved)
    if Hk:
        near(ko, k, pos, freq, axis, interleaved)
    else:
        assert ko is None
    # float positions that hold the same integers give the same bits
    if far < 2 ** 24:
        fo, _ = S.rotary_apply(plan, q, None, p.float())
        assert torch.equal(fo, qo)


def test_rotary_in_place_in_a_fused_projection(S):
    """Queries and keys turned where they are; the values beside them and the rows behind stay."""
    r = np.random.default_rng(5)
    T, Hq, Hk, D = 41, 6, 2, 128
    qkv = rows(r, (T + 3, Hq + 2 * Hk, D), "bf16")
    before = qkv.clone()
    pos = r.integers(0, 1000, (T, 3))
    plan = S.RotaryPlan(D, [16, 56, 56])
    freq, axis = O.ladder([16, 56, 56], 10000.0, True)
    q, k = qkv[:T, :Hq], qkv[:T, Hq:Hq + Hk]
    announce("rotary in place")
    qo, ko = S.rotary_apply(plan, q, k, torch.from_numpy(pos.astype(np.int32)).cuda(), q_out=q, k_out=k)
    assert qo is q and ko is k
    near(q, before[:T, :Hq], pos, freq, axis, True)
    near(k, before[:T, Hq:Hq + Hk], pos, freq, axis, True)
    assert torch.equal(qkv[:T, Hq + Hk:], before[:T, Hq + Hk:]) and torch.equal(qkv[T:], before[T:])


def test_rotary_per_head_layout_and_other_output_strides(S):
    r = np.random.default_rng(6)
    T, H, D = 19, 3, 64
    q = rows(r, (H, T, D), "fp16").permute(1, 0, 2)
    out = torch.full((T, 2 * H, D + 8), 7.0, dtype=torch.float16, device="cuda")
    pos = r.integers(0, 99, (T, 1))
    plan = S.RotaryPlan(D, [32], interleaved=False)
    freq, axis = O.ladder([32], 10000.0, True)
    announce("rotary to strided rows")
    S.rotary_apply(plan, q, None, torch.from_numpy(pos.astype(np.int32)).cuda(), q_out=out[:, ::2, :D])
    near(out[:, ::2, :D], q, pos, freq, axis, False)
    assert (out[:, 1::2] == 7).all() and (out[..., D:] == 7).all()


def test_rotary_fractional_positions_tables_and_back(S):
    """Fractions of a step, axes that take turns, and a turn back by negated positions."""
    r = np.random.default_rng(7)
    T, H, D, n = 50, 4, 128, 60
    freq = 10000.0 ** (-np.arange(n) / n) * np.where(np.arange(n) > 30, 0.25, 1.0)
    axis = np.arange(n) % 3
    plan = S.RotaryPlan.from_tables(D, freq, axis)
    pos = (r.random((T, 3)) * 200).astype(np.float32)
    q = rows(r, (T, H, D), "fp16")
    p = torch.from_numpy(pos).cuda()
    announce("rotary by fractions")
    y, _ = S.rotary_apply(plan, q, None, p)
    near(y, q, pos, freq, axis, True)
    back, _ = S.rotary_apply(plan, y, None, -p)
    near(back, y, -pos, freq, axis, True)
    # two roundings of 2^-11 of a pair's size
    size = f64(q)[..., :2 * n].reshape(T, H, n, 2)
    size = np.abs(size).sum(-1, keepdims=True).repeat(2, -1).reshape(T, H, 2 * n)
    assert (np.abs(f64(back) - f64(q))[..., :2 * n] <= 2.1 * 2.0 ** -10 * size + 2.0 ** -20 * size).all()


def test_rotary_infinities_stay_in_their_pair(S):
    q = torch.ones(2, 1, 16, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 2], q[0, 0, 9], q[1, 0, 15] = float("inf"), float("nan"), -float("inf")
    plan = S.RotaryPlan(16, [8])
    pos = torch.tensor([[1], [2]], dtype=torch.int32, device="cuda")
    announce("rotary of infinities")
    y, _ = S.rotary_apply(plan, q, None, pos)
    bad = ~torch.isfinite(y)
    assert bad[0, 0].tolist() == [False, False, True, True] + 5 * [False] + [True] + 6 * [False]
    assert bad[1, 0].tolist() == 15 * [False] + [True] and y[1, 0, 15] == -float("inf")
    # a position that is no number: the pairs of its axis, and no other row
    y, _ = S.rotary_apply(plan, torch.ones_like(q), None, torch.tensor([[float("nan")], [1.0]], device="cuda"))
    assert torch.isnan(y[0, 0, :8]).all() and torch.isfinite(y[0, 0, 8:]).all() and torch.isfinite(y[1]).all()


def test_rotary_many_tokens_and_empty_calls(S):
    r = np.random.default_rng(8)
    T, H, D = 70001, 2, 64
    q = rows(r, (T, H, D), "bf16")
    pos = r.integers(0, 100000, (T, 2))
    plan = S.RotaryPlan(D, [32, 32])
    freq, axis = O.ladder([32, 32], 10000.0, True)
    announce("rotary of 70001 tokens")
    y, _ = S.rotary_apply(plan, q, None, torch.from_numpy(pos.astype(np.int32)).cuda())
    near(y, q, pos, freq, axis, True)
    y, z = S.rotary_apply(plan, q[:0], q[:0], torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    assert y.shape == z.shape == (0, H, D)


def test_rotary_stream_and_graph(S):
    """On another stream, and captured: each replay turns what the buffers then hold."""
    r = np.random.default_rng(9)
    T, H, D = 37, 4, 128
    plan = S.RotaryPlan(D, [16, 56, 56])
    x = [rows(r, (T, H, D), "bf16") for _ in range(4)]
    p = torch.from_numpy(r.integers(0, 500, (T, 3)).astype(np.int32)).cuda()
    want = [S.rotary_apply(plan, a, None, p)[0] for a in x]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    announce("rotary on a side stream")
    with torch.cuda.stream(s):
        got = S.rotary_apply(plan, x[0], None, p)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want[0])
    buf, out = x[0].clone(), torch.empty_like(x[0])
    torch.cuda.synchronize()
    announce("rotary in a graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.rotary_apply(plan, buf, None, p, q_out=out)
    for a, w in zip(x, want):
        buf.copy_(a)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
