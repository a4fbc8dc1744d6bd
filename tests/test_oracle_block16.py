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
    assert f(1, 4096, 512, 16, 16, 128, 0) >= 1 and f(2, 4096, 4100, 16, 16, 72, 1) >= 4 * 2 * 4100
    assert f(8, 1, 1500, 20, 20, 64, 0) > 0 and f(0, 0, 0, 1, 1, 8, 0) >= 1
    for bad in ((-1, 1, 1, 1, 1, 64), (65537, 1, 1, 1, 1, 64), (1, -1, 1, 1, 1, 64), (1, 1, -1, 1, 1, 64), (1, 1, (1 << 30) + 1, 1, 1, 64),
                (1, 1, 1, 0, 1, 64), (1, 1, 1, 1, 0, 64), (1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 0), (1, 1, 1, 1, 1, 60),
                (1, 1, 1, 1, 1, 264), (2, 1 << 27, 1, 2, 1, 64), (65536, 1, 1, 17, 17, 64), (1, 2 ** 31 - 1, 1, 2 ** 31 - 1, 1, 64)):
        assert f(*bad, 0) == 0, bad


def test_cross_argument_errors():
    need = S._lib.svdq_cross_attention_workspace_bytes(2, 4, 5000, 4, 2, 64, 1)
    row = dict(q=(FAKE, 1024, 256, 64), k=(FAKE, 8192, 128, 64), v=(FAKE, 8192, 128, 64))

    def go(dt=S.BF16, B=2, Lq=4, Lk=5000, Hq=4, Hkv=2, D=64, lens=None, mask=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=need, **kw):
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


# ------------------------------------------------- linear in 8-bit floating point
def test_fp8_oracle_grid():
    """Decoding agrees with torch's e4m3, and rounding with its conversion, ties and subnormals among them."""
    from oracle import fp8
    codes = np.arange(256, dtype=np.uint8)
    table = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.decode(codes), table, equal_nan=True)
    grid = np.sort(table[np.isfinite(table)])
    v = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, np.random.default_rng(3).standard_normal(2000) * 30])
    v = v[np.abs(v) <= 448].astype(np.float32)
    assert np.array_equal(fp8.e4m3(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())
    x = np.array([[448.0, 1.0] + [0.0] * 126 + [450.0, -0.001], [0.0] * 130])
    val, e = fp8.quantize_rows(x)
    assert e.tolist() == [[0, 1], [-127, -127]] and val[0, 0] == 448 and val[0, 128] == 224 and val[0, 129] == 0.0


@pytest.mark.parametrize("N,K", [(1, 8), (128, 128), (130, 264), (300, 1000)])
def test_fp8_weight_quantiser(N, K):
    from oracle import fp8
    r = np.random.default_rng(N + K)
    W = (r.standard_normal((N, K)) * np.exp2(r.integers(-20, 20, (N, K)))).astype(np.float32)
    W[:, ::5] = 0
    codes, scales = S.fp8_quantize_weights(W)
    assert codes.dtype == np.uint8 and codes.shape == (N, K) and scales.shape == (-(-N // 128), fp8.blocks(K))
    for nb in range(scales.shape[0]):
        for kb in range(scales.shape[1]):
            at = np.s_[128 * nb:128 * nb + 128, 128 * kb:128 * kb + 128]
            s = np.abs(W[at]).max() / np.float32(448)
            assert scales[nb, kb] == (s if s > 0 else 1)
            assert np.array_equal(fp8.decode(codes[at]), fp8.e4m3(np.clip(W[at] / scales[nb, kb], -448, 448)))
    again, s2 = S.fp8_quantize_weights(torch.from_numpy(W))
    assert np.array_equal(again, codes) and np.array_equal(s2, scales)


def test_fp8_weight_quantiser_edges():
    W = np.zeros((2, 256), np.float32)
    W[0, 0], W[1, 130], W[0, 131] = 1e-44, 3.4e38, -1.0            # a scale that rounds to zero; the largest numbers
    codes, scales = S.fp8_quantize_weights(W)
    assert scales[0, 0] == 1 and not codes[:, :128].any() and codes[1, 130] == 0x7E and codes[0, 131] == 0x80
    for bad in (np.inf, np.nan):
        W[1, 5] = bad
        with pytest.raises(S.SvdqError):
            S.fp8_quantize_weights(W)
    for shape in ((2, 12), (0, 8), (2, 0)):
        with pytest.raises(S.SvdqError):
            S.fp8_quantize_weights(np.zeros(shape, np.float32))
    with pytest.raises(ValueError):
        S.fp8_quantize_weights(np.zeros(8, np.float32))
    assert S._lib.svdq_fp8_quantize_weights(None, 1, 8, FAKE, FAKE) == INV


def test_fp8_argument_errors():
    lib = S._lib
    assert lib.svdq_fp8_device_weights_bytes(33, 136) == 2 * 2 * 4104
    for bad in ((0, 8), (1, 0), (1, 12), (-1, 8), ((1 << 20) + 1, 8), (1, (1 << 20) + 8), (1 << 20, 1 << 14)):
        assert lib.svdq_fp8_device_weights_bytes(*bad) == 0
    assert lib.svdq_fp8_workspace_bytes(0, 1, 8) >= 1 and lib.svdq_fp8_workspace_bytes(100, 64, 256) >= 100 * 256
    for bad in ((-1, 1, 8), (1, 1, 12), ((1 << 22) + 1, 1, 8), (1 << 20, 1 << 15, 8), (1 << 20, 8, 1 << 15)):
        assert lib.svdq_fp8_workspace_bytes(*bad) == 0

    def pack(codes=FAKE, scales=FAKE, N=33, K=136, blob=FAKE, n=4 * 4104):
        return lib.svdq_fp8_pack_on_device(codes, scales, N, K, blob, n, None)
    assert pack(codes=0) == INV and pack(scales=0) == INV and pack(blob=0) == INV and pack(codes=FAKE + 8) == INV
    assert pack(blob=FAKE + 4) == INV and pack(scales=FAKE + 2) == INV and pack(K=132) == SHAPE and pack(N=0) == SHAPE
    assert pack(n=4 * 4104 - 1) == WS
    w = S.Fp8Weights(FAKE, None, 64, 256)
    need = lib.svdq_fp8_workspace_bytes(100, 64, 256)

    def go(w=w, x=FAKE, row=256, dt=S.BF16, M=100, out=FAKE, odt=S.BF16, epi=0, ws=FAKE, n=need):
        return lib.svdq_fp8_linear_forward(ctypes.byref(w) if w else None, x, row, dt, M, out, odt, epi, ws, n, None)
    assert go(w=None) == INV and go(w=S.Fp8Weights(None, None, 64, 256)) == INV and go(w=S.Fp8Weights(FAKE + 8, None, 64, 256)) == INV
    assert go(w=S.Fp8Weights(FAKE, FAKE + 2, 64, 256)) == INV and go(w=S.Fp8Weights(FAKE, None, 64, 100)) == SHAPE
    assert go(x=0) == INV and go(x=FAKE + 8) == INV and go(row=257) == INV and go(row=-8) == INV and go(dt=S.FP32) == INV
    assert go(out=0) == INV and go(out=FAKE + 2) == INV and go(odt=S.FP32) == INV and go(epi=2) == INV and go(ws=0) == INV
    assert go(ws=FAKE + 4) == INV and go(n=need - 1) == WS and go(M=-1) == SHAPE and go(M=(1 << 22) + 1) == SHAPE
    assert go(M=0, x=0, out=0) == 0

    def quantise(x=FAKE, row=256, dt=S.BF16, M=3, K=256, codes=FAKE, scales=FAKE):
        return lib.svdq_fp8_quantize_activations(x, row, dt, M, K, codes, scales, None)
    assert quantise(x=0) == INV and quantise(codes=0) == INV and quantise(scales=0) == INV and quantise(codes=FAKE + 8) == INV
    assert quantise(row=4) == INV and quantise(dt=S.FP32) == INV and quantise(K=12) == SHAPE and quantise(M=-1) == SHAPE
    assert quantise(M=0, x=0) == 0
    if not torch.cuda.is_available():
        assert go() == NODEV and pack() == NODEV and quantise() == NODEV


def test_fp8_wrapper_checks():
    codes, scales = torch.zeros(200, 136, dtype=torch.uint8), torch.ones(2, 2)
    for bad in (dict(codes=codes.int()), dict(codes=codes[0]), dict(scales=scales[:1]), dict(scales=scales.double()),
                dict(scales=scales * math.inf), dict(bias=torch.zeros(199)), dict(codes=codes[:, :132])):
        with pytest.raises((ValueError, S.SvdqError)):
            S.Fp8Linear(**{**dict(codes=codes, scales=scales, device="cpu"), **bad})
    with pytest.raises(TypeError):
        S.Fp8Linear([1], scales, device="cpu")
    with pytest.raises(ValueError, match="not on cpu"):
        S.Fp8Linear(codes, scales, device="cpu")
    layer = S.Fp8Linear.__new__(S.Fp8Linear)
    layer.N, layer.K, layer.device = 200, 136, torch.device("cpu")
    layer._ref = ctypes.byref(S.Fp8Weights(FAKE, None, 200, 136))
    x = torch.zeros(5, 136, dtype=torch.bfloat16)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=x[0]), dict(x=x.t().contiguous().t()), dict(out=x), dict(out_dtype=torch.float32),
                dict(out=torch.zeros(5, 200)), dict(out=torch.zeros(5, 200).bfloat16(), out_dtype=torch.float16),
                dict(workspace=torch.zeros(5))):
        with pytest.raises(ValueError):
            S.fp8_linear_forward(**{**dict(layer=layer, x=x), **bad})
    with pytest.raises(TypeError):
        S.fp8_linear_forward(layer, [1])
    with pytest.raises(ValueError, match="not on cpu"):
        S.fp8_linear_forward(layer, x)
    with pytest.raises(ValueError, match="not on cpu"):
        S.fp8_quantize_activations(x)
    with pytest.raises(TypeError):
        S.fp8_quantize_activations([1])
    with pytest.raises(ValueError, match="32-bit"):
        layer.new_workspace((1 << 32) + 1)


def test_outputs_that_overlap_inputs_are_found():
    """Against the elements themselves, for dense outputs anywhere in a buffer and inputs of any strides."""
    r = np.random.default_rng(7)
    buf = torch.arange(4000, dtype=torch.int16)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        shape = tuple(int(n) for n in r.integers(1, 5, r.integers(1, 4))) + (int(r.integers(1, 9)),)
        t = buf.as_strided(shape, tuple(int(s) for s in r.choice([0, 1, 8, 9, 24, 40, 130, 300], len(shape) - 1)) + (1,), int(r.integers(0, 400)))
        out = buf[int(r.integers(0, 1900)):][:int(r.integers(1, 120))]
        apart = not np.intersect1d(t.numpy(), out.numpy()).size
        seen[apart] += 1
        if apart:
            S._need_apart(out, t, "t")
        else:
            with pytest.raises(ValueError, match="must not overlap t"):
                S._need_apart(out, t, "t")
    assert min(seen.values()) > 200
    S._need_apart(buf, buf.clone(), "a copy")
    S._need_apart(buf[:0], buf, "nothing")


def test_wrappers_refuse_outputs_that_overlap_inputs():
    layer = S.Fp8Linear.__new__(S.Fp8Linear)
    layer.N, layer.K, layer.device = 136, 136, torch.device("cpu")
    layer._ref = ctypes.byref(S.Fp8Weights(FAKE, None, 136, 136))
    buf = torch.zeros(40, 136, dtype=torch.bfloat16)
    for out in (buf[:5], buf[4:9], buf[:5].half().view(torch.bfloat16)):
        apart = out.data_ptr() < buf.data_ptr() or out.data_ptr() >= buf.data_ptr() + buf.numel() * 2
        with pytest.raises(ValueError, match="not on cpu" if apart else "overlap x"):
            S.fp8_linear_forward(layer, buf[:5], out=out)
    with pytest.raises(ValueError, match="not on cpu"):      # between the rows
        S.fp8_linear_forward(layer, buf[::10][:2], out=buf[4:6])
    q, kv = torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 6, 8, 64, dtype=torch.bfloat16)
    k, v = kv[:, :, :4], kv[:, :, 4:]
    for args, out, why in (((q, k, v), q, "not on cpu"), ((q, q, v), q, "overlap k"), ((q, k, q), q, "overlap v"),
                           ((k, q.clone(), v.clone()), kv.view(-1)[:q.numel()].view(q.shape), "overlap q"),
                           ((q, k, v), kv.view(-1)[-q.numel():].view(q.shape), "overlap k")):
        with pytest.raises(ValueError, match=why):
            S.cross_attention(*args, out=out, workspace=torch.zeros(1, dtype=torch.uint8))
