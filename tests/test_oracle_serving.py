"""Pins of the serving oracles (key/value cache, attention, router, experts)
and the argument checks of their entry points, which come before any device
work."""
import ctypes

import numpy as np
import pytest
import torch

import w4a4_rank_corrected_smooth_amd as S
from oracle import awq, kv4, moe

INV, SHAPE, NODEV, WS = 1, 2, 3, 5
FAKE = 1 << 20


# ------------------------------------------------------------------ oracles
def test_cache_values_by_hand():
    x = np.zeros((2, 64))
    x[0, :4] = [6.0, -1.1, 0.25, 0.75]              # e = 0: 0.25 ties to 0, 0.75 to 1
    x[0, 32:35] = [48.0, 10.0, -14.0]               # e = 3: 1.25 ties to 1, 1.75 to 2
    x[1, 5] = np.inf
    v = kv4.values(x)
    assert v[0, :4].tolist() == [6.0, -1.0, 0.0, 1.0]
    assert v[0, 32:35].tolist() == [48.0, 8.0, -16.0]
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all()


def test_attention_by_hand():
    k = np.zeros((3, 1, 64))
    v = np.arange(3.0)[:, None, None] * np.ones((3, 1, 64))
    q = np.ones((2, 2, 2, 64))
    out, _, _, terms = kv4.attend(q, [k, k[:1]], [v, v[:1]], [3, 1], 0.125)
    assert np.allclose(out[0, 0], 0.5) and np.allclose(out[0, 1], 1.0)     # tokens 0..1, 0..2
    assert (out[1, 0] == 0).all() and (out[1, 1] == 0).all() and terms[1, 0, 0] == 0


def test_attention_against_pairs():
    r = np.random.default_rng(3)
    q, k, v = r.standard_normal((1, 1, 4, 64)), r.standard_normal((9, 2, 64)), r.standard_normal((9, 2, 64))
    out, *_ = kv4.attend(q, [k], [v], [9], 0.3)
    for h in range(4):
        w = [np.exp(0.3 * float(sum(q[0, 0, h, d] * k[t, h // 2, d] for d in range(64)))) for t in range(9)]
        for d in (0, 17, 63):
            assert abs(out[0, 0, h, d] - sum(w[t] * v[t, h // 2, d] for t in range(9)) / sum(w)) < 1e-12


def test_route_by_hand():
    w = np.eye(4, 8)
    x = np.zeros((2, 8))
    x[0, :4] = [0.0, np.log(2.0), 0.0, np.log(4.0)]
    ids, wt = moe.route(x, w, 3)
    assert ids.tolist() == [[3, 1, 0], [0, 1, 2]]            # ties go to the lower index
    assert np.allclose(wt[0], np.array([4, 2, 1]) / 7)
    ids, wt = moe.route(x, w, 2, bias=[0.9, 0.0, 0.0, 0.0], score="sigmoid", normalize=False)
    assert ids[0].tolist() == [0, 3] and np.allclose(wt[0], [0.5, 0.8])


def test_expert_layer_against_dense_matrices():
    r = np.random.default_rng(5)
    K, I, E = 128, 64, 3
    experts = [[awq.quantize((r.standard_normal(s) / 8).astype(np.float16)) for _ in range(E)] for s in ((2 * I, K), (K, I))]
    x = r.standard_normal((2, K))
    ids, wt = [[2, -1], [1, 1]], [[0.7, 0.3], [0.25, 0.5]]
    y, bound = moe.layer(x, *experts, ids, wt)
    for t, want in ((0, [(2, 0.7)]), (1, [(1, 0.75)])):
        ref = 0
        for e, w in want:
            m, d = awq.dequantize(*experts[0][e]), awq.dequantize(*experts[1][e])
            g, u = m[:I] @ x[t], m[I:] @ x[t]
            ref = ref + w * (d @ (g / (1 + np.exp(-g)) * u))
        assert np.allclose(y[t], ref, atol=1e-12)
    # a worst case over every order and sign: 286 |x| s a term, 2^-24 (64 + 2 + 8) of it
    assert (bound > 0).all() and (bound < 0.05 * np.abs(y).max()).all()


# --------------------------------------------------------------- refusals (C)
def _cache(pages=4, page=64, heads=2, dim=128, data=FAKE):
    return S.Kv4CacheStruct(data, pages, page, heads, dim)


def test_size_queries():
    lib = S._lib
    assert lib.svdq_kv4_cache_bytes(4, 64, 2, 128) == 4 * 2 * 64 * (128 + 8)
    for bad in ((0, 64, 2, 128), (4, 48, 2, 128), (4, 8, 2, 128), (4, 512, 2, 128), (4, 64, 0, 128), (4, 64, 2, 96),
                (1 << 27, 16, 2, 128)):
        assert lib.svdq_kv4_cache_bytes(*bad) == 0
    assert lib.svdq_kv4_attention_workspace_bytes(1, 1, 8, 2, 128) > 0
    for bad in ((1, 0, 8, 2, 128), (1, 1, 7, 2, 128), (1, 257, 8, 2, 128), (-1, 1, 8, 2, 128), (65537, 1, 2, 2, 128),
                (1, 1, 8, 2, 80)):
        assert lib.svdq_kv4_attention_workspace_bytes(*bad) == 0
    assert lib.svdq_moe_route_workspace_bytes(3, 8) >= 3 * 8 * 8
    assert lib.svdq_moe_route_workspace_bytes(3, 1025) == 0 and lib.svdq_moe_route_workspace_bytes(-1, 8) == 0
    assert lib.awq_moe_workspace_bytes(2, 2, 128, 64) > 0
    for bad in ((2, 0, 128, 64), (2, 33, 128, 64), (129, 32, 128, 64), (2, 2, 100, 64), (2, 2, 128, 96), (-1, 2, 128, 64)):
        assert lib.awq_moe_workspace_bytes(*bad) == 0


def test_cache_argument_errors():
    lib, c = S._lib, _cache()

    def append(cache=c, k=FAKE, kr=256, kh=128, v=FAKE, vr=256, vh=128, dt=S.BF16, T=3, slots=FAKE):
        return lib.svdq_kv4_append(ctypes.byref(cache) if cache else None, k, kr, kh, v, vr, vh, dt, T, slots, None)
    assert append(cache=None) == INV and append(cache=_cache(data=0)) == INV and append(cache=_cache(data=FAKE + 8)) == INV
    assert append(cache=_cache(page=24)) == SHAPE and append(cache=_cache(dim=32)) == SHAPE
    assert append(k=0) == INV and append(v=0) == INV and append(slots=0) == INV and append(k=FAKE + 2) == INV
    assert append(kr=100) == INV and append(vh=-128) == INV and append(dt=S.FP32) == INV and append(T=-1) == SHAPE
    assert append(T=0) == 0

    def read(T=3, k=FAKE, dt=S.BF16, slots=FAKE):
        return lib.svdq_kv4_read(ctypes.byref(c), slots, T, k, FAKE, dt, None)
    assert read(T=-1) == SHAPE and read(k=0) == INV and read(k=FAKE + 8) == INV and read(dt=S.FP16) == INV
    assert read(slots=FAKE + 1) == INV and read(T=0) == 0

    need = lib.svdq_kv4_attention_workspace_bytes(2, 1, 8, 2, 128)

    def attend(q=FAKE, qs=(1024, 1024, 128), dt=S.BF16, B=2, Q=1, Hq=8, table=FAKE, width=3, lens=FAKE, scale=0.1,
               out=FAKE, ws=FAKE, n=need):
        return lib.svdq_kv4_attention(ctypes.byref(c), q, *qs, dt, B, Q, Hq, table, width, lens, scale, out, ws, n, None)
    assert attend(q=0) == INV and attend(table=0) == INV and attend(lens=0) == INV and attend(out=0) == INV
    assert attend(ws=0) == INV and attend(q=FAKE + 2) == INV and attend(out=FAKE + 8) == INV and attend(table=FAKE + 2) == INV
    assert attend(qs=(1024, 1024, 100)) == INV and attend(dt=S.FP32) == INV
    assert attend(scale=float("nan")) == INV and attend(scale=float("inf")) == INV
    assert attend(scale=2.0 ** 127) == INV and attend(scale=-(2.0 ** 127)) == INV
    assert attend(width=0) == SHAPE and attend(Hq=7) == SHAPE and attend(Q=0) == SHAPE and attend(B=-1) == SHAPE
    assert attend(n=need - 1) == WS and attend(B=0) == 0


def test_moe_argument_errors():
    lib = S._lib
    need = lib.svdq_moe_route_workspace_bytes(3, 8)

    def route(x=FAKE, w=FAKE, bias=None, dt=S.BF16, T=3, E=8, K=64, k=2, score=0, ids=FAKE, wt=FAKE, ws=FAKE, n=need):
        return lib.svdq_moe_route(x, w, bias, dt, T, E, K, k, score, 1, ids, wt, ws, n, None)
    assert route(x=0) == INV and route(w=0) == INV and route(ids=0) == INV and route(wt=0) == INV and route(ws=0) == INV
    assert route(x=FAKE + 8) == INV and route(bias=FAKE + 1) == INV and route(dt=S.FP32) == INV and route(score=2) == INV
    assert route(E=0) == SHAPE and route(K=12) == SHAPE and route(k=9) == SHAPE and route(k=0) == SHAPE
    assert route(T=65536) == SHAPE and route(n=need - 1) == WS and route(T=0) == 0

    need = lib.awq_moe_workspace_bytes(3, 2, 128, 64)
    good = S.MoeWeights(FAKE, FAKE, 4, 128, 64)

    def layer(w=good, x=FAKE, dt=S.BF16, T=3, ids=FAKE, wt=FAKE, k=2, act=0, y=FAKE, ws=FAKE, n=need):
        return lib.awq_moe_forward(ctypes.byref(w) if w else None, x, dt, T, ids, wt, k, act, y, ws, n, None)
    assert layer(w=None) == INV and layer(w=S.MoeWeights(0, FAKE, 4, 128, 64)) == INV
    assert layer(w=S.MoeWeights(FAKE, FAKE + 8, 4, 128, 64)) == INV
    assert layer(w=S.MoeWeights(FAKE, FAKE, 0, 128, 64)) == SHAPE and layer(w=S.MoeWeights(FAKE, FAKE, 4, 100, 64)) == SHAPE
    assert layer(x=0) == INV and layer(ids=0) == INV and layer(wt=0) == INV and layer(y=0) == INV and layer(ws=0) == INV
    assert layer(y=FAKE + 2) == INV and layer(dt=S.FP32) == INV and layer(act=5) == INV
    assert layer(T=-1) == SHAPE and layer(k=33) == SHAPE and layer(T=2049) == SHAPE
    assert layer(n=need - 1) == WS and layer(T=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device_is_reported():
    lib, c = S._lib, _cache()
    assert lib.svdq_kv4_append(ctypes.byref(c), FAKE, 256, 128, FAKE, 256, 128, S.BF16, 1, FAKE, None) == NODEV
    assert lib.svdq_kv4_read(ctypes.byref(c), FAKE, 1, FAKE, FAKE, S.BF16, None) == NODEV
    assert lib.svdq_kv4_attention(ctypes.byref(c), FAKE, 256, 256, 128, S.BF16, 1, 1, 2, FAKE, 1, FAKE, 0.1, FAKE, FAKE,
                                  1 << 40, None) == NODEV
    assert lib.svdq_moe_route(FAKE, FAKE, None, S.BF16, 1, 8, 64, 2, 0, 1, FAKE, FAKE, FAKE, 1 << 20, None) == NODEV
    w = S.MoeWeights(FAKE, FAKE, 4, 128, 64)
    assert lib.awq_moe_forward(ctypes.byref(w), FAKE, S.BF16, 1, FAKE, FAKE, 2, 0, FAKE, FAKE, 1 << 20, None) == NODEV


# ---------------------------------------------------------- refusals (Python)
def test_wrappers_check_their_operands():
    """Nothing reaches the library with operands that its arguments do not describe."""
    cache = S.Kv4Cache(4, 16, 2, 64, device="cpu")
    bf = torch.bfloat16
    k, slots = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, dtype=torch.int32)
    for bad in ((k[:, :1], k, slots), (k, k.half(), slots), (k, k[:2], slots), (k, k, slots.long()), (k, k, slots[:2]),
                (k.transpose(1, 2).contiguous().transpose(1, 2), k, slots), (k.float(), k.float(), slots)):
        with pytest.raises(ValueError):
            S.kv4_append(cache, *bad)
    with pytest.raises(TypeError):
        S.kv4_append(cache, [1], k, slots)
    with pytest.raises(ValueError):
        S.kv4_read(cache, slots, dtype=torch.float16)
    q, table, lens = torch.zeros(2, 1, 4, 64, dtype=bf), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in ((q[..., :32], table, lens), (q, table[:1], lens), (q, table.t().contiguous().t(), lens), (q, table, lens[:1]),
                (q, table.long(), lens), (q.float(), table, lens)):
        with pytest.raises(ValueError):
            S.kv4_attention(cache, *bad)
    with pytest.raises(ValueError):
        S.kv4_attention(cache, q, table, lens, out=torch.zeros(2, 1, 4, 64))
    with pytest.raises(S.SvdqError):
        S.kv4_attention(cache, torch.zeros(2, 1, 3, 64, dtype=bf), table, lens)      # 3 heads over 2
    # operands that fit, in CPU memory
    for call in (lambda: S.kv4_append(cache, k, k, slots), lambda: S.kv4_read(cache, slots),
                 lambda: S.kv4_attention(cache, q, table, lens)):
        with pytest.raises(ValueError, match="not on cpu"):
            call()
    with pytest.raises(S.SvdqError):
        S.Kv4Cache(4, 20, 2, 64, device="cpu")
    x, w = torch.zeros(3, 64, dtype=bf), torch.zeros(8, 64, dtype=bf)
    for bad in (dict(x=x.half()), dict(w_router=w[:, :32]), dict(top_k=9), dict(top_k=0), dict(score="top"),
                dict(bias=torch.zeros(7)), dict(bias=torch.zeros(8).half()), dict(x=x[:, ::2])):
        with pytest.raises(ValueError):
            S.moe_route(**{**dict(x=x, w_router=w, top_k=2), **bad})
    r = np.random.default_rng(0)

    def part(E, N, K):
        return (r.integers(0, 256, (E, N, K // 2), dtype=np.uint8), np.ones((E, N, K // 64), np.float16),
                np.full((E, N, K // 64), 8, np.float16))
    layer = S.AwqMoe(part(2, 128, 128), part(2, 128, 64), device="cpu")
    assert (layer.E, layer.K, layer.I) == (2, 128, 64)
    with pytest.raises(ValueError):
        S.AwqMoe(part(2, 128, 128), part(3, 128, 64), device="cpu")
    with pytest.raises(ValueError):
        S.AwqMoe(part(2, 128, 128), part(2, 192, 64), device="cpu")
    q8, s8, z8 = part(2, 128, 128)
    z8[1, 5, 0] = 16                                       # zero points are 0..15
    with pytest.raises(S.SvdqError):
        S.AwqMoe((q8, s8, z8), part(2, 128, 64), device="cpu")
    x, ids, wt = torch.zeros(3, 128, dtype=bf), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    for bad in ((x[:, :64], ids, wt), (x, ids[:2], wt), (x, ids.long(), wt), (x, ids, wt[:, :1]), (x, ids, wt.half())):
        with pytest.raises(ValueError):
            S.awq_moe_forward(layer, *bad)
    with pytest.raises(ValueError):
        S.awq_moe_forward(layer, x, ids, wt, activation="relu")
    for call in (lambda: S.awq_moe_forward(layer, x, ids, wt), lambda: S.moe_route(x, torch.zeros(8, 128, dtype=bf), 2)):
        with pytest.raises(ValueError, match="not on cpu"):
            call()


@pytest.mark.parametrize("E,N,K", [(1, 64, 64), (3, 128, 192), (2, 192, 256)])
def test_expert_blob_layout(E, N, K):
    """A reader of the documented blocks finds every code, scale and zero point in its place."""
    r = np.random.default_rng(E)
    G, P = K // 64, (K // 64 + 1) // 2
    codes = r.integers(0, 16, (E, N, K), dtype=np.uint8)
    s = r.standard_normal((E, N, G)).astype(np.float16)
    z = r.integers(0, 16, (E, N, G)).astype(np.float16)
    blob = S._moe_blob((awq.pack(codes), s, z), N, K, "cpu").numpy().reshape(E, N // 16, P, 1152)
    for e in range(E):
        for n in r.permutation(N)[:40]:
            for g in range(G):
                block = blob[e, n // 16, g // 2]
                words = block[1024 + 8 * (n % 16) + 4 * (g % 2):][:4].view(np.float16)
                assert words[0] == s[e, n, g] and words[1] == z[e, n, g]
                for k in r.permutation(64)[:16]:
                    lane = block[(n % 16 + 16 * (k // 16)) * 16 + 8 * (g % 2):][:8]
                    word = int(lane[4 * (k % 16 // 8):][:4].view(np.uint32)[0])
                    assert word >> (16 * (k % 2) + 4 * (k % 8 // 2)) & 15 == codes[e, n, 64 * g + k]
    if G % 2:
        last = blob[:, :, -1]
        assert not last[..., 1024:].reshape(E, -1, 16, 8)[..., 4:].any()
        assert not last[..., :1024].reshape(E, -1, 64, 16)[..., 8:].any()


def test_expert_blob_refusals():
    lib = S._lib
    assert lib.awq_moe_device_weights_bytes(2, 128, 192) == 2 * 8 * 2 * 1152
    for bad in ((0, 128, 128), (1025, 128, 128), (1, 100, 128), (1, 128, 96), (1, 0, 128), (1, 1 << 16, 1 << 16)):
        assert lib.awq_moe_device_weights_bytes(*bad) == 0
    q, s, z = np.zeros((1, 64, 32), np.uint8), np.ones((1, 64, 1), np.float16), np.zeros((1, 64, 1), np.float16)
    blob = np.zeros(4 * 1152, np.uint8)

    def pack(q=q, s=s, z=z, n=blob.size, K=64):
        return lib.awq_moe_pack_device_weights(S._ptr(q), S._ptr(s), S._ptr(z), 1, 64, K, S._ptr(blob), n)
    assert pack() == 0 and pack(q=None) == INV and pack(K=96) == SHAPE and pack(n=blob.size - 1) == WS
    for bad in (0.5, 16.0, -1.0, np.nan):
        assert pack(z=np.full_like(z, bad)) == INV
    assert pack(s=np.full_like(s, np.inf)) == 6

    def on_device(q=FAKE, s=FAKE, z=FAKE, E=1, K=64, blob=FAKE, n=blob.size):
        return lib.awq_moe_pack_on_device(q, s, z, E, 64, K, blob, n, None)
    assert on_device(q=0) == INV and on_device(s=0) == INV and on_device(blob=0) == INV and on_device(q=FAKE + 8) == INV
    assert on_device(z=FAKE + 1) == INV and on_device(blob=FAKE + 4) == INV and on_device(K=96) == SHAPE
    assert on_device(E=0) == SHAPE and on_device(n=blob.size - 1) == WS


def test_attention_refuses_tables_past_its_token_numbers():
    """A length past 2^30 tokens would be cut off there, and a line of work past 2^31 would wrap.  (The calls have no
    workspace, so one that is taken ends there.)"""
    def attend(B, width, page=64, Q=1, Hq=8):
        return S._lib.svdq_kv4_attention(ctypes.byref(_cache(page=page)), FAKE, 1024, 1024, 128, S.BF16, B, Q, Hq, FAKE,
                                         width, FAKE, 0.1, FAKE, FAKE, 0, None)
    assert attend(1, (1 << 24) + 1) == SHAPE and attend(1, (1 << 22) + 1, page=256) == SHAPE and attend(1, 2 ** 31 - 1) == SHAPE
    assert attend(65536, 1 << 16) == SHAPE and attend(1000, 1 << 17, Q=256) == SHAPE
    assert attend(1, 1 << 24) == WS and attend(1, 1 << 22, page=256) == WS and attend(65536, 1 << 10) == WS
    assert attend(1000, 1 << 15, Q=256) == WS


def test_wrappers_refuse_sizes_past_32_bits():
    """2^32 + n would reach the library as n."""
    more = 1 << 32
    for bad in ((more + 4, 16, 2, 64), (4, more + 16, 2, 64), (4, 16, more + 2, 64), (4, 16, 2, more + 64), (4 - more, 16, 2, 64)):
        with pytest.raises(ValueError, match="32-bit"):
            S.Kv4Cache(*bad, device="meta")
    cache = S.Kv4Cache(4, 16, 2, 64, device="meta")
    rows = torch.empty(more + 1, 2, 64, dtype=torch.bfloat16, device="meta")
    slots = torch.empty(more + 1, dtype=torch.int32, device="meta")
    for call in (lambda: S.kv4_append(cache, rows, rows, slots), lambda: S.kv4_read(cache, slots),
                 lambda: S.kv4_attention_workspace(cache, torch.empty(more + 1, 1, 2, 64, device="meta")),
                 lambda: S.kv4_attention(cache, rows[:1, None], slots[None], slots[:1]),
                 lambda: S.moe_route(rows[:, 0, :8].contiguous(), rows[:4, 0, :8].contiguous(), 2)):
        with pytest.raises(ValueError, match="32-bit"):
            call()
    part = [np.zeros((1, 128, 64), np.uint8), np.ones((1, 128, 2), np.float16), np.zeros((1, 128, 2), np.float16)]
    layer = S.AwqMoe(part, [np.zeros((1, 128, 32), np.uint8), *(a[..., :1] for a in part[1:])], device="cpu")
    for sizes in ((more + 3, 2), (3, more + 2)):
        with pytest.raises(ValueError, match="32-bit"):
            layer.new_workspace(*sizes)
