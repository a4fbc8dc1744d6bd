"""Cross attention on the GPU against the float64 oracle.

Tolerance.  With u half a step of the 16-bit type (eps / 2) and, per element,
mean = sum p |v| / sum p:
  - a score's float32 sum over D channels and its product with scale log2(e) are off
    by at most (D + 4) 2^-23 size (size: the row's largest |scale| sum |q k|; a step of the matrix
    instruction counted as 2^-23), the exponent's argument by 2^-23 of itself (below 2 size) and the exponential by 2^-22:
    a relative error E of each weight, at most 2 E mean in the result;
  - the weights are rounded to the type: u mean (float16's below 2^-14 of 2^7 by an
    absolute 2^-25 of at least 2^7: n 2^-32 of the largest value);
  - the two sums over n states: 2 n 2^-23 mean at most;
  - the result is rounded: u |out|.
"""
import numpy as np
import pytest
import torch

from oracle import cross as O
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


def rows(r, shape, dtype, scale=1.0):
    x = r.standard_normal(shape) * scale
    x[..., ::29] *= 3.0
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def near(got, q, k, v, visible=None, scale=None):
    q, k, v = f64(q), f64(k), f64(v)
    B, Lk, D = k.shape[0], k.shape[1], q.shape[3]
    visible = np.ones((B, Lk), bool) if visible is None else visible
    want, mean, size = O.attend(q, k, v, visible, D ** -0.5 if scale is None else scale)
    u = torch.finfo(got.dtype).eps / 2
    E = (D + 6) * 2.0 ** -23 * size + 2.0 ** -22
    tol = u * np.abs(want) + (u + 2 * E + 2 * Lk * 2.0 ** -23) * mean * (1 + 2.0 ** -6)
    if got.dtype == torch.float16:
        vis = np.where(visible[:, :, None, None], np.abs(v), 0)
        tol = tol + 2.0 ** -25 + Lk * 2.0 ** -32 * (vis.max() if vis.size else 0)
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    off = np.abs(got - want)
    fine = np.isfinite(want)
    assert (off[fine] <= tol[fine]).all(), (off[fine].max(), (off[fine] / np.maximum(tol[fine], 1e-30)).max())


CASES = [  # B, Lq, Lk, Hq, Hkv, D
    (1, 1, 1, 1, 1, 64),
    (2, 1, 1500, 4, 4, 64),
    (3, 1, 257, 8, 2, 128),
    (1, 32, 31, 1, 1, 96),
    (1, 33, 33, 2, 1, 8),
    (2, 5, 700, 6, 3, 72),
    (1, 128, 64, 2, 2, 128),
    (2, 129, 65, 3, 3, 128),
    (1, 300, 1000, 2, 1, 64),
    (1, 77, 513, 2, 2, 80),
    (2, 64, 2050, 8, 2, 128),
    (1, 200, 96, 2, 2, 160),
    (1, 3, 95, 2, 2, 160),
    (1, 140, 130, 2, 1, 256),
    (2, 1, 999, 2, 1, 256),
    (1, 40, 100, 2, 2, 200),
    (1, 1000, 300, 8, 8, 72),
    (1, 31, 4097, 1, 1, 104),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D", CASES)
@pytest.mark.parametrize("hide", ["none", "lens", "mask", "both"])
def test_cross_attention_against_the_oracle(S, B, Lq, Lk, Hq, Hkv, D, hide, dtype):
    announce(f"cross B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D} {hide} {dtype}")
    r = np.random.default_rng(Lq * 1000 + Lk + D)
    q, kv = rows(r, (B, Lq, Hq, D), dtype), rows(r, (B, Lk, 2 * Hkv, D), dtype)
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:]
    visible = np.ones((B, Lk), bool)
    lens = mask = None
    if hide in ("lens", "both"):
        n = r.integers(1, Lk + 1, B)
        if B > 1:
            n[1] = 0
        lens = torch.from_numpy(n.astype(np.int32)).cuda()
        visible &= np.arange(Lk) < n[:, None]
    if hide in ("mask", "both"):
        m = r.random((B, Lk)) < 0.6
        mask = torch.from_numpy(m).cuda()
        visible &= m
    # what is not visible may be anything
    hidden = torch.from_numpy(~visible).cuda()
    k[hidden], v[hidden] = float("nan"), float("inf")
    got = S.cross_attention(q, k, v, key_lens=lens, mask=mask)
    assert got.shape == q.shape and got.dtype == q.dtype and got.is_contiguous()
    k, v = k.masked_fill(hidden[..., None, None], 0), v.masked_fill(hidden[..., None, None], 0)
    near(got, q, k, v, visible)
    assert not got[torch.from_numpy(~visible.any(1)).cuda()].any()


@pytest.mark.parametrize("Lq", [1, 200])
def test_cross_attention_strides_and_scales(S, Lq):
    """Heads before tokens, shared batches (stride 0), negative, zero and large scales."""
    r = np.random.default_rng(3)
    B, Lk, H, D = 2, 300, 4, 64
    q = rows(r, (B, H, Lq, D), "bf16").transpose(1, 2)
    k = rows(r, (1, H, Lk, D), "bf16").transpose(1, 2).expand(B, -1, -1, -1)
    v = rows(r, (Lk, B, H, D), "bf16").transpose(0, 1)
    for scale in (None, -0.3, 0.0, 20.0):
        announce(f"cross of strided rows, scale {scale}, Lq={Lq}")
        near(S.cross_attention(q, k, v, scale=scale), q, k, v, scale=scale)


@pytest.mark.parametrize("Lq", [3, 150])
def test_cross_attention_edge_values(S, Lq):
    """Infinities and NaN in queries stay in their row; in visible states they reach the rows that see them."""
    r = np.random.default_rng(4)
    q, k, v = rows(r, (2, Lq, 2, 64), "bf16"), rows(r, (2, 70, 2, 64), "bf16"), rows(r, (2, 70, 2, 64), "bf16")
    want = S.cross_attention(q, k, v)
    bad = q.clone()
    bad[0, 1, 0, 5], bad[1, 2, 1, 63] = float("nan"), float("inf")
    announce(f"cross with a NaN and an infinity in queries, Lq={Lq}")
    got = S.cross_attention(bad, k, v)
    hit = torch.zeros(2, Lq, 2, dtype=torch.bool, device="cuda")
    hit[0, 1, 0] = hit[1, 2, 1] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])
    bv = v.clone()
    bv[0, 69, 1, 7] = float("nan")
    got = S.cross_attention(q, k, bv)
    assert torch.isnan(got[0, :, 1, 7]).all()
    got[0, :, 1, 7] = want[0, :, 1, 7]
    assert torch.equal(got, want)
    # scores of -inf only: 0 / 0; one finite score among them: its value
    k2, q2 = torch.zeros_like(k), torch.ones_like(q)
    k2[..., 0] = -float("inf")
    k2[1, 40] = 0
    announce(f"cross with scores of -inf, Lq={Lq}")
    got = S.cross_attention(q2, k2, v)
    assert torch.isnan(got[0]).all() and torch.equal(got[1], v[1, 40].expand(Lq, -1, -1))


@pytest.mark.parametrize("Lq", [1, 130])
def test_cross_attention_rising_scores(S, Lq):
    """Scores that climb from tile to tile, in steps below and above the slack of the running maximum, and a late giant."""
    r = np.random.default_rng(5)
    Lk, D = 900, 64
    for step in (0.02, 0.3, 3.0):
        q = torch.ones(1, Lq, 1, D, dtype=torch.float16, device="cuda")
        t = np.arange(Lk) * step / D
        t[-3] += 200.0 / D
        k = torch.from_numpy(np.broadcast_to(t[:, None], (Lk, D)).copy()).half().cuda()[None, :, None]
        v = rows(r, (1, Lk, 1, D), "fp16")
        announce(f"cross with scores rising by {step}, Lq={Lq}")
        near(S.cross_attention(q, k, v, scale=1.0), q, k, v, scale=1.0)


def test_cross_attention_many_small_weights(S):
    """One state of weight 1 and 16000 of weight e^-17: in float16 as such they would all vanish."""
    Lk, D = 16001, 64
    k = torch.zeros(1, Lk, 1, D, dtype=torch.float16, device="cuda")
    k[0, 77, 0, 0] = 17.0
    q = torch.zeros(1, 40, 1, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    v = torch.full((1, Lk, 1, D), 1000.0, dtype=torch.float16, device="cuda")
    v[0, 77] = 0.0
    announce("cross with many small weights")
    near(S.cross_attention(q, k, v, scale=1.0), q, k, v, scale=1.0)


def test_cross_attention_empty_calls(S):
    bf = dict(dtype=torch.bfloat16, device="cuda")
    announce("cross of empty calls")
    assert S.cross_attention(torch.empty(0, 4, 2, 64, **bf), torch.empty(0, 4, 2, 64, **bf), torch.empty(0, 4, 2, 64, **bf)).numel() == 0
    assert S.cross_attention(torch.empty(2, 0, 2, 64, **bf), torch.empty(2, 4, 2, 64, **bf), torch.empty(2, 4, 2, 64, **bf)).numel() == 0
    for Lq in (2, 200):
        q = torch.ones(2, Lq, 2, 64, **bf)
        none = torch.empty(2, 0, 2, 64, **bf)
        assert not S.cross_attention(q, none, none).any()
        assert not S.cross_attention(q, none, none, mask=torch.empty(2, 0, dtype=torch.bool, device="cuda")).any()
        k = torch.ones(2, 50, 2, 64, **bf)
        out = torch.full_like(q, 3.0)
        assert not S.cross_attention(q, k, k, mask=torch.zeros(2, 50, dtype=torch.bool, device="cuda"), out=out).any()
        assert not S.cross_attention(q, k, k, key_lens=torch.tensor([-5, 0], dtype=torch.int32, device="cuda")).any()
        assert torch.equal(S.cross_attention(q, k, k, key_lens=torch.tensor([51, 1 << 30], dtype=torch.int32, device="cuda")), q)


def gpu_reference(q, k, v, visible, scale):
    """The same reference as near()'s, in float64 on the GPU, for many rows: out, mean and size."""
    B, Lq, Hq, D = q.shape
    g = Hq // k.shape[2]
    q, k, v = q.double(), k.double(), v.double()
    out, mean, size = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(B, Lq, Hq, 1, dtype=torch.float64, device="cuda")
    for b in range(B):
        at = torch.nonzero(visible[b])[:, 0]
        for h in range(Hq if len(at) else 0):
            kk, vv = k[b, at, h // g], v[b, at, h // g]
            p = torch.softmax(scale * (q[b, :, h] @ kk.t()), -1)
            out[b, :, h], mean[b, :, h] = p @ vv, p @ vv.abs()
            size[b, :, h] = abs(scale) * (q[b, :, h].abs() @ kk.abs().t()).amax(-1, keepdim=True)
    return out, mean, size


@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D", [(6, 64, 3001, 4, 1, 128), (7, 3, 5000, 2, 2, 64), (64, 1, 900, 2, 1, 96), (65, 1, 900, 2, 1, 64),
                                              (2, 200, 2500, 1, 1, 256), (20, 2, 1100, 3, 3, 128)])
@pytest.mark.parametrize("kind", ["spread", "one", "none", "equal"])
def test_cross_attention_ragged_lengths(S, B, Lq, Lk, Hq, Hkv, D, kind):
    """Parts shared out by length: very different lengths, all states in one batch row, none anywhere, all alike."""
    announce(f"cross of ragged lengths B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D} {kind}")
    r = np.random.default_rng(B * Lk)
    lens = {"spread": np.exp(r.uniform(0, np.log(Lk), B)).astype(int), "one": np.zeros(B, int), "none": np.zeros(B, int),
            "equal": np.full(B, Lk)}[kind]
    if kind == "spread":
        lens[0], lens[-1] = Lk, 0
    if kind == "one":
        lens[B // 2] = Lk
    g = torch.Generator(device="cuda").manual_seed(B)
    q = torch.randn(B, Lq, Hq, D, device="cuda", generator=g).half()
    k, v = (torch.randn(B, Lk, Hkv, D, device="cuda", generator=g).half() for _ in range(2))
    n = torch.from_numpy(lens.astype(np.int32)).cuda()
    visible = torch.arange(Lk, device="cuda") < n[:, None]
    k[~visible], v[~visible] = float("nan"), float("inf")
    got = S.cross_attention(q, k, v, key_lens=n)
    want, mean, size = gpu_reference(q, k, v, visible, D ** -0.5)
    u = 2.0 ** -11
    tol = u * want.abs() + (u + 2 * ((D + 6) * 2.0 ** -23 * size + 2.0 ** -22) + 2 * Lk * 2.0 ** -23) * mean * (1 + 2.0 ** -6) + 2.0 ** -25
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("hide", ["none", "lens", "mask"])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D", [
    (1, 4100, 77, 16, 16, 64), (2, 2049, 576, 32, 16, 40), (1, 2200, 577, 32, 32, 64), (3, 5000, 1, 6, 6, 72), (2, 2048, 300, 32, 16, 72),
    (1, 5500, 384, 12, 12, 96), (1, 2050, 385, 32, 32, 96), (2, 4097, 256, 8, 8, 128), (1, 3000, 64, 24, 24, 104),
    (1, 2100, 257, 32, 32, 128), (300, 40, 9, 4, 4, 32)])
def test_cross_attention_many_rows_few_states(S, B, Lq, Lk, Hq, Hkv, D, hide):
    """The form that keeps a head's states in LDS, at its largest lengths and one past them."""
    announce(f"cross of many rows B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D} {hide}")
    dtype = torch.float16 if (Lq + Lk) % 2 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(Lq + Lk)
    q = torch.randn(B, Lq, Hq, D, device="cuda", generator=g).to(dtype)
    kv = torch.randn(B, Lk, 2 * Hkv, D, device="cuda", generator=g).to(dtype)
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:]
    visible = torch.ones(B, Lk, dtype=torch.bool, device="cuda")
    lens = mask = None
    if hide == "lens":
        lens = torch.randint(0, Lk + 1, (B,), device="cuda", generator=g).int()
        lens[0] = Lk
        visible = torch.arange(Lk, device="cuda") < lens[:, None]
    if hide == "mask":
        mask = visible = torch.rand(B, Lk, device="cuda", generator=g) < 0.7
    k[~visible], v[~visible] = float("nan"), float("inf")
    got = S.cross_attention(q, k, v, key_lens=lens, mask=mask)
    want, mean, size = gpu_reference(q, k, v, visible, D ** -0.5)
    u = torch.finfo(dtype).eps / 2
    tol = u * want.abs() + (u + 2 * ((D + 6) * 2.0 ** -23 * size + 2.0 ** -22) + 2 * Lk * 2.0 ** -23) * mean * (1 + 2.0 ** -6) + 2.0 ** -25
    assert ((got.double() - want).abs() <= tol).all()


def test_cross_attention_large(S):
    """Row tiles, heads and states beyond one round of workgroups, against float32 products on the GPU."""
    B, Lq, Lk, H, D = 1, 5000, 3000, 6, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(B, n, H, D, device="cuda", generator=g).bfloat16() for n in (Lq, Lk, Lk))
    announce("cross of 5000 queries over 3000 states")
    got = S.cross_attention(q, k, v)
    for h in range(H):
        p = torch.softmax(q[0, :, h].double() @ k[0, :, h].double().t() / D ** 0.5, -1)
        want, mean = p @ v[0, :, h].double(), p @ v[0, :, h].double().abs()
        # scores below 30: an error of 140 2^-23 30 in a weight, and the sums' 3000 2^-23, beside 2^-8
        assert ((got[0, :, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -9) * mean).all()


@pytest.mark.parametrize("hide", ["none", "lens", "mask"])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D", [
    (8, 1, 1500, 20, 20, 64), (16, 1, 448, 16, 16, 64), (43, 2, 2048, 6, 3, 40), (130, 7, 250, 4, 1, 64), (17, 32, 33, 8, 8, 8),
    (64, 4, 256, 12, 3, 56), (16, 3, 2049, 16, 16, 64), (150, 1, 1, 1, 1, 64)])
def test_cross_attention_few_rows_of_many_heads(S, B, Lq, Lk, Hq, Hkv, D, hide):
    """The form with a workgroup of eight wavefronts to a head, at its limits: 129 to 256 heads, 2048 states."""
    announce(f"cross of many heads B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D} {hide}")
    dtype = torch.float16 if (B + Lk) % 2 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(B + Lk)
    q = torch.randn(B, Lq, Hq, D, device="cuda", generator=g).to(dtype)
    kv = torch.randn(B, Lk, 2 * Hkv, D, device="cuda", generator=g).to(dtype)
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:]
    visible = torch.ones(B, Lk, dtype=torch.bool, device="cuda")
    lens = mask = None
    if hide == "lens":
        lens = torch.randint(0, Lk + 1, (B,), device="cuda", generator=g).int()
        lens[1] = 0
        visible = torch.arange(Lk, device="cuda") < lens[:, None]
    if hide == "mask":
        mask = visible = torch.rand(B, Lk, device="cuda", generator=g) < 0.7
        mask[1] = False
    k[~visible], v[~visible] = float("nan"), float("inf")
    near(S.cross_attention(q, k, v, key_lens=lens, mask=mask), q, k, v, visible.cpu().numpy())


@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D", [
    (2, 3, 40, 4, 2, 64), (2, 3, 1500, 4, 2, 128), (1, 200, 70, 4, 1, 96), (1, 200, 3000, 2, 2, 128), (1, 150, 500, 4, 2, 160),
    (1, 4100, 300, 16, 16, 72)])
@pytest.mark.parametrize("mask", [False, True])
def test_cross_attention_over_its_queries(S, B, Lq, Lk, Hq, Hkv, D, mask):
    """The output in the queries' place, in every form."""
    g = torch.Generator(device="cuda").manual_seed(Lk)
    q, k, v = (torch.randn(B, *s, D, device="cuda", generator=g).bfloat16() for s in ((Lq, Hq), (Lk, Hkv), (Lk, Hkv)))
    m = torch.rand(B, Lk, device="cuda", generator=g) < 0.5 if mask else None
    want = S.cross_attention(q, k, v, mask=m)
    announce(f"cross in place B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D}")
    assert torch.equal(S.cross_attention(q, k, v, mask=m, out=q), want) and torch.equal(q, want)


def test_cross_attention_streams_graphs_and_two_at_once(S):
    """Two captured calls with workspaces of their own, replayed against eager results over changing inputs."""
    r = np.random.default_rng(6)
    shapes = [(2, 1, 900, 8, 4, 64), (1, 150, 400, 2, 2, 128)]
    sets = []
    for B, Lq, Lk, Hq, Hkv, D in shapes:
        q = [rows(r, (B, Lq, Hq, D), "fp16") for _ in range(3)]
        k, v = rows(r, (B, Lk, Hkv, D), "fp16"), rows(r, (B, Lk, Hkv, D), "fp16")
        mask = [torch.from_numpy(r.random((B, Lk)) < x).cuda() for x in (0.9, 0.5, 0.0)]
        sets.append((q, k, v, mask, [S.cross_attention(a, k, v, mask=m) for a, m in zip(q, mask)]))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    announce("cross on two streams")
    got = []
    for s, (q, k, v, mask, want) in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append([S.cross_attention(a, k, v, mask=m) for a, m in zip(q, mask)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, s in zip(got, sets) for a, b in zip(g, s[4]))
    graphs = []
    announce("cross in two graphs")
    for q, k, v, mask, want in sets:
        bufs = (q[0].clone(), mask[0].clone(), torch.empty_like(q[0]), S.cross_attention_workspace(q[0], k))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.cross_attention(bufs[0], k, v, mask=bufs[1], out=bufs[2], workspace=bufs[3])
        graphs.append((g, bufs))
    for i in (1, 2, 0, 1):
        for (g, bufs), (q, k, v, mask, want) in zip(graphs, sets):
            bufs[0].copy_(q[i])
            bufs[1].copy_(mask[i])
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bufs[2], s[4][i]) for (g, bufs), s in zip(graphs, sets))


@pytest.mark.parametrize("top", [125.0, 127.99])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D,lens", [
    (8, 1, 1500, 20, 20, 64, False), (1, 4, 1500, 2, 2, 64, False), (16, 3, 900, 16, 16, 96, False), (16, 3, 900, 16, 16, 128, False),
    (1, 8, 20000, 8, 8, 96, False), (1, 200, 900, 2, 2, 128, False), (4, 150, 3001, 2, 1, 128, True), (1, 200, 900, 2, 2, 160, False),
    (1, 200, 900, 2, 2, 256, False), (1, 4100, 300, 16, 16, 64, False), (2, 4097, 256, 8, 8, 128, False)])
def test_cross_attention_large_values_behind_a_low_maximum(S, B, Lq, Lk, Hq, Hkv, D, lens, top):
    """The last state's score is 7.9 (log2) above all others', which the running maximum need not follow, and its values are
    next to the end of bfloat16's range: the result is finite."""
    announce(f"cross of values 2^{top} B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D}")
    r = np.random.default_rng(Lk)
    q = torch.zeros(B, Lq, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros(B, Lk, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = rows(r, (B, Lk, Hkv, D), "bf16")
    k[:, -1, :, 0] = 5.46875
    v[:, -1] = (torch.rand(B, Hkv, D, device="cuda").sub(0.5).sign() * 2.0 ** (top - 7) * 2.0 ** 7).bfloat16()
    n = torch.full((B,), Lk, dtype=torch.int32, device="cuda") if lens else None
    got = S.cross_attention(q, k, v, scale=1.0, key_lens=n)
    # all rows of a head are alike
    assert torch.equal(got, got[:, :1].expand_as(got))
    near(got[:, :1], q[:, :1], k, v, scale=1.0)


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, 3e-39, -1e-38, 6e-38])
@pytest.mark.parametrize("Lq,Lk,H,D,hide", [(2, 333, 2, 64, "none"), (40, 333, 2, 128, "none"), (40, 333, 2, 160, "lens"),
                                            (4100, 300, 16, 72, "none"), (2, 333, 2, 64, "mask")])
def test_cross_attention_smallest_scales_of_large_products(S, Lq, Lk, H, D, hide, scale):
    """Products of 1e37 at scales that bring them to 0 (equal weights) and to scores below 1."""
    announce(f"cross of products of 1e37, scale {scale}, Lq={Lq} D={D} {hide}")
    scale = float(np.float32(scale))
    r = np.random.default_rng(Lq)
    q, k, v = (rows(r, (1, n, H, D), "bf16") for n in (Lq, Lk, Lk))
    q[..., 3], k[..., 3] = 1e19, torch.from_numpy(r.uniform(-1e18, 1e18, (1, Lk, H))).cuda().bfloat16()
    n = Lk - 30 if hide == "lens" else Lk
    visible = np.arange(Lk)[None] < n
    mask = None
    if hide == "mask":
        visible = r.random((1, Lk)) < 0.5
        mask = torch.from_numpy(visible).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda") if hide == "lens" else None
    got = S.cross_attention(q, k, v, scale=scale, key_lens=lens, mask=mask)
    some = slice(0, None, 64) if Lq > 1000 else slice(None)
    near(got[:, some], q[:, some], k, v, visible, scale=scale)


@pytest.mark.parametrize("kind", ["alike", "rising", "negative"])
@pytest.mark.parametrize("dtype,power", [("fp16", 12), ("fp16", 15), ("bf16", 15), ("bf16", 30), ("bf16", 58)])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D", [
    (8, 2, 1500, 20, 20, 64), (1, 4, 1, 2, 2, 64), (16, 3, 900, 16, 16, 96), (1, 8, 20000, 8, 8, 128), (1, 200, 900, 2, 2, 128),
    (1, 200, 900, 2, 2, 160), (1, 200, 900, 2, 2, 256), (1, 4100, 300, 16, 16, 64)])
def test_cross_attention_scores_far_from_zero(S, B, Lq, Lk, Hq, Hkv, D, dtype, power, kind):
    """Scores of 2^24 to 2^122, where a step of float32 is many units of the exponent: those that are alike weigh the same,
    and the others, lower by a sixteenth or more, nothing.  All products and their sums are exact (powers of two times up
    to 16); a score's own rounding is the same for all that are alike.  Row 0 is an ordinary one among them."""
    announce(f"cross of scores far from zero B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D} {dtype} 2^{power} {kind}")
    r = np.random.default_rng(Lk + power)
    q = rows(r, (B, Lq, Hq, D), dtype)
    q[:, 1:] = 2.0 ** power
    steps = {"alike": np.full(Lk, 13), "rising": 1 + 15 * np.arange(Lk) // max(1, Lk - 1), "negative": -16 + 14 * np.arange(Lk) // Lk}[kind]
    steps = torch.from_numpy(steps).cuda()
    k = (steps * 2.0 ** (power - 4))[None, :, None, None].expand(B, Lk, Hkv, D).to(DT[dtype])
    v = rows(r, (B, Lk, Hkv, D), dtype)
    best = steps == steps.max()
    want, mean = (x[:, best].double().mean(1).repeat_interleave(Hq // Hkv, 1)[:, None] for x in (v, v.abs()))
    u = torch.finfo(DT[dtype]).eps / 2
    tol = u * want.abs() + (u + 2 * 2.0 ** -22 + 2 * Lk * 2.0 ** -23) * mean * (1 + 2.0 ** -6) + (2.0 ** -25 if dtype == "fp16" else 0)
    for scale in (0.3, 0.11, 0.71, 0.0625):
        got = S.cross_attention(q, k, v, scale=scale)
        assert ((got[:, 1:].double() - want).abs() <= tol).all(), scale
        q2 = q.clone()
        q2[:, 1:] = 0.25
        assert torch.equal(got[:, 0], S.cross_attention(q2, k, v, scale=scale)[:, 0], ), scale
