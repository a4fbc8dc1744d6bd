"""The router and the W4A16 expert layer on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import awq, moe as O
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


# ---------------------------------------------------------------------- router
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,K,k,score,bias", [
    (1, 1, 8, 1, "softmax", False), (1, 64, 2048, 6, "softmax", False), (3, 8, 64, 8, "sigmoid", True),
    (5, 65, 520, 32, "softmax", True), (17, 128, 1000, 8, "sigmoid", False), (4, 257, 264, 3, "softmax", False),
    (2, 1024, 128, 4, "sigmoid", True), (250, 60, 96, 4, "softmax", False)])
@pytest.mark.parametrize("normalize", [True, False])
def test_route(S, T, E, K, k, score, bias, normalize, dtype):
    announce(f"route T={T} E={E} K={K} k={k} {score} bias={bias} normalize={normalize} {dtype}")
    r = np.random.default_rng(T * 7 + E)
    x = torch.from_numpy(r.standard_normal((T, K))).to(DT[dtype]).cuda()
    w = torch.from_numpy(r.standard_normal((E, K)) / np.sqrt(K)).to(DT[dtype]).cuda()
    b = torch.from_numpy(r.standard_normal(E) * 0.1).float().cuda() if bias else None
    ids, wt = S.moe_route(x, w, k, bias=b, score=score, normalize=normalize)
    rid, rwt = O.route(f64(x), f64(w), k, None if b is None else f64(b), score, normalize)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), rid)
    # one rounding to float32; the float64 logits, scores and sums are 2^-40 off at the most here
    assert (np.abs(f64(wt) - rwt) <= (2.0 ** -24 + 2.0 ** -40) * rwt + 2.0 ** -149).all()


@pytest.mark.parametrize("T,E,K,k", [
    (256, 64, 2048, 6), (256, 128, 1024, 8), (3, 129, 1000, 2), (7, 256, 512, 8),              # one kernel
    (257, 64, 64, 4), (257, 90, 72, 8), (3, 200, 1024, 32), (1, 256, 520, 5), (2, 300, 64, 8), (1, 600, 72, 1),
    (400, 64, 72, 4), (200, 128, 1032, 8), (100, 256, 520, 8), (60, 512, 136, 3), (30, 1000, 264, 16)])      # tiles
def test_route_forms(S, T, E, K, k):
    """Every way in which the logits are formed, with every number of experts a lane holds."""
    announce(f"route T={T} E={E} K={K} k={k}")
    r = np.random.default_rng(T + E)
    dtype = ("bf16", "fp16")[K // 8 % 2]
    x = torch.from_numpy(r.standard_normal((T, K))).to(DT[dtype]).cuda()
    w = torch.from_numpy(r.standard_normal((E, K)) / np.sqrt(K)).to(DT[dtype]).cuda()
    ids, wt = S.moe_route(x, w, k)
    rid, rwt = O.route(f64(x), f64(w), k)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(f64(wt) - rwt) <= (2.0 ** -24 + 2.0 ** -40) * rwt + 2.0 ** -149).all()


def test_route_ties_go_to_the_lower_index(S):
    w = torch.ones(200, 64, dtype=torch.bfloat16, device="cuda")
    w[[70, 150]] *= 2
    x = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    announce("route with ties")
    assert S.moe_route(x, w, 5)[0].tolist() == [[70, 150, 0, 1, 2]] * 2
    assert S.moe_route(-x, w, 5)[0].tolist() == [[0, 1, 2, 3, 4]] * 2


def test_route_of_rows_that_are_not_finite(S):
    """NaN and infinite rows keep valid, different ids and leave the other rows alone."""
    r = np.random.default_rng(2)
    x = torch.from_numpy(r.standard_normal((4, 64))).bfloat16().cuda()
    w = torch.from_numpy(r.standard_normal((70, 64))).bfloat16().cuda()
    want = S.moe_route(x, w, 4)
    y = x.clone()
    y[1, 3], y[2, 5] = float("nan"), float("inf")
    announce("route of rows that are not finite")
    for score in ("softmax", "sigmoid"):
        ids, wt = S.moe_route(y, w, 4, score=score)
        for t in range(4):
            assert len(set(ids[t].tolist())) == 4 and 0 <= min(ids[t].tolist()) and max(ids[t].tolist()) < 70
        assert torch.isnan(wt[1]).all()
        if score == "softmax":
            assert torch.equal(ids[[0, 3]], want[0][[0, 3]]) and torch.equal(wt[[0, 3]], want[1][[0, 3]])


# --------------------------------------------------------------------- experts
def experts(r, E, K, I):
    out = []
    for N, D in ((2 * I, K), (K, I)):
        q = r.integers(0, 16, (E, N, D), dtype=np.uint8)
        s = ((0.5 + r.random((E, N, D // 64))) * 0.25 / np.sqrt(D)).astype(np.float16)
        z = r.integers(0, 16, (E, N, D // 64)).astype(np.float16)
        out.append((q, s, z))
    return out


def device_layer(S, parts):
    return S.AwqMoe(*((awq.pack(q), s, z) for q, s, z in parts))


def check(got, x, parts, ids, wt, act):
    per = [[tuple(a[e] for a in p) for e in range(len(p[0]))] for p in parts]
    y, bound = O.layer(f64(x), *per, ids.cpu().numpy(), f64(wt), act)
    half = torch.finfo(x.dtype).eps / 2
    err = np.abs(f64(got) - y)
    tol = half * (np.abs(y) + bound) + bound + torch.finfo(x.dtype).tiny
    assert got.dtype == x.dtype and (err <= tol).all(), f"{(err / np.maximum(tol, 1e-300)).max()} of the bound"
    # the bound is a worst case over the terms' signs; the errors' squares add up to far less: 2^-12
    # is 16 times what independent roundings of the same terms give
    assert np.linalg.norm(err) <= (half + 2.0 ** -12) * np.linalg.norm(y) + 1e-30


SHAPES = [
    # T, E, K, I, k
    (1, 1, 64, 64, 1), (1, 8, 128, 192, 2), (3, 5, 192, 64, 3), (7, 16, 448, 320, 4), (2, 64, 512, 128, 8),
    (16, 4, 256, 128, 2), (17, 1, 128, 128, 1), (40, 2, 320, 192, 2), (64, 40, 128, 64, 6), (130, 3, 64, 128, 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_expert_layer(S, case, act, dtype):
    T, E, K, I, k = SHAPES[case]
    announce(f"experts T={T} E={E} K={K} I={I} k={k} {act} {dtype}")
    r = np.random.default_rng(case)
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, K))).to(DT[dtype]).cuda()
    ids = torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    wt = torch.from_numpy(r.random((T, k)) + 0.05).float().cuda()
    got = S.awq_moe_forward(layer, x, ids, wt, activation=act)
    check(got, x, parts, ids, wt, act)
    ws = torch.full_like(layer.new_workspace(T, k), 0xFF)
    again = S.awq_moe_forward(layer, x, ids, wt, activation=act, out=torch.full_like(got, float("nan")), workspace=ws)
    assert torch.equal(got, again)


@pytest.mark.parametrize("E,N,K", [(1, 64, 64), (5, 192, 320), (33, 128, 1024)])
def test_packing_on_the_device(S, E, N, K):
    """The bytes of the host's packing, from any strides."""
    announce(f"expert packing E={E} N={N} K={K}")
    r = np.random.default_rng(E)
    q = r.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    s = r.standard_normal((E, N, K // 64)).astype(np.float16)
    z = r.integers(0, 16, (E, N, K // 64)).astype(np.float16)
    want = S._moe_blob((q, s, z), N, K, "cpu")
    dev = [torch.from_numpy(t).cuda() for t in (q, s, z)]
    assert torch.equal(S._moe_blob(dev, N, K, "cuda").cpu(), want)
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in dev]
    assert torch.equal(S._moe_blob(turned, N, K, "cuda").cpu(), want)
    for i, bad in ((2, 16.0), (2, 2.5), (2, -1.0), (2, float("nan")), (1, float("inf"))):
        broken = [t.clone() for t in dev]
        broken[i][0, 5, 0] = bad
        with pytest.raises(ValueError):
            S._moe_blob(broken, N, K, "cuda")


# every way in which a call is split: pairs an expert, pairs in all, tiles of columns, steps of weights
SPLITS = [
    # T, E, K, I, k
    (16, 20, 64, 128, 1), (8, 16, 64, 1152, 2),       # 16 pairs: few steps, and too many for the small form
    (8, 6, 64, 1152, 2), (16, 8, 4160, 192, 1), (16, 9, 64, 64, 1),         # ... taken, in two turns, and too many experts
    (10, 8, 320, 192, 2), (20, 16, 64, 704, 2),       # up to 5 pairs an expert, at most 64: few tiles, many tiles
    (40, 64, 192, 64, 3), (40, 64, 64, 256, 2),       # the same above 64 pairs
    (64, 16, 128, 704, 2), (32, 4, 448, 64, 1),       # 8 pairs an expert: above 64 pairs, and not
    (128, 16, 64, 704, 2), (100, 4, 192, 320, 1),     # 16 and 25 pairs an expert
    (32, 64, 2048, 64, 1), (48, 32, 2048, 64, 4), (128, 32, 2048, 64, 4),   # down products of many tiles
    # many steps of weights: eight wavefronts a workgroup, at up to 5, 8 and 16 pairs an expert (odd groups too)
    (12, 8, 3136, 1344, 2), (32, 8, 3200, 1344, 2), (36, 8, 3136, 1344, 2), (64, 8, 3200, 1408, 2),
    (20, 2, 64, 3136, 1), (33, 3, 64, 3200, 3), (20, 4, 64, 3200, 2),
    (128, 4, 64, 64, 4), (300, 2, 64, 64, 2), (1, 32, 128, 64, 32),   # as many choices as experts
]


@pytest.mark.parametrize("case", range(len(SPLITS)))
def test_expert_layer_splits(S, case):
    T, E, K, I, k = SPLITS[case]
    dtype, act = ("bf16", "fp16")[case % 2], ("silu", "gelu")[case // 2 % 2]
    announce(f"experts split {case}: T={T} E={E} K={K} I={I} k={k} {act} {dtype}")
    r = np.random.default_rng(100 + case)
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, K))).to(DT[dtype]).cuda()
    ids = torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    ids[::7, -1] = -1
    wt = torch.from_numpy(r.random((T, k)) + 0.05).float().cuda()
    check(S.awq_moe_forward(layer, x, ids, wt, activation=act), x, parts, ids, wt, act)


# larger calls: the experts are two experts' matrices in turn and the tokens six rows in
# turn, so that six rows' oracle checks all
LARGE = [
    # T, E, K, I, k: over 24 steps and 1536 tiles of gate and up, at 2, 7 and 13 pairs an expert
    (24, 20, 3136, 1344, 2), (24, 20, 3200, 1408, 2), (70, 20, 3136, 1344, 2), (70, 20, 3200, 1408, 2),
    (130, 20, 3136, 1344, 2), (131, 20, 3200, 1408, 2),
    # over 1024 pairs: 16 and more an expert, 8, and 5
    (300, 4, 64, 64, 4), (260, 64, 64, 192, 4), (260, 64, 3136, 384, 4), (260, 64, 64, 384, 4), (300, 4, 64, 3136, 4),
    (260, 64, 1024, 64, 4), (130, 128, 64, 64, 8), (130, 128, 64, 128, 8), (130, 128, 3136, 192, 8),
    (130, 128, 64, 192, 8), (130, 128, 64, 3136, 8), (130, 128, 512, 64, 8), (150, 256, 64, 64, 8),
    (150, 256, 64, 3136, 8), (150, 256, 256, 64, 8),
    (100, 20, 64, 1344, 3), (12, 4, 64, 3136, 1), (40, 16, 64, 3136, 2),    # at most 1024 pairs
    # as many as a call takes, and 1024 of a kind
    (128, 1024, 64, 64, 32), (4096, 3, 64, 64, 1), (1024, 1, 64, 64, 1), (32, 1024, 64, 64, 32),
]


@pytest.mark.parametrize("case", range(len(LARGE)))
def test_expert_layer_of_many_pairs_or_weights(S, case):
    T, E, K, I, k = LARGE[case]
    dtype, act = ("bf16", "fp16")[case % 2], ("silu", "gelu")[case // 2 % 2]
    announce(f"experts large {case}: T={T} E={E} K={K} I={I} k={k} {act} {dtype}")
    r = np.random.default_rng(200 + case)
    two = min(E, 2)
    parts = experts(r, two, K, I)
    turns = torch.arange(E, device="cuda") % two
    layer = S.AwqMoe(*(tuple(torch.from_numpy(t).cuda()[turns] for t in (awq.pack(q), s, z)) for q, s, z in parts))
    turn = np.arange(T) % 6
    x = torch.from_numpy(r.standard_normal((6, K))).to(DT[dtype]).cuda()[turn]
    kinds = r.integers(0, two, (6, k))[turn]
    ids = torch.from_numpy((kinds + two * r.integers(0, E // two, (T, k))).astype(np.int32)).cuda()
    wt = torch.from_numpy(r.random((6, k)) + 0.05).float().cuda()[turn]
    got = S.awq_moe_forward(layer, x, ids, wt, activation=act)
    check(got[:6], x[:6], parts, ids[:6] % two, wt[:6], act)
    assert torch.equal(got, got[:6][turn])


def test_expert_layer_all_tokens_to_one_expert(S):
    r = np.random.default_rng(29)
    E, K, I, T = 6, 128, 192, 90
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, K))).half().cuda()
    ids = torch.full((T, 1), 4, dtype=torch.int32, device="cuda")
    ids[50] = 1
    wt = torch.ones(T, 1, device="cuda")
    announce("experts: 89 tokens to one expert")
    check(S.awq_moe_forward(layer, x, ids, wt), x, parts, ids, wt, "silu")


def test_expert_layer_ids_outside_and_twice(S):
    r = np.random.default_rng(30)
    E, K, I, T, k = 4, 128, 64, 9, 3
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, K))).bfloat16().cuda()
    ids = torch.from_numpy(r.integers(-1, E + 1, (T, k)).astype(np.int32)).cuda()
    ids[0] = 2                                   # the same expert three times
    ids[1] = -1                                  # no expert at all
    ids[2, 0], ids[2, 1] = 2 ** 31 - 1, -(2 ** 31)
    wt = torch.from_numpy(r.standard_normal((T, k))).float().cuda()
    wt[1] = float("nan")                         # weights of choices that do not count
    announce("experts with ids outside and twice")
    got = S.awq_moe_forward(layer, x, ids, wt)
    assert not got[1].any()
    check(got[[0] + list(range(2, T))], x[[0] + list(range(2, T))], parts, ids[[0] + list(range(2, T))],
          wt[[0] + list(range(2, T))], "silu")
    ids.fill_(E)
    assert not S.awq_moe_forward(layer, x, ids, wt).any()


@pytest.mark.parametrize("T", [5, 30, 70, 600])
def test_expert_layer_of_padding_rows(S, T):
    """Batches of which no token, or only the last, has an expert here."""
    r = np.random.default_rng(31)
    E, K, I, k = 9, 128, 64, 2
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, K))).bfloat16().cuda()
    x[:-1] = float("nan")
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    ids[::2, 1] = E
    wt = torch.ones(T, k, device="cuda")
    out = torch.full_like(x, float("nan"))
    announce(f"experts: {T} rows of padding")
    assert not S.awq_moe_forward(layer, x, ids, wt, out=out).any()
    ids[-1, 0] = 8
    got = S.awq_moe_forward(layer, x, ids, wt, out=torch.full_like(x, float("nan")))
    assert not got[:-1].any()
    check(got[-1:], x[-1:], parts, ids[-1:], wt[-1:], "silu")


def test_expert_layer_rows_do_not_touch_each_other(S):
    """A token of NaN or infinities spoils its own row only, and a token alone gives its row up to the order of sums."""
    r = np.random.default_rng(31)
    E, K, I, T, k = 3, 192, 128, 21, 2
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    for dtype in DT.values():
        x = torch.from_numpy(r.standard_normal((T, K))).to(dtype).cuda()
        ids = torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
        wt = torch.from_numpy(r.random((T, k))).float().cuda()
        announce(f"experts: rows apart {dtype}")
        want = S.awq_moe_forward(layer, x, ids, wt)
        y = x.clone()
        y[4, 7], y[11] = float("nan"), float("inf")
        got = S.awq_moe_forward(layer, y, ids, wt)
        rest = [t for t in range(T) if t not in (4, 11)]
        assert not torch.isfinite(got[[4, 11]]).any() and torch.equal(got[rest], want[rest])
        for t in (0, 20):
            one = slice(t, t + 1)
            check(S.awq_moe_forward(layer, x[one], ids[one], wt[one]), x[one], parts, ids[one], wt[one], "silu")


def test_expert_layer_large_gated_products(S):
    """h beyond fp16's range on its way to an output inside it."""
    r = np.random.default_rng(32)
    E, K, I = 2, 64, 64
    parts = experts(r, E, K, I)
    parts[0][1][:] *= np.float16(64)
    parts[1][1][:] *= np.float16(2.0 ** -9)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((2, K)) * 8).half().cuda()
    ids, wt = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"), torch.ones(2, 1, device="cuda")
    announce("experts with large gated products")
    check(S.awq_moe_forward(layer, x, ids, wt), x, parts, ids, wt, "silu")


def test_route_and_experts_in_a_graph(S):
    """Router and experts captured together and replayed on new tokens equal the eager calls, as do two
    graphs that share a workspace."""
    r = np.random.default_rng(33)
    E, K, I, T, k = 6, 128, 64, 5, 2
    layer = device_layer(S, experts(r, E, K, I))
    w = torch.from_numpy(r.standard_normal((E, K))).bfloat16().cuda()
    ws = layer.new_workspace(T, k)
    xs = [torch.zeros(T, K, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(x, ws):
        ids, wt = S.moe_route(x, w, k)
        return S.awq_moe_forward(layer, x, ids, wt, workspace=ws)

    announce("router and experts: capture")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in xs:
            step(x, ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x, ws))
        graphs.append(g)
    for i in range(6):
        for x in xs:
            x.copy_(torch.from_numpy(r.standard_normal((T, K))).bfloat16())
        for g in graphs:
            g.replay()
        want = [step(x, None) for x in xs]
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert torch.equal(o, v), f"replay {i}"


@pytest.mark.parametrize("power", [(70, 70), (-70, -70), (120, 5), (-120, -5), (0, 100)])
@pytest.mark.parametrize("T,E,K,k", [(3, 64, 512, 3), (256, 100, 136, 4), (3, 300, 512, 3), (100, 256, 520, 2)])
def test_route_over_the_range_of_bf16(S, T, E, K, k, power):
    """Products past float32's largest number and below its normal range, in every form in which the logits are formed."""
    announce(f"route T={T} E={E} K={K} k={k}, rows times 2^{power[0]} and matrix times 2^{power[1]}")
    r = np.random.default_rng(T + E + K)
    x = torch.from_numpy(r.standard_normal((T, K)) * 2.0 ** power[0]).bfloat16().cuda()
    w = torch.from_numpy(r.standard_normal((E, K)) / np.sqrt(K) * 2.0 ** power[1]).bfloat16().cuda()
    for score in ("softmax", "sigmoid"):
        ids, wt = S.moe_route(x, w, k, score=score)
        with np.errstate(over="ignore"):
            rid, rwt = O.route(f64(x), f64(w), k, None, score)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert (np.abs(f64(wt) - rwt) <= (2.0 ** -24 + 2.0 ** -40) * rwt + 2.0 ** -149).all()


def test_route_of_saturated_scores(S):
    """A sigmoid of 38 and one of 40 are both 1 in float64: without a bias the order is the logits', with one
    (zeros too) it is the scores' and the lower index goes first.  The weights are the scores' either way."""
    w = torch.zeros(70, 64, dtype=torch.bfloat16, device="cuda")
    w[5, 0], w[66, 0], w[7, 1] = 38, 40, 1
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    announce("route of saturated scores")
    ids, wt = S.moe_route(x, w, 3, score="sigmoid", normalize=False)
    assert ids.tolist() == [[66, 5, 0]] * 2 and wt.tolist() == [[1, 1, 0.5]] * 2
    ids, wt = S.moe_route(x, w, 3, bias=torch.zeros(70, device="cuda"), score="sigmoid", normalize=False)
    assert ids.tolist() == [[5, 66, 0]] * 2 and wt.tolist() == [[1, 1, 0.5]] * 2


def wide_range_experts(r, E):
    """Experts of 128 x 64 whose gates take channel 0 alone out of the first group, and whose ups take nothing of it."""
    (q, s, z), (qd, sd, zd) = experts(r, E, 128, 64)
    z[..., 0] = 8
    q[:, :64, 0] = r.integers(9, 16, (E, 64))
    q[:, 64:, 0] = 8
    return (q, s, z), (qd, sd, zd)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,E", [(1, 1), (3, 2), (20, 8), (40, 3), (90, 2)])
def test_expert_layer_over_float32s_range(S, T, E, act):
    """Rows up to 2^125 and gated products near 2^118, past which 128 + 15 times 64 of them is no float32 number any
    more, where neither the gate's and the up's results nor the output are."""
    announce(f"experts over float32's range, T={T} E={E} {act}")
    r = np.random.default_rng(T)
    parts = wide_range_experts(r, E)
    parts[0][1][..., 0] = 2.0 ** -11
    parts[1][1][:] = (r.choice([-1.0, 1.0], parts[1][1].shape) * 2.0 ** -20).astype(np.float16)
    layer = device_layer(S, parts)
    x = r.standard_normal((T, 128))
    x[:, :64] = 0
    x[:, 0] = 2.0 ** 125
    x = torch.from_numpy(x).bfloat16().cuda()
    ids = torch.from_numpy(r.integers(0, E, (T, 1)).astype(np.int32)).cuda()
    wt = torch.ones(T, 1, device="cuda")
    got = S.awq_moe_forward(layer, x, ids, wt, activation=act)
    with np.errstate(over="ignore"):
        check(got, x, parts, ids, wt, act)


@pytest.mark.parametrize("T", [1, 20])
def test_expert_layer_of_the_largest_gated_products(S, T):
    """h = 1023 x 2^118 is a float32 number, and the bf16 number next to it is not."""
    r = np.random.default_rng(5)
    (q, s, z), (qd, sd, zd) = wide_range_experts(r, 4)
    s[:], z[:], q[:] = 1.0, 8, 8
    q[:, :64, 0], q[:, :64, 1], q[:, 64:, 64] = 9, 7, 9          # gate: x0 - x1, up: x64
    sd[:] = 2.0 ** -24
    layer = device_layer(S, ((q, s, z), (qd, sd, zd)))
    x = torch.zeros(T, 128)
    x[:, 0], x[:, 1], x[:, 64] = 2.0 ** 70, 2.0 ** 60, 2.0 ** 58
    x = x.bfloat16().cuda()
    ids, wt = (torch.arange(T, dtype=torch.int32, device="cuda") % 4)[:, None], torch.ones(T, 1, device="cuda")
    announce(f"experts of the largest gated products, T={T}")
    with np.errstate(over="ignore"):
        check(S.awq_moe_forward(layer, x, ids, wt), x, ((q, s, z), (qd, sd, zd)), ids, wt, "silu")


@pytest.mark.parametrize("T,E", [(1, 1), (20, 8), (90, 2)])
def test_expert_layer_of_small_rows(S, T, E):
    """Gated products near 2^-118, whose second pieces are near the end of float32's range."""
    announce(f"experts of small rows, T={T} E={E}")
    r = np.random.default_rng(T + 7)
    parts = experts(r, E, 128, 64)
    for p in parts:
        p[1][:] = (0.5 + r.random(p[1].shape)).astype(np.float16)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, 128)) * 2.0 ** -64).bfloat16().cuda()
    ids = torch.from_numpy(r.integers(0, E, (T, 1)).astype(np.int32)).cuda()
    wt = torch.ones(T, 1, device="cuda")
    check(S.awq_moe_forward(layer, x, ids, wt), x, parts, ids, wt, "silu")


@pytest.mark.parametrize("T,k", [(5, 3), (16, 1), (1, 16), (2, 8)])
def test_expert_layer_of_few_pairs_outside_and_twice(S, T, k):
    """Experts named twice, three times and not at all by a call of up to 16 pairs."""
    r = np.random.default_rng(34)
    E, K, I = 4, 128, 64
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    for dtype in DT.values():
        x = torch.from_numpy(r.standard_normal((T, K))).to(dtype).cuda()
        ids = torch.from_numpy(r.integers(-1, E + 1, (T, k)).astype(np.int32)).cuda()
        ids[0] = 2
        if T > 2:
            ids[1], ids[2, 0] = -1, 2 ** 31 - 1
        wt = torch.from_numpy(r.standard_normal((T, k))).float().cuda()
        wt[(ids < 0) | (ids >= E)] = float("nan")
        announce(f"experts: {T} tokens of {k} choices, outside and twice, {dtype}")
        got = S.awq_moe_forward(layer, x, ids, wt)
        check(got, x, parts, ids, wt, "silu")
        if T > 2:
            assert not got[1].any()


def test_route_and_experts_on_two_streams(S):
    r = np.random.default_rng(35)
    E, K, I, T, k = 6, 128, 64, 40, 2
    layer = device_layer(S, experts(r, E, K, I))
    w = torch.from_numpy(r.standard_normal((E, K))).bfloat16().cuda()
    xs = [torch.from_numpy(r.standard_normal((T, K))).bfloat16().cuda() for _ in range(2)]

    def step(x):
        ids, wt = S.moe_route(x, w, k)
        return S.awq_moe_forward(layer, x, ids, wt)

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    announce("router and experts on two streams")
    streams, outs = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(step(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,K,k", [(65535, 3, 8, 2), (2, 4, 1 << 20, 2), (1, 1024, 8, 32), (24576, 1, 8, 1), (300, 1024, 8, 1)])
def test_route_at_the_largest_sizes(S, T, E, K, k, dtype):
    announce(f"route T={T} E={E} K={K} k={k} {dtype}")
    r = np.random.default_rng(K)
    x = torch.from_numpy(r.standard_normal((T, K))).to(DT[dtype]).cuda()
    w = torch.from_numpy(r.standard_normal((E, K)) / np.sqrt(K)).to(DT[dtype]).cuda()
    ids, wt = S.moe_route(x, w, k)
    rid, rwt = O.route(f64(x), f64(w), k)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(f64(wt) - rwt) <= (2.0 ** -24 + 2.0 ** -40) * rwt + 2.0 ** -149).all()


@pytest.mark.parametrize("T,E,K,I,k", [(1, 2, 32768, 64, 2), (20, 2, 32768, 64, 1), (1, 2, 64, 16384, 2), (40, 3, 64, 16384, 2)])
def test_expert_layer_of_long_rows(S, T, E, K, I, k):
    announce(f"experts of long rows T={T} E={E} K={K} I={I} k={k}")
    r = np.random.default_rng(K + I)
    parts = experts(r, E, K, I)
    layer = device_layer(S, parts)
    for dtype in DT.values():
        x = torch.from_numpy(r.standard_normal((T, K))).to(dtype).cuda()
        ids = torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
        wt = torch.from_numpy(r.random((T, k)) + 0.05).float().cuda()
        check(S.awq_moe_forward(layer, x, ids, wt), x, parts, ids, wt, "silu")


@pytest.mark.parametrize("T", [1, 20, 90])
def test_expert_layer_of_subnormal_rows(S, T):
    """fp16 rows below 2^-14 under large scales."""
    announce(f"experts of subnormal fp16 rows, T={T}")
    r = np.random.default_rng(T + 9)
    parts = experts(r, 3, 128, 64)
    for p in parts:
        p[1][:] = (p[1].astype(np.float64) * 2.0 ** 12).astype(np.float16)
    layer = device_layer(S, parts)
    x = torch.from_numpy(r.standard_normal((T, 128)) * 2.0 ** -18).half().cuda()
    ids = torch.from_numpy(r.integers(0, 3, (T, 1)).astype(np.int32)).cuda()
    wt = torch.ones(T, 1, device="cuda")
    check(S.awq_moe_forward(layer, x, ids, wt), x, parts, ids, wt, "silu")
