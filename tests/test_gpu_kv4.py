"""The MXFP4 key/value cache and its attention on the GPU against the float64
oracle: every value of the cache bit for bit, attention within the bounds of
its float32 arithmetic."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
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
    x[..., ::29] *= 9.0
    return torch.from_numpy(x).to(DT[dtype]).cuda()


# ------------------------------------------------------------ append and read
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (37, 3, 128, 16), (70, 2, 256, 64), (129, 5, 64, 256)])
def test_append_then_read(S, T, H, D, page, dtype):
    announce(f"kv4 append/read T={T} H={H} D={D} page={page} {dtype}")
    r = np.random.default_rng(T + D)
    pages = T // page + 3
    cache = S.Kv4Cache(pages, page, H, D)
    k, v = rows(r, (T, H, D), dtype), rows(r, (T, H, D), dtype, 0.01)
    slots = torch.from_numpy(r.permutation(pages * page)[:T].astype(np.int32)).cuda()
    S.kv4_append(cache, k, v, slots)
    for out in (torch.bfloat16, torch.float32):
        gk, gv = S.kv4_read(cache, slots, dtype=out)
        assert gk.dtype == out and np.array_equal(f64(gk), O.values(f64(k))) and np.array_equal(f64(gv), O.values(f64(v)))
    # slots that were not named still hold what a new cache holds
    rest = np.setdiff1d(np.arange(pages * page), slots.cpu().numpy()).astype(np.int32)
    gk, gv = S.kv4_read(cache, torch.from_numpy(rest).cuda())
    assert not gk.any() and not gv.any()


@pytest.mark.parametrize("run", [1, 15, 16, 17, 40, 64])
@pytest.mark.parametrize("first", [0, 5, 16])
def test_append_runs_of_slots(S, run, first):
    """Rows that fill units of 16 tokens whole, in part, and from the middle, after others' rows were there."""
    announce(f"kv4 append of {run} rows from slot {first}")
    r = np.random.default_rng(run * 100 + first)
    H, D = 2, 128
    cache = S.Kv4Cache(6, 16, H, D)
    k0, v0 = rows(r, (96, H, D), "bf16"), rows(r, (96, H, D), "bf16")
    S.kv4_append(cache, k0, v0, torch.arange(96, dtype=torch.int32, device="cuda"))
    k, v = rows(r, (run, H, D), "bf16"), rows(r, (run, H, D), "bf16")
    S.kv4_append(cache, k, v, torch.arange(first, first + run, dtype=torch.int32, device="cuda"))
    gk, gv = S.kv4_read(cache, torch.arange(96, dtype=torch.int32, device="cuda"))
    for got, old, new in ((gk, k0, k), (gv, v0, v)):
        want = O.values(f64(old))
        want[first:first + run] = O.values(f64(new))
        assert np.array_equal(f64(got), want)


def test_append_takes_rows_where_they_are_and_skips_slots_outside(S):
    r = np.random.default_rng(8)
    T, H, D, page = 21, 2, 64, 16
    qkv = rows(r, (T, 8, D), "bf16")
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    cache = S.Kv4Cache(2, page, H, D)
    slots = torch.from_numpy(r.permutation(32)[:T].astype(np.int32)).cuda()
    slots[3], slots[7], slots[9] = -1, 32, 2 ** 31 - 1
    announce("kv4 append of strided rows, three of them to no slot")
    S.kv4_append(cache, k, v, slots)
    gk, gv = S.kv4_read(cache, slots)
    for got, x in ((gk, k), (gv, v)):
        want = O.values(f64(x))
        want[[3, 7, 9]] = 0
        assert np.array_equal(f64(got), want)
    # per-head layout [H, T, D]
    t = k.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    S.kv4_append(cache, t, v, slots)
    assert torch.equal(S.kv4_read(cache, slots)[0], gk)


def test_append_edge_values(S):
    """Zeros of both signs, the smallest and largest values, ties, infinities and NaN."""
    x = np.zeros((8, 1, 64))
    x[0, 0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    x[0, 0, 32:40] = [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -7.0]
    x[1, 0, 0], x[1, 0, 33] = -0.0, 2.0 ** -133
    x[2, 0, :3] = [3.0e38, -1.0e38, 1.0]
    x[3, 0, 5], x[3, 0, 40] = np.inf, -np.inf
    x[4, 0, 63] = np.nan
    x[5, 0, :4] = [2.0 ** -126, 2.0 ** -127, -2.0 ** -128, 2.0 ** -130]
    x[6, 0, :] = 1.9921875
    k = torch.from_numpy(x).to(torch.bfloat16).cuda()
    cache = S.Kv4Cache(1, 16, 1, 64)
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    announce("kv4 append of edge values")
    S.kv4_append(cache, k, k, slots)
    for got in S.kv4_read(cache, slots, dtype=torch.float32):
        want = O.values(f64(k))
        assert np.array_equal(f64(got), want, equal_nan=True)
        assert not np.signbit(f64(got)[1]).any()


# ------------------------------------------------------------------- attention
class Batch:
    """Sequences scattered over a cache whose every other slot holds large values."""

    def __init__(self, S, seed, lens, H, D, page, dtype, spare=2, width_more=0):
        r = np.random.default_rng(seed)
        per = [-(-n // page) for n in lens]
        self.pages = sum(per) + spare
        order = r.permutation(self.pages).astype(np.int32)
        width = max(1, max(per)) + width_more
        table = r.integers(0, self.pages, (len(lens), width)).astype(np.int32)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.cache = S.Kv4Cache(self.pages, page, H, D)
        n = self.pages * page
        k, v = rows(r, (n, H, D), dtype), rows(r, (n, H, D), dtype)
        used = np.zeros(n, bool)
        for b, m in enumerate(lens):
            t = np.arange(m)
            used[table[b, t // page] * page + t % page] = True
        k[torch.from_numpy(~used).cuda()] = float("inf")    # old rows behind a sequence's end
        v[torch.from_numpy(~used).cuda()] = float("nan")
        S.kv4_append(self.cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
        kv, vv = (O.values(f64(t)) for t in (k, v))
        self.k, self.v = [], []
        for b, m in enumerate(lens):
            t = np.arange(m)
            s = table[b, t // page] * page + t % page
            self.k.append(kv[s])
            self.v.append(vv[s])
        self.lens, self.D, self.dtype = lens, D, dtype
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.r = r

    def queries(self, Q, Hq, scale=1.0):
        return torch.from_numpy(self.r.standard_normal((len(self.lens), Q, Hq, self.D)) * scale).to(DT[self.dtype]).cuda()


def check(got, q, b, scale):
    """|error| <= half a step of the output, plus what float32 does to it: a
    score is a sum of D products in any order, a scaling and a difference,
    (D + 4) 2^-24 of its terms, twice (a piece may be joined to another's
    maximum); exp2 and the joins 2^-20; a weight has 2^-17 of its own; the
    sum over n tokens n 2^-24.  All of it on sum p |v|, and once more for the
    denominator."""
    out, mass, largest, terms = O.attend(f64(q), b.k, b.v, b.lens, scale)
    D = q.shape[-1]
    u = 2.0 ** -24
    rel = 2 * (2 * (D + 4) * u * largest + 2.0 ** -20 + 2.0 ** -17 + terms * u)
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(out) * (1 + rel) + rel * mass + torch.finfo(q.dtype).tiny
    err = np.abs(f64(got) - out)
    assert got.dtype == q.dtype and (err <= tol).all(), f"{(err / np.maximum(tol, 1e-300)).max()} of the bound"


CASES = [
    # lens, Q, Hq, Hkv, D, page, dtype
    ([1], 1, 1, 1, 64, 16, "bf16"),
    ([1, 0, 2], 1, 4, 2, 128, 16, "fp16"),
    ([15, 16, 17, 31, 32, 33, 127, 128, 129], 1, 8, 2, 128, 16, "bf16"),
    ([15, 16, 17, 31, 32, 33, 127, 128, 129], 1, 8, 2, 128, 128, "fp16"),
    ([700], 1, 32, 8, 128, 64, "bf16"),
    ([513, 3, 0, 1000, 64, 90], 1, 5, 1, 64, 32, "fp16"),
    ([300, 1], 1, 32, 2, 256, 16, "bf16"),
    ([257, 40], 1, 16, 16, 64, 256, "bf16"),
    ([3000, 2999], 1, 17, 1, 128, 32, "fp16"),          # 17 rows: two tiles
    ([640, 5], 3, 10, 5, 128, 16, "bf16"),              # drafted tokens
    ([100, 2, 0, 1], 5, 8, 1, 64, 32, "fp16"),          # 40 rows: two blocks, sequences shorter than Q
    ([90], 7, 32, 2, 256, 64, "bf16"),                  # 112 rows
    ([40] * 150, 1, 2, 1, 64, 16, "bf16"),              # more sequences than lanes
    ([1, 2000] * 70, 1, 4, 4, 64, 64, "fp16"),
    ([20000], 1, 8, 1, 128, 256, "bf16"),               # one sequence over many workgroups
    ([333, 9], 1, 9, 1, 64, 16, "bf16"), ([333, 9], 1, 16, 1, 128, 16, "fp16"), ([50], 4, 4, 1, 128, 16, "bf16"),
    ([200, 31], 1, 12, 1, 64, 32, "fp16"), ([130], 3, 4, 1, 256, 16, "fp16"), ([90, 300], 8, 3, 1, 256, 64, "fp16"),
    ([200], 6, 16, 4, 64, 16, "bf16"), ([100], 1, 8, 8, 256, 16, "fp16"), ([64, 70], 33, 2, 1, 64, 16, "bf16"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(S, case):
    lens, Q, Hq, H, D, page, dtype = CASES[case]
    announce(f"kv4 attention case {case}: B={len(lens)} max={max(lens)} Q={Q} Hq={Hq}/{H} D={D} page={page} {dtype}")
    b = Batch(S, case, lens, H, D, page, dtype)
    q = b.queries(Q, Hq)
    got = S.kv4_attention(b.cache, q, b.table, b.seq_lens)
    check(got, q, b, D ** -0.5)
    again = S.kv4_attention(b.cache, q, b.table, b.seq_lens, out=torch.full_like(got, float("nan")),
                            workspace=torch.full_like(S.kv4_attention_workspace(b.cache, q), 0xFF))
    assert torch.equal(got, again)


def test_attention_peaked_and_negative_scales(S):
    b = Batch(S, 50, [400, 77], 2, 128, 16, "fp16")
    for scale, size in ((0.7, 3.0), (-0.2, 1.0), (0.0, 1.0)):
        announce(f"kv4 attention scale {scale}")
        q = b.queries(1, 8, size)
        check(S.kv4_attention(b.cache, q, b.table, b.seq_lens, scale=scale), q, b, scale)


def test_attention_of_strided_queries_and_a_wide_table(S):
    b = Batch(S, 51, [130, 0, 45], 2, 64, 32, "bf16", width_more=40)
    qkv = b.queries(2, 12)
    q = qkv[:, :, 3:7]
    announce("kv4 attention with strided queries")
    got = S.kv4_attention(b.cache, q, b.table, b.seq_lens)
    check(got, q, b, 0.125)
    assert torch.equal(got, S.kv4_attention(b.cache, q.contiguous(), b.table, b.seq_lens))


def test_attention_hides_bad_pages_and_clamps_lengths(S):
    page = 16
    b = Batch(S, 52, [100, 64, 48], 1, 64, page, "bf16")
    q = b.queries(1, 4)
    width = b.table.shape[1]
    lens = b.seq_lens.clone()
    lens[0], lens[2] = 2 ** 31 - 1, -5
    table = b.table.clone()
    t = np.arange(width * page)
    # the long row: as far as the table goes, pages that exist only where the sequence had some
    table[0, 7:] = -1
    table[0, 2], table[1, 1] = b.pages, -(2 ** 31)
    announce("kv4 attention with bad pages, a length past the table and a negative one")
    got = f64(S.kv4_attention(b.cache, q, table, lens))
    seen0 = [i for i in t if i // page < 7 and i // page != 2 and i < 100]
    tail = list(range(100, 112))                # the seventh page's old rows: not finite, so the row is not either
    assert tail and not np.isfinite(got[0]).any()
    assert (got[2] == 0).all()
    k, v = b.k[1], b.v[1]
    keep = [i for i in range(64) if i // page != 1]
    bb = type("B", (), dict(k=[k[keep]], v=[v[keep]], lens=[len(keep)]))
    check(torch.from_numpy(got[1:2]).to(torch.bfloat16), q[1:2], bb, 0.125)
    lens[0] = 100
    got = S.kv4_attention(b.cache, q, table, lens)
    bb = type("B", (), dict(k=[b.k[0][seen0]], v=[b.v[0][seen0]], lens=[len(seen0)]))
    check(got[:1], q[:1], bb, 0.125)
    table.fill_(-1)
    assert not S.kv4_attention(b.cache, q, table, lens).any()


def test_attention_carries_nan_and_infinity(S):
    """A NaN in a sequence's cache, or in one query head, reaches the rows that see it and no others."""
    b = Batch(S, 53, [50, 50], 2, 64, 16, "bf16")
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    v[0, 1, 3] = float("nan")
    slot = (b.table[0, 0] * 16 + 7).reshape(1).to(torch.int32)
    announce("kv4 attention over a NaN")
    S.kv4_append(b.cache, k, v, slot)
    q = b.queries(1, 4)
    q[1, 0, 0, 5] = float("nan")
    got = f64(S.kv4_attention(b.cache, q, b.table, b.seq_lens))
    assert np.isnan(got[0, 0, 2:, :32]).all() and np.isfinite(got[0, 0, :2]).all() and np.isfinite(got[0, 0, 2:, 32:]).all()
    assert np.isnan(got[1, 0, 0]).all() and np.isfinite(got[1, 0, 1:]).all()


def test_attention_slots_past_32_bit_offsets(S):
    """A cache of more than 4 GiB: pages at its far end."""
    H, D, page = 8, 128, 256
    pages = (1 << 32) // (H * page * (D + 8)) + 8
    announce(f"kv4 cache of {pages} pages, {pages * H * page * (D + 8) / 2 ** 30:.2f} GiB")
    cache = S.Kv4Cache(pages, page, H, D)
    r = np.random.default_rng(9)
    n = 300
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    t = np.arange(n)
    slots = torch.from_numpy((table.cpu().numpy()[0][t // page].astype(np.int64) * page + t % page).astype(np.int32)).cuda()
    k, v = rows(r, (n, H, D), "bf16"), rows(r, (n, H, D), "bf16")
    S.kv4_append(cache, k, v, slots)
    assert np.array_equal(f64(S.kv4_read(cache, slots)[1]), O.values(f64(v)))
    q = torch.from_numpy(r.standard_normal((1, 1, 16, D))).to(torch.bfloat16).cuda()
    got = S.kv4_attention(cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    bb = type("B", (), dict(k=[O.values(f64(k))], v=[O.values(f64(v))], lens=[n]))
    check(got, q, bb, D ** -0.5)


def test_attention_over_shared_pages(S):
    """Sequences of one prompt: every row of the table names the same pages, far more of them than a register holds."""
    r = np.random.default_rng(12)
    n, H, D, page, B = 4000, 8, 64, 16, 64
    cache = S.Kv4Cache(n // page, page, H, D)
    k, v = rows(r, (n, H, D), "bf16"), rows(r, (n, H, D), "bf16")
    order = r.permutation(n // page).astype(np.int32)
    t = np.arange(n)
    S.kv4_append(cache, k, v, torch.from_numpy((order[t // page] * page + t % page).astype(np.int32)).cuda())
    lens = [int(x) for x in r.integers(3000, n + 1, B)]
    table = torch.from_numpy(np.tile(order, (B, 1))).cuda()
    q = torch.from_numpy(r.standard_normal((B, 1, H, D))).to(torch.bfloat16).cuda()
    announce("kv4 attention over shared pages")
    got = S.kv4_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    bb = type("B", (), dict(k=[O.values(f64(k))] * B, v=[O.values(f64(v))] * B, lens=lens))
    check(got, q, bb, D ** -0.5)


def test_attention_of_queries_that_are_not_finite(S):
    for dtype in DT:
        b = Batch(S, 55, [70, 33], 1, 128, 16, dtype)
        q = b.queries(1, 5)
        want = f64(S.kv4_attention(b.cache, q, b.table, b.seq_lens))
        q[0, 0, 1, 9], q[1, 0, 4, 2] = float("inf"), float("nan")
        announce(f"kv4 attention of queries that are not finite, {dtype}")
        got = f64(S.kv4_attention(b.cache, q, b.table, b.seq_lens))
        assert np.isnan(got[0, 0, 1]).all() and np.isnan(got[1, 0, 4]).all()
        got[0, 0, 1], got[1, 0, 4] = want[0, 0, 1], want[1, 0, 4]
        assert np.array_equal(got, want)


def test_two_graphs_share_a_workspace(S):
    bs = [Batch(S, 56 + i, [900, 5], 2, 128, 32, "bf16") for i in range(2)]
    qs = [b.queries(1, 8) for b in bs]
    ws = S.kv4_attention_workspace(bs[0].cache, qs[0])
    outs, graphs = [torch.empty_like(q) for q in qs], []
    announce("kv4 attention: two graphs on one workspace")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for b, q, o in zip(bs, qs, outs):
            S.kv4_attention(b.cache, q, b.table, b.seq_lens, out=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for b, q, o in zip(bs, qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.kv4_attention(b.cache, q, b.table, b.seq_lens, out=o, workspace=ws)
        graphs.append(g)
    for i in range(4):
        for b, q in zip(bs, qs):
            q.copy_(b.queries(1, 8))
        for g in graphs:
            g.replay()
        want = [S.kv4_attention(b.cache, q, b.table, b.seq_lens) for b, q in zip(bs, qs)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {i}"


def test_append_and_attention_in_a_graph(S):
    """A decode step captured once and replayed as the sequences grow equals the eager calls."""
    page, H, D, B = 16, 2, 64, 3
    r = np.random.default_rng(11)
    lens = torch.tensor([5, 0, 30], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(r.permutation(12).reshape(B, 4).astype(np.int32)).cuda()
    caches = [S.Kv4Cache(12, page, H, D) for _ in range(2)]
    k0, v0 = rows(r, (192, H, D), "bf16"), rows(r, (192, H, D), "bf16")
    for c in caches:
        S.kv4_append(c, k0, v0, torch.arange(192, dtype=torch.int32, device="cuda"))
    q, k, v = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device="cuda") for h in (4, H, H))
    out = torch.empty_like(q)
    ws = S.kv4_attention_workspace(caches[0], q)

    def step(c, lens, out, ws):
        at = lens.long()
        slots = (table.gather(1, (at // page)[:, None])[:, 0] * page + at % page).to(torch.int32)
        S.kv4_append(c, k[:, 0], v[:, 0], slots)
        lens += 1
        return S.kv4_attention(c, q, table, lens, out=out, workspace=ws)

    announce("kv4 decode step: capture")
    glens = lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(caches[0], glens, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    S.kv4_append(caches[0], k0, v0, torch.arange(192, dtype=torch.int32, device="cuda"))
    glens.copy_(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], glens, out, ws)
    glens.copy_(lens)
    S.kv4_append(caches[0], k0, v0, torch.arange(192, dtype=torch.int32, device="cuda"))
    elens = lens.clone()
    for i in range(20):
        for t in (q, k, v):
            t.copy_(torch.from_numpy(r.standard_normal(tuple(t.shape))).to(torch.bfloat16))
        graph.replay()
        want = step(caches[1], elens, torch.empty_like(q), None)
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
    assert torch.equal(caches[0].data, caches[1].data) and torch.equal(glens, elens)


def test_attention_on_two_streams(S):
    b = Batch(S, 54, [900, 400, 20], 2, 128, 32, "bf16")
    qs = [b.queries(1, 8) for _ in range(2)]
    want = [S.kv4_attention(b.cache, q, b.table, b.seq_lens) for q in qs]
    torch.cuda.synchronize()
    announce("kv4 attention on two streams")
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(S.kv4_attention(b.cache, qs[i], b.table, b.seq_lens))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def put(S, b, seq, token, k, v):
    """Token `token` of sequence `seq` of a batch anew: k, v [H, D] float64, NaN blocks and all."""
    page = b.cache.page_size
    slot = b.table[seq, token // page] * page + token % page
    rows16 = [torch.from_numpy(x[None]).to(DT[b.dtype]).cuda() for x in (k, v)]
    S.kv4_append(b.cache, *rows16, slot.reshape(1).to(torch.int32))
    b.k[seq][token], b.v[seq][token] = (O.values(f64(x))[0] for x in rows16)


def check_nan(got, q, b, scale):
    """Not a number where the oracle's sum has one, and the bound of `check` everywhere else."""
    with np.errstate(invalid="ignore"):
        nan = np.isnan(O.attend(f64(q), b.k, b.v, b.lens, scale)[0])
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(f64(got)), nan)
    clean = type("B", (), dict(k=[np.nan_to_num(x) for x in b.k], v=[np.nan_to_num(x) for x in b.v], lens=b.lens))
    fill = torch.from_numpy(O.attend(f64(q), clean.k, clean.v, b.lens, scale)[0]).to(got)
    check(torch.where(torch.from_numpy(nan).cuda(), fill, got), q, clean, scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Q,group", [(2, 3), (3, 2), (3, 5), (5, 3), (5, 4), (3, 16), (40, 1)])
def test_new_tokens_do_not_see_what_is_not_finite_after_them(S, Q, group, D, dtype):
    """An infinity or a NaN in a new token's value or key reaches that token and those after it, and none before:
    the last one's, a middle one's and the first one's, on both sides of a unit's, a page's and a chunk's end."""
    H, lens = 2, [130, 35, 259, 3, 70]
    announce(f"kv4 attention, not finite among {Q} new tokens, {Q * group} rows, D={D} {dtype}")
    b = Batch(S, 60 + Q + group, lens, H, D, 16, dtype)
    r = b.r
    for seq, back, head, channel, bad, key in ((0, 1, 0, 3, np.nan, False), (0, 2, 1, D - 1, np.inf, False),
                                               (1, 1, 1, 40, -np.inf, False), (2, 2, 0, 0, np.nan, True),
                                               (2, Q, 1, 33, np.inf, False), (3, 1, 0, D - 2, np.nan, False)):
        n = lens[seq]
        k, v = r.standard_normal((2, H, D))
        (k if key else v)[head, channel] = bad
        put(S, b, seq, max(n - back, 0), k, v)
    q = b.queries(Q, H * group)
    check_nan(S.kv4_attention(b.cache, q, b.table, b.seq_lens), q, b, D ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Q,group,D", [(1, 4, 128), (1, 12, 64), (3, 8, 128), (1, 20, 256)])
def test_a_row_of_infinite_scores_is_not_a_row_without_tokens(S, Q, group, D, dtype):
    """Scores that are all minus infinity leave 0 / 0, whether one workgroup or many take the row; a row
    that sees no token is zero whatever its query holds."""
    lens = [40, 0, 5000, 1, 64]
    b = Batch(S, 80, lens, 1, D, 16, dtype)
    for x in b.k:
        x[:] = 1.0
    n = b.pages * 16
    ones = torch.ones(n, 1, D, dtype=DT[dtype], device="cuda")
    S.kv4_append(b.cache, ones, ones, torch.arange(n, dtype=torch.int32, device="cuda"))
    b.table[4] = -1                                  # a sequence of which no page is here
    announce(f"kv4 attention of infinite scores, {Q * group} rows, D={D} {dtype}")
    q = b.queries(Q, group)
    want = S.kv4_attention(b.cache, q, b.table, b.seq_lens)
    q[:, :, 1] = 0
    q[:, :, 1, 7] = -float("inf")
    got = S.kv4_attention(b.cache, q, b.table, b.seq_lens)
    for seq, m in enumerate(lens):
        for i in range(Q):
            sees = m - Q + i + 1 > 0 and seq != 4
            assert torch.isnan(got[seq, i, 1]).all() if sees else not got[seq, i, 1].any(), (seq, i)
    got[:, :, 1] = want[:, :, 1]
    assert torch.equal(got, want)


def test_attention_of_thousands_of_sequences(S):
    """A batch of many short sequences, every fifth slot of it empty."""
    r = np.random.default_rng(90)
    lens = [0 if b % 5 == 3 else int(x) for b, x in enumerate(r.integers(1, 40, 3000))]
    b = Batch(S, 91, lens, 1, 64, 16, "bf16")
    q = b.queries(1, 2)
    announce("kv4 attention of 3000 sequences")
    got = S.kv4_attention(b.cache, q, b.table, b.seq_lens)
    check(got, q, b, 0.125)
    assert not got[3::5].any()


@pytest.mark.parametrize("Q,group,H,D,lens,dtype", [
    (128, 8, 1, 64, [300, 130, 100], "bf16"), (256, 4, 1, 128, [256], "fp16"), (64, 8, 2, 128, [65, 400], "bf16"),
    (1024, 1, 1, 64, [1500, 700], "fp16"), (33, 31, 1, 64, [90], "bf16"), (130, 4, 1, 256, [140, 20], "fp16")])
def test_attention_of_a_prompts_chunk(S, Q, group, H, D, lens, dtype):
    """Up to 1024 rows of a key/value head, sequences shorter than the chunk among them."""
    announce(f"kv4 attention of {Q} new tokens of {H * group} heads, D={D} {dtype}")
    b = Batch(S, 92, lens, H, D, 16, dtype)
    q = b.queries(Q, H * group)
    check(S.kv4_attention(b.cache, q, b.table, b.seq_lens), q, b, D ** -0.5)


def test_attention_of_expanded_queries(S):
    """One token's query for every sequence, and one head's for all, by strides of zero."""
    b = Batch(S, 93, [200, 31, 64], 2, 64, 32, "fp16")
    q = b.queries(1, 8)
    announce("kv4 attention of expanded queries")
    for e in (q[:1].expand(3, 1, 8, 64), q[:, :, :1].expand(3, 1, 8, 64)):
        got = S.kv4_attention(b.cache, e, b.table, b.seq_lens)
        check(got, e, b, 0.125)
        assert torch.equal(got, S.kv4_attention(b.cache, e.contiguous(), b.table, b.seq_lens))


def test_attention_at_the_largest_sizes(S):
    """65536 sequences, most of them empty or one token long, and 1024 key/value heads."""
    r = np.random.default_rng(94)
    B, pages, D = 65536, 40, 64
    cache = S.Kv4Cache(pages, 16, 1, D)
    k, v = rows(r, (pages * 16, 1, D), "bf16"), rows(r, (pages * 16, 1, D), "bf16")
    S.kv4_append(cache, k, v, torch.arange(pages * 16, dtype=torch.int32, device="cuda"))
    lens = r.integers(0, 3, B)
    lens[[0, 777, B - 1]] = 16
    table = r.integers(0, pages, (B, 1)).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((B, 1, 1, D))).to(torch.bfloat16).cuda()
    announce("kv4 attention of 65536 sequences")
    got = S.kv4_attention(cache, q, torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda())
    kv, vv = O.values(f64(k)), O.values(f64(v))
    bb = type("B", (), dict(k=[kv[16 * t[0]:16 * t[0] + n] for t, n in zip(table, lens)],
                            v=[vv[16 * t[0]:16 * t[0] + n] for t, n in zip(table, lens)], lens=lens))
    check(got, q, bb, 0.125)
    announce("kv4 attention of 1024 heads")
    b = Batch(S, 95, [20, 0, 33], 1024, D, 16, "fp16")
    q = b.queries(1, 1024)
    check(S.kv4_attention(b.cache, q, b.table, b.seq_lens), q, b, 0.125)


@pytest.mark.parametrize("Q,group", [(1, 4), (1, 16), (3, 7)])
def test_attention_of_the_smallest_keys_and_values(S, Q, group):
    """Blocks of the smallest scales, whose numbers are bf16's subnormal ones, under large queries."""
    r = np.random.default_rng(96)
    lens, D = [100, 7], 64
    b = Batch(S, 97, lens, 1, D, 16, "bf16")
    n = b.pages * 16
    k = torch.from_numpy(r.standard_normal((n, 1, D)) * 2.0 ** -127).to(torch.bfloat16).cuda()
    v = torch.from_numpy(r.standard_normal((n, 1, D)) * 2.0 ** -100).to(torch.bfloat16).cuda()
    S.kv4_append(b.cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    kv, vv = O.values(f64(k)), O.values(f64(v))
    t = b.table.cpu().numpy()
    for s, m in enumerate(lens):
        at = t[s, np.arange(m) // 16] * 16 + np.arange(m) % 16
        b.k[s], b.v[s] = kv[at], vv[at]
    assert (np.abs(kv[kv != 0]) < 2.0 ** -126).any()
    q = b.queries(Q, group, 2.0 ** 112)
    announce(f"kv4 attention of the smallest keys, {Q * group} rows")
    check(S.kv4_attention(b.cache, q, b.table, b.seq_lens, scale=2.0 ** 12), q, b, 2.0 ** 12)


@pytest.mark.parametrize("scale", [0.0, 3e-39, -1e-38, 6e-38])
def test_attention_of_smallest_scales_and_large_products(S, scale):
    """Products of 1e37 at scales that bring them to 0 (equal weights) and to scores below 1."""
    scale = float(np.float32(scale))
    r = np.random.default_rng(98)
    lens, D = [333, 40], 64
    b = Batch(S, 99, lens, 1, D, 16, "bf16")
    n = b.pages * 16
    k = rows(r, (n, 1, D), "bf16")
    k[..., 3] = torch.from_numpy(r.uniform(-1e18, 1e18, (n, 1))).to(k)
    v = rows(r, (n, 1, D), "bf16")
    S.kv4_append(b.cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    kv, vv = O.values(f64(k)), O.values(f64(v))
    t = b.table.cpu().numpy()
    for s, m in enumerate(lens):
        at = t[s, np.arange(m) // 16] * 16 + np.arange(m) % 16
        b.k[s], b.v[s] = kv[at], vv[at]
    q = b.queries(2, 4)
    q[..., 3] = 1e19
    announce(f"kv4 attention of products of 1e37, scale {scale}")
    check(S.kv4_attention(b.cache, q, b.table, b.seq_lens, scale=scale), q, b, scale)


@pytest.mark.parametrize("kind", ["alike", "rising", "negative"])
@pytest.mark.parametrize("lens,Q,Hq,H,D,page,dtype,power", [
    ([700, 33], 1, 8, 2, 128, 16, "bf16", 40), ([700, 33], 3, 4, 1, 64, 32, "bf16", 56), ([20000], 1, 8, 1, 128, 256, "bf16", 30),
    ([300], 1, 32, 2, 256, 64, "fp16", 15), ([1000, 5], 1, 17, 1, 128, 32, "bf16", 20)])
def test_attention_of_scores_far_from_zero(S, lens, Q, Hq, H, D, page, dtype, power, kind):
    """Scores of 2^30 to 2^118, where a step of float32 is many units of the exponent: those that are alike weigh the same,
    and the others, lower by a sixteenth or more, nothing.  All products and their sums are exact."""
    b = Batch(S, 120, lens, H, D, page, dtype)
    top = max(power, 30)
    announce(f"kv4 attention of scores far from zero, {lens} Q={Q} {Hq}/{H} D={D} {dtype} 2^{power} {kind}")
    q = torch.full((len(lens), Q, Hq, D), 2.0 ** power, dtype=DT[dtype], device="cuda")
    n = b.pages * page
    k = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
    v = rows(b.r, (n, H, D), "bf16")
    t = b.table.cpu().numpy()
    slots = [t[s, np.arange(m) // page] * page + np.arange(m) % page for s, m in enumerate(lens)]
    steps = {"alike": lambda i: np.full(len(i), 3.0), "rising": lambda i: np.array([0.5, 1, 1.5, 2, 3, 4, 6])[7 * i // len(i)],
             "negative": lambda i: -np.array([6, 4, 3, 2, 1.5, 1, 0.5])[7 * i // len(i)]}[kind]
    for at in slots:
        k[torch.from_numpy(at).long().cuda()] = torch.from_numpy(steps(np.arange(len(at))) * 2.0 ** (top - 2))[:, None, None].to(k)
    S.kv4_append(b.cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    vv = O.values(f64(v))
    for scale in (0.3, 0.11, 0.71, 0.0625):
        got = f64(S.kv4_attention(b.cache, q, b.table, b.seq_lens, scale=scale))
        for s, m in enumerate(lens):
            for i in range(Q):
                seen = m - Q + i + 1
                x = steps(np.arange(m))[:seen]
                best = vv[slots[s][:seen][x == x.max()]]
                want, mean = (np.repeat(y.mean(0), Hq // H, 0) for y in (best, np.abs(best)))
                # the weights are all 1, the sums over them as above, and the result is rounded
                tol = torch.finfo(DT[dtype]).eps / 2 * np.abs(want) * (1 + 2.0 ** -6) + (2.0 ** -20 + 2 * m * 2.0 ** -24) * mean
                assert (np.abs(got[s, i] - want) <= tol).all(), (scale, s, i)
