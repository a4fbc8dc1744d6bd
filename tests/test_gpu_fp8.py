"""The 8-bit floating point linear on the GPU against the float64 oracle: the
quantiser bit for bit, results bit for bit where every sum is exact, and within the
roundings of their sums elsewhere.

Tolerance.  A result is a sum of K products, one block of 128 at a time, each block
times a float32 scale.  The matrix instruction adds eight neighbouring products
at a time, each cut off below 2^-13 of the largest: at most 7 2^-13 of it for the
eight, 7 2^-13 size for the result (size: the sum of the terms' magnitudes).  These
sums, the blocks and the scale are added in float32, K / 8 + K / 128 + 2 steps
of 2^-23 size at most.  The GELU passes an error on by at most 1.13 and its own float32
steps are below 2^-18 of the result.  Then half a step (eps / 2) of the result's type.
The instruction leaves zero for a result below 2^-126: K / 64 times that at most, where scales are below 1.
On average the cuts are far smaller: a cut is below 2^-13 of the group's largest
term, so K of them with random signs have a root mean square below 2^-13 sqrt(K
/ 3) times that of the largest terms."""
import numpy as np
import pytest
import torch

from oracle import fp8 as O
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


def rows(r, M, K, dtype):
    x = r.standard_normal((M, K))
    x[:, ::37] *= 8.0
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def weight(r, N, K):
    """Codes of a normal matrix and scales that are no powers of two."""
    codes = (r.integers(0, 126, (N, K)) | r.integers(0, 2, (N, K)) << 7).astype(np.uint8)
    return codes, (r.random((-(-N // 128), O.blocks(K))) + 0.5).astype(np.float32) / 3e4


def near(got, want, size, K, gelu=False):
    tol = (7 * 2.0 ** -13 + (K / 8 + K / 128 + 2) * 2.0 ** -23) * size
    tol = tol + K / 64 * 2.0 ** -126
    if gelu:
        want = O.gelu(want)
        tol = 1.13 * tol + 2.0 ** -18 * np.abs(want)
    tol = tol * (1 + 2.0 ** -6) + torch.finfo(got.dtype).eps / 2 * np.abs(want) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    off = np.abs(f64(got) - want)
    assert (off <= tol).all(), ((off / tol).max(), np.unravel_index((off / tol).argmax(), off.shape))


CASES = [  # M, N, K
    (1, 1, 8), (1, 64, 128), (1, 4100, 520), (11, 4200, 264), (1, 300, 1000), (2, 1152, 4608), (5, 33, 136), (8, 96, 3000), (7, 96, 4096), (9, 40, 4096), (16, 50, 1536), (16, 50, 1544), (17, 70, 1024), (31, 65, 2056), (80, 70, 1000), (96, 40, 520),
    (32, 64, 1024), (33, 64, 256), (64, 200, 520), (65, 130, 384), (77, 2121, 1160), (100, 31, 8), (128, 128, 128),
    (129, 257, 264), (200, 1000, 640), (513, 384, 2048),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", CASES)
def test_fp8_linear_against_the_oracle(S, M, N, K, dtype):
    r = np.random.default_rng(M + N + K)
    codes, scales = weight(r, N, K)
    bias = r.standard_normal(N).astype(np.float32)
    x = rows(r, M, K, dtype)
    want, size = O.forward(f64(x), codes, scales)
    layers = S.Fp8Linear(codes, scales), S.Fp8Linear(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn),
                                                     torch.from_numpy(scales).cuda(), torch.from_numpy(bias).cuda())
    for out in (None, "bf16", "fp16"):
        announce(f"fp8 linear M={M} N={N} K={K} {dtype} -> {out}")
        got = S.fp8_linear_forward(layers[0], x, out_dtype=None if out is None else DT[out])
        assert got.dtype == DT[out or dtype] and got.shape == (M, N)
        near(got, want, size, K)
    announce(f"fp8 linear M={M} N={N} K={K} {dtype} with bias and GELU")
    near(S.fp8_linear_forward(layers[1], x), want + bias, size + np.abs(bias), K)
    near(S.fp8_linear_forward(layers[1], x, gelu=True), want + bias, size + np.abs(bias), K, gelu=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", CASES)
def test_fp8_linear_exact_sums(S, M, N, K, dtype):
    """Small integers and scales of few bits: no product is cut and every float32 sum is exact, so the
    result is the exact one rounded once, and a term left out or taken twice shows.
    (Integers up to 3 in both: products of codes are 2^7 times integers up to 9; sums of up
    to 5000 of them times 1, 2, 3 or 4 eighths are below 2^18 eighths.)"""
    r = np.random.default_rng(M * N + K)
    xi, wi = r.integers(-3, 4, (M, K)).astype(float), r.integers(-3, 4, (N, K)).astype(float)
    scales = (r.integers(1, 5, (-(-N // 128), O.blocks(K))) / 8).astype(np.float32)
    codes = torch.from_numpy(wi).float().to(torch.float8_e4m3fn)
    bias = (r.integers(-20, 21, N) / 8).astype(np.float32)
    w = wi * np.repeat(np.repeat(scales, 128, 0)[:N], 128, 1)[:, :K]
    want = torch.from_numpy(xi @ w.T)
    x = torch.from_numpy(xi).to(DT[dtype]).cuda()
    announce(f"fp8 linear with exact sums M={M} N={N} K={K} {dtype}")
    assert torch.equal(S.fp8_linear_forward(S.Fp8Linear(codes, scales), x).cpu(), want.to(DT[dtype]))
    assert torch.equal(S.fp8_linear_forward(S.Fp8Linear(codes, scales, bias), x).cpu(), (want + torch.from_numpy(bias)).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 128), (33, 136), (70, 1000), (1, 5000)])
def test_fp8_quantiser_bit_for_bit(S, M, K, dtype):
    r = np.random.default_rng(M * K)
    # magnitudes over the type's whole range
    x = r.standard_normal((M, K)) * np.exp2(r.integers(-24 if dtype == "fp16" else -140, 14 if dtype == "fp16" else 120, (M, K)).astype(float))
    x = torch.from_numpy(x).to(DT[dtype]).cuda()
    announce(f"fp8 quantiser M={M} K={K} {dtype}")
    codes, scales = S.fp8_quantize_activations(x)
    v, e = O.quantize_rows(f64(x))
    assert codes.dtype == torch.float8_e4m3fn and np.array_equal(O.decode(codes.view(torch.uint8).cpu().numpy()), v)
    assert np.array_equal(scales.cpu().numpy().astype(int) - 127, e)


def test_fp8_quantiser_every_border(S):
    """Every value, tie and neighbour of a tie of the grid, at the block's largest scale and at small ones."""
    grid = O.decode(np.arange(127, dtype=np.uint8))
    ties = (grid[1:] + grid[:-1]) / 2
    near_ties = np.concatenate([ties * (1 + 2.0 ** -7), ties * (1 - 2.0 ** -7)])
    v = np.concatenate([grid, ties, near_ties, -grid, -ties])
    v = v[v <= 448]
    x = np.zeros((3, 128 * (len(v) // 100 + 1)))
    for i in range(0, len(v), 100):
        part = v[i:i + 100]
        x[0, 128 * (i // 100):][:len(part)] = part
        x[1, 128 * (i // 100):][:len(part)] = part * 2.0 ** -100
        x[2, 128 * (i // 100):][:len(part)] = part * 2.0 ** 100
    x[:, 127::128] = np.array([[448], [448 * 2.0 ** -100], [448 * 2.0 ** 100]])
    x = torch.from_numpy(x).to(torch.bfloat16).cuda()
    announce("fp8 quantiser at every border")
    codes, scales = S.fp8_quantize_activations(x)
    want, e = O.quantize_rows(f64(x))
    assert np.array_equal(O.decode(codes.view(torch.uint8).cpu().numpy()), want) and (e == [[0], [-100], [100]]).all()
    assert np.array_equal(scales.cpu().numpy().astype(int) - 127, e)


def test_fp8_edge_values(S):
    """Zeros, the smallest and largest numbers, borders of the scale, infinities and NaN."""
    x = np.zeros((9, 256))
    x[1, 3], x[1, 200] = 2.0 ** -133, -2.0 ** -126
    x[2, 0], x[2, 130] = 3.3e38, 1.0
    x[3, 5] = np.inf
    x[4, 255] = np.nan
    x[5, :] = 448.0
    x[6, 1], x[6, 129] = 450.0, 1.75
    x[7, 1], x[7, 2] = 1.7578125, 2.0 ** -9
    x[8, :128] = -0.0
    x = torch.from_numpy(x).to(torch.bfloat16).cuda()
    announce("fp8 quantiser of edge values")
    codes, scales = S.fp8_quantize_activations(x)
    v, e = O.quantize_rows(f64(x))
    assert np.array_equal(O.decode(codes.view(torch.uint8).cpu().numpy()), v, equal_nan=True)
    assert np.array_equal(scales.cpu().numpy().astype(int) - 127, e)
    r = np.random.default_rng(1)
    w, s = weight(r, 40, 256)
    layer = S.Fp8Linear(w, s)
    want, size = O.forward(f64(x), w, s)
    bad = np.isnan(want)
    assert bad[3].all() and bad[4].all() and bad.sum() == 80
    for repeat in (1, 8, 40):                    # few rows, more, and a tile
        announce(f"fp8 linear of edge values, {9 * repeat} rows")
        got = S.fp8_linear_forward(layer, x.repeat(repeat, 1))
        for part in got.reshape(repeat, 9, 40):
            assert np.array_equal(torch.isnan(part).cpu().numpy(), bad)
            fine = ~bad[:, 0]
            near(part[torch.from_numpy(fine).cuda()], want[fine], size[fine], 256)


@pytest.mark.parametrize("M", [3, 50, 300])
def test_fp8_linear_strided_rows_and_padding_stays(S, M):
    r = np.random.default_rng(2)
    N, K = 72, 200
    codes, scales = weight(r, N, K)
    layer = S.Fp8Linear(codes, scales)
    big = rows(r, M, K + 56, "bf16")
    x = big[:, 16:16 + K]
    buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    announce(f"fp8 linear of strided rows, M={M}")
    S.fp8_linear_forward(layer, x, out=buf[1:M + 1])
    want, size = O.forward(f64(x), codes, scales)
    near(buf[1:M + 1], want, size, K)
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
    # one row for all
    one = x[:1].expand(M, K)
    near(S.fp8_linear_forward(layer, one), np.repeat(want[:1], M, 0), np.repeat(size[:1], M, 0), K)
    assert S.fp8_linear_forward(layer, x[:0]).shape == (0, N)


def test_fp8_weights_quantised_here(S):
    """A float matrix through the library's quantiser and the layer: within half a step of e4m3 of both operands."""
    r = np.random.default_rng(3)
    N, K, M = 200, 500, 20
    W = r.standard_normal((N, 504)) / 20
    K = 504
    codes, scales = S.fp8_quantize_weights(W)
    layer = S.Fp8Linear(codes, scales)
    x = rows(r, M, K, "bf16")
    want, size = O.forward(f64(x), codes, scales)
    announce("fp8 linear of weights quantised here")
    near(S.fp8_linear_forward(layer, x), want, size, K)
    full = f64(x) @ W.T
    bound = np.abs(f64(x)) @ np.abs(W).T * 2.2 * 2.0 ** -4
    # codes below 2^-6 of the largest 448 are off by half of 2^-9: 2^-10 / 448 of the block's largest
    bound += (np.abs(f64(x)).sum(1)[:, None] * np.abs(W).max() + np.abs(f64(x)).max() * np.abs(W).sum(1)) * 2.0 ** -9 / 448 * 2
    assert (np.abs(want - full) <= bound).all()


def test_fp8_linear_large(S):
    """Tiles beyond one round of workgroups, in each of the tile's forms, against float64 products on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for M, N, K in ((1500, 1300, 1024), (4608, 8192, 640), (4100, 8200, 384)):
        x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
        W = torch.randn(N, K, device="cuda", generator=g)
        scales = torch.rand(-(-N // 128), -(-K // 128), device="cuda", generator=g) * 0.01 + 0.01
        codes = (W * 50).clamp(-448, 448).to(torch.float8_e4m3fn)
        layer = S.Fp8Linear(codes, scales)
        announce(f"fp8 linear M={M} N={N} K={K}")
        got = S.fp8_linear_forward(layer, x)
        q, e = S.fp8_quantize_activations(x)
        xq = q.double() * torch.exp2(e.double() - 127).repeat_interleave(128, 1)[:, :K]
        w = codes.double() * scales.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        want, size = xq @ w.t(), xq.abs() @ w.abs().t()
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + (7 * 2.0 ** -13 + (K / 8 + K / 128 + 2) * 2.0 ** -23) * size).all()


@pytest.mark.parametrize("M,N", [(2100, 1000), (2900, 1500), (4100, 1500), (4500, 2700), (1500, 300)])
@pytest.mark.parametrize("K", [8, 128, 136, 384, 504, 640])
def test_fp8_linear_every_tile_form_short_k(S, M, N, K):
    """Tiles of 128 x 128 with four stages, of 192 x 128, of 128 x 128 with two, of 256 x 256 and of 64 x 64, over fewer blocks of K than
    stages and a few more: small integers, as above, so that the result is the exact one rounded once."""
    announce(f"fp8 linear of small integers M={M} N={N} K={K}")
    g = torch.Generator(device="cuda").manual_seed(M + K)
    xi, wi = (torch.randint(-3, 4, (n, K), device="cuda", generator=g).double() for n in (M, N))
    scales = torch.randint(1, 5, (-(-N // 128), -(-K // 128)), device="cuda", generator=g).float() / 8
    bias = torch.randint(-20, 21, (N,), device="cuda", generator=g).float() / 8
    layer = S.Fp8Linear(wi.float().to(torch.float8_e4m3fn), scales, bias)
    w = wi * scales.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    want = xi @ w.t() + bias.double()
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(S.fp8_linear_forward(layer, xi.to(dtype)), want.to(dtype))


@pytest.mark.parametrize("M", [8, 60, 400])
def test_fp8_linear_error_on_average(S, M):
    r = np.random.default_rng(12)
    N, K = 256, 2048
    codes, scales = weight(r, N, K)
    x = rows(r, M, K, "fp16")
    want, _ = O.forward(f64(x), codes, scales)
    announce(f"fp8 linear on average, M={M}")
    off = f64(S.fp8_linear_forward(S.Fp8Linear(codes, scales), x)) - want
    # the largest term of any group of eight, at most: the row's and the column's largest values
    v, e = O.quantize_rows(f64(x))
    top = np.abs(v * np.exp2(np.repeat(e, 128, 1).astype(float)))
    w = np.abs(O.decode(codes) * np.repeat(np.repeat(scales.astype(float), 128, 0)[:N], 128, 1))
    big = np.sqrt((top ** 2).reshape(M, -1, 8).max(-1) @ (w ** 2).reshape(N, -1, 8).max(-1).T / (K / 8))
    cut = 2.0 ** -13 * np.sqrt(K / 3) * big
    rounding = 2.0 ** -11 / np.sqrt(3) * np.abs(want)
    assert np.sqrt((off ** 2).mean()) <= 1.1 * np.sqrt((cut ** 2 + rounding ** 2).mean())


def test_fp8_linear_of_a_slice_of_rows(S):
    """Codes that start in the middle of a larger matrix, at an address that is no multiple of 16."""
    r = np.random.default_rng(9)
    codes, _ = weight(r, 200, 136)
    scales = np.ones((1, 2), np.float32)
    whole = torch.from_numpy(codes).cuda()
    x = rows(r, 5, 136, "bf16")
    announce("fp8 linear of a slice of rows")
    got = S.fp8_linear_forward(S.Fp8Linear(whole[3:103], torch.from_numpy(scales).cuda()), x)
    assert torch.equal(got, S.fp8_linear_forward(S.Fp8Linear(codes[3:103], scales), x))


def test_fp8_linear_streams_and_graphs(S):
    """Two layers on two streams at once, and captured with workspaces of their own."""
    r = np.random.default_rng(6)
    sets = []
    for M, N, K in ((2, 100, 512), (150, 300, 640)):
        layer = S.Fp8Linear(*weight(r, N, K), bias=np.ones(N, np.float32))
        x = [rows(r, M, K, "fp16") for _ in range(3)]
        sets.append((layer, x, [S.fp8_linear_forward(layer, a) for a in x]))
    torch.cuda.synchronize()
    announce("fp8 linear on two streams")
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for s, (layer, x, want) in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append([S.fp8_linear_forward(layer, a) for a in x])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, s in zip(got, sets) for a, b in zip(g, s[2]))
    graphs = []
    announce("fp8 linear in two graphs")
    for layer, x, want in sets:
        bufs = (x[0].clone(), torch.empty_like(want[0]), layer.new_workspace(x[0].shape[0]))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.fp8_linear_forward(layer, bufs[0], out=bufs[1], workspace=bufs[2])
        graphs.append((g, bufs))
    for i in (1, 2, 0, 1):
        for (g, bufs), (layer, x, want) in zip(graphs, sets):
            bufs[0].copy_(x[i])
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bufs[1], s[2][i]) for (g, bufs), s in zip(graphs, sets))


@pytest.mark.parametrize("M", [1, 16, 20, 50, 130, 700])
def test_fp8_linear_scales_over_the_whole_range(S, M):
    """Weight scales of zero, negative, subnormal and up to 2^127, under activations that bring the results back into
    range: small integers times powers of two, so that every sum is exact and the result is rounded once."""
    r = np.random.default_rng(M)
    bases = np.array([0.0, -0.125, 2.0 ** -149, 2.0 ** -130, 2.0 ** -126, 2.0 ** 100, 2.0 ** 125])
    N, K = 128 * len(bases), 264
    xi, wi = r.integers(-3, 4, (M, K)).astype(float), r.integers(-3, 4, (N, K)).astype(float)
    scales = (bases[:, None] * r.integers(1, 5, (len(bases), O.blocks(K)))).astype(np.float32)
    scales[-1, -1] = 2.0 ** 127
    w = wi * np.repeat(np.repeat(scales.astype(float), 128, 0), 128, 1)[:, :K]
    layer = S.Fp8Linear(torch.from_numpy(wi).float().to(torch.float8_e4m3fn), scales)
    reached = set()
    for power in (-100, 0, 60, 110):
        x = torch.from_numpy(xi * 2.0 ** power).bfloat16().cuda()
        announce(f"fp8 linear of scales over the whole range, M={M}, rows of 2^{power}")
        got = S.fp8_linear_forward(layer, x).cpu()
        want = torch.from_numpy((xi * 2.0 ** power) @ w.T).bfloat16()
        for i, b in enumerate(np.abs(bases)):
            # 264 products of up to 9 by 4 times the base: below 2^14 times it; at the other end the instruction's
            # products are multiples of 2^power times a base's power of two, 2^-126 for subnormal ones
            if b == 0 or (2.0 ** (power + 14) * b < 2.0 ** 127 and 2.0 ** power * max(b, 2.0 ** -126) >= 2.0 ** -126
                          and 2.0 ** power * b >= 2.0 ** -126):
                at = slice(128 * i, 128 * i + 128)
                assert torch.equal(got[:, at], want[:, at]), (power, b)
                reached.add(i)
    assert reached == set(range(len(bases)))
