"""An attention block of the three operators as a program would run it: 8-bit linears make
the queries and, in one fused projection, the keys and values of an encoder's states;
the queries and keys turn with their positions; the queries attend over the
states; an 8-bit linear with GELU takes the result.  Every step reads views of what the one before
it wrote.  And tensors whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from oracle import cross, fp8, rotary
from tests import test_gpu_cross, test_gpu_fp8, test_gpu_rotary
from tests.conftest import announce
from tests.test_gpu_fp8 import DT, S, f64, rows, weight   # noqa: F401  (S: the library's fixture)

pytestmark = pytest.mark.gpu


class Block:
    """One block with its layers, workspaces and buffers."""

    def __init__(self, S, r, B, Lq, Lk, Hq, Hkv, D, C, dtype, widths):
        self.S, self.shape, self.widths = S, (B, Lq, Lk, Hq, Hkv, D, C), widths
        sizes = {"q": (Hq * D, C), "kv": (2 * Hkv * D, C), "out": (C, Hq * D)}
        self.parts = {n: weight(r, *s) for n, s in sizes.items()}
        self.bias = {n: r.standard_normal(s[0]).astype(np.float32) for n, s in sizes.items()}
        self.layer = {n: S.Fp8Linear(*self.parts[n], bias=self.bias[n]) for n in sizes}
        self.plan = S.RotaryPlan(D, widths)
        new = lambda *s: torch.full(s, 9.0, dtype=DT[dtype], device="cuda")
        self.x, self.ctx = new(B * Lq, C), new(B * Lk, C)
        self.q, self.kv, self.y = new(B * Lq, Hq * D), new(B * Lk, 2 * Hkv * D), new(B, Lq, Hq, D)
        self.turned_q, self.turned_k = new(B * Lq, Hq, D), new(B * Lk, Hkv, D)
        self.out = new(B * Lq, C)
        self.pos_q = torch.from_numpy(r.integers(0, 90, (B * Lq, len(widths))).astype(np.int32)).cuda()
        self.pos_k = torch.from_numpy(r.integers(0, 90, (B * Lk, len(widths))).astype(np.int32)).cuda()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ws = {"q": self.layer["q"].new_workspace(B * Lq), "kv": self.layer["kv"].new_workspace(B * Lk),
                   "out": self.layer["out"].new_workspace(B * Lq)}
        self.attend_ws = S.cross_attention_workspace(self.y, self.turned_k.view(B, Lk, Hkv, D))

    def set(self, r):
        B, Lq, Lk = self.shape[:3]
        for t in (self.x, self.ctx):
            t.copy_(torch.from_numpy(r.standard_normal(t.shape)))
        self.lens.copy_(torch.from_numpy(r.integers(0, Lk + 1, B).astype(np.int32)))

    def run(self):
        S, (B, Lq, Lk, Hq, Hkv, D, C) = self.S, self.shape
        S.fp8_linear_forward(self.layer["q"], self.x, out=self.q, workspace=self.ws["q"])
        S.fp8_linear_forward(self.layer["kv"], self.ctx, out=self.kv, workspace=self.ws["kv"])
        q, kv = self.q.view(B * Lq, Hq, D), self.kv.view(B * Lk, 2 * Hkv, D)
        S.rotary_apply(self.plan, q, None, self.pos_q, q_out=self.turned_q)
        S.rotary_apply(self.plan, kv[:, :Hkv], None, self.pos_k, q_out=self.turned_k)
        S.cross_attention(self.turned_q.view(B, Lq, Hq, D), self.turned_k.view(B, Lk, Hkv, D),
                          kv[:, Hkv:].view(B, Lk, Hkv, D), key_lens=self.lens, out=self.y, workspace=self.attend_ws)
        S.fp8_linear_forward(self.layer["out"], self.y.view(B * Lq, Hq * D), gelu=True, out=self.out,
                             workspace=self.ws["out"])
        return [t.clone() for t in (self.q, self.kv, self.turned_q, self.turned_k, self.y, self.out)]

    def check(self, got):
        """Each step against its own oracle and tolerance, from what the step read."""
        B, Lq, Lk, Hq, Hkv, D, C = self.shape
        q, kv, turned_q, turned_k, y, out = got
        for n, x, z in (("q", self.x, q), ("kv", self.ctx, kv), ("out", y.view(B * Lq, Hq * D), out)):
            want, size = fp8.forward(f64(x), *self.parts[n])
            test_gpu_fp8.near(z, want + self.bias[n], size + np.abs(self.bias[n]), x.shape[1], gelu=n == "out")
        kv = kv.view(B * Lk, 2 * Hkv, D)
        freq, axis = rotary.ladder(self.widths, 10000.0, True)
        test_gpu_rotary.near(turned_q, q.view(B * Lq, Hq, D), self.pos_q.cpu().numpy(), freq, axis, True)
        test_gpu_rotary.near(turned_k, kv[:, :Hkv], self.pos_k.cpu().numpy(), freq, axis, True)
        visible = np.arange(Lk) < self.lens.cpu().numpy()[:, None]
        test_gpu_cross.near(y, turned_q.view(B, Lq, Hq, D), turned_k.view(B, Lk, Hkv, D),
                            kv[:, Hkv:].view(B, Lk, Hkv, D), visible)


SHAPES = [  # B, Lq, Lk, Hq, Hkv, D, C, widths
    (2, 1, 333, 4, 2, 64, 256, [32, 32]),
    (3, 30, 700, 4, 1, 128, 200, [16, 56, 56]),
    (1, 300, 77, 3, 3, 72, 136, [24, 24, 24]),
    (2, 140, 45, 6, 2, 96, 576, [96]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hkv,D,C,widths", SHAPES)
def test_block_against_the_oracles(S, B, Lq, Lk, Hq, Hkv, D, C, widths, dtype):
    r = np.random.default_rng(Lq + Lk)
    announce(f"block B={B} Lq={Lq} Lk={Lk} Hq={Hq} Hkv={Hkv} D={D} C={C} {dtype}")
    block = Block(S, r, B, Lq, Lk, Hq, Hkv, D, C, dtype, widths)
    block.set(r)
    block.check(block.run())


def test_blocks_in_graphs_on_two_streams(S):
    """Blocks captured one by one, replayed on two streams at once over changing inputs, with eager calls of the same
    layers in between: every replay's results are the eager ones."""
    r = np.random.default_rng(4)
    blocks = [Block(S, r, *s[:7], "bf16", s[7]) for s in SHAPES[:3:2]]
    states = []
    for b in blocks:
        for _ in range(3):
            b.set(r)
            states.append((b.x.clone(), b.ctx.clone(), b.lens.clone(), b.run()))
    torch.cuda.synchronize()
    announce("blocks in graphs on two streams")
    graphs, streams = [], [torch.cuda.Stream() for _ in blocks]
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    for i in (1, 0, 2, 2, 1):
        for n, (b, g, s) in enumerate(zip(blocks, graphs, streams)):
            x, ctx, lens, _ = states[3 * n + i]
            with torch.cuda.stream(s):
                b.x.copy_(x), b.ctx.copy_(ctx), b.lens.copy_(lens)
                g.replay()
        torch.cuda.synchronize()
        for n, b in enumerate(blocks):
            want = states[3 * n + i][3]
            got = (b.q, b.kv, b.turned_q, b.turned_k, b.y, b.out)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            assert torch.equal(b.run()[-1], want[-1])


# ------------------------------------------------- offsets past 32 bits
def sparse(buf, shape, strides, at=0):
    """A view of the buffer, filled with normal values."""
    t = buf.as_strided(shape, strides, at)
    t.copy_(torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(at + sum(shape))))
    return t


def test_rotary_offsets_past_32_bits(S):
    buf = torch.empty(5 * 2 ** 30, dtype=torch.bfloat16, device="cuda")
    q = sparse(buf, (5, 3, 64), (2 ** 30 - 8, 80, 1))
    k = sparse(buf, (5, 2, 64), (8192, 2 ** 32, 1), 2 ** 20)
    plan, positions = S.RotaryPlan(64, [64]), torch.arange(5, dtype=torch.int32, device="cuda")[:, None]
    want = S.rotary_apply(plan, q.contiguous(), k.contiguous(), positions)
    announce("rotary of rows 2^30 apart and heads 2^32 apart")
    got = S.rotary_apply(plan, q, k, positions, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rotary_of_65536_heads(S):
    """A token's channels, and a workgroup's, past 2^24 and 2^31 if they were not cut: one pair of 256 channels."""
    T, H, D = 300, 65536, 256
    plan = S.RotaryPlan(D, [2], interleaved=False)
    x = torch.randn(T, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    positions = torch.arange(T, dtype=torch.int32, device="cuda")[:, None]
    want, _ = S.rotary_apply(plan, x, None, positions)
    out = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    announce("rotary of 65536 heads of 256")
    S.rotary_apply(plan, x.expand(T, H, D), None, positions, q_out=out)
    for t in range(0, T, 50):
        assert torch.equal(out[t:t + 50], want[t:t + 50].expand(-1, H, D))


@pytest.mark.parametrize("Lq,Lk", [(3, 600), (20, 2600), (200, 600), (200, 2600), (66000, 300)])
@pytest.mark.parametrize("mask", [False, True])
def test_cross_attention_offsets_past_32_bits(S, Lq, Lk, mask):
    """States so far apart that a batch row's span passes 2^32 bytes, batch rows 2^32 elements apart."""
    step = (2 ** 32 // Lk + 256) // 8 * 8        # elements; times Lk: past 2^32 elements
    buf = torch.empty(2 ** 32 + 2 * step * Lk, dtype=torch.float16, device="cuda")
    k = sparse(buf, (2, Lk, 1, 64), (2 ** 32 + 8, step, 64, 1))
    v = sparse(buf, (2, Lk, 1, 64), (2 ** 32 + 8, step, 64, 1), 128)
    q = torch.randn(2, Lq, 1, 64, device="cuda").half()
    m = torch.rand(2, Lk, device="cuda") < 0.6 if mask else None
    want = S.cross_attention(q, k.contiguous(), v.contiguous(), mask=m)
    announce(f"cross over {Lk} states {step} elements apart, Lq={Lq}, {'a mask' if mask else 'no mask'}")
    assert torch.equal(S.cross_attention(q, k, v, mask=m), want)
    if Lq <= 200:
        wide = sparse(buf, (2, Lq, 1, 64), (2 ** 32, 2 ** 32 // Lq // 8 * 8, 64, 1), 256)
        want = S.cross_attention(wide.contiguous(), k, v, mask=m)
        assert torch.equal(S.cross_attention(wide, k, v, mask=m), want)


def test_fp8_linear_offsets_past_32_bits(S):
    g = torch.Generator(device="cuda").manual_seed(3)

    def integers(shape):                          # 0 to 3: sums are exact
        return torch.randint(0, 4, shape, device="cuda", generator=g, dtype=torch.uint8)

    def check(layer, w, x, rows_at, got):
        want = x[rows_at].double() @ w.double().t()
        assert torch.equal(got[rows_at], want.to(got.dtype))

    announce("fp8 linear of rows 2^28 elements apart")
    buf = torch.empty(40 * 2 ** 28, dtype=torch.float16, device="cuda")
    w = integers((96, 264))
    layer = S.Fp8Linear(w.float().to(torch.float8_e4m3fn), torch.ones(1, 3, device="cuda"))
    for M in (2, 20, 40):
        x = buf.as_strided((M, 264), (2 ** 28, 1), 8)
        x.copy_(integers((M, 264)))
        check(layer, w, x, slice(None), S.fp8_linear_forward(layer, x))
    x = buf.as_strided((300, 264), (2 ** 25, 1), 8)
    x.copy_(integers((300, 264)))
    check(layer, w, x, slice(None), S.fp8_linear_forward(layer, x))
    del buf, x

    announce("fp8 linear of 2^20 rows of 4200")
    M, K = 2 ** 20 + 5, 4200
    x = torch.empty(M, K, dtype=torch.float16, device="cuda")
    for i in range(0, M, 2 ** 16):
        x[i:i + 2 ** 16] = integers(x[i:i + 2 ** 16].shape)
    w = integers((33, K))
    layer = S.Fp8Linear(w.float().to(torch.float8_e4m3fn), torch.ones(1, 33, device="cuda"))
    at = torch.tensor([0, 1, 2 ** 18, 2 ** 20 - 1, 2 ** 20, M - 1], device="cuda")
    check(layer, w, x, at, S.fp8_linear_forward(layer, x))
    del x

    announce("fp8 linear of 2^20 channels of 4200")
    N = 2 ** 20                                   # the limit: one more is refused
    with pytest.raises(S.SvdqError):
        S.Fp8Linear(torch.zeros(N + 1, 8, dtype=torch.uint8, device="cuda"), torch.ones(2 ** 13 + 1, 1, device="cuda"))
    w = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
    for i in range(0, N, 2 ** 16):
        w[i:i + 2 ** 16] = integers((min(2 ** 16, N - i), K)).half().to(torch.float8_e4m3fn)
    layer = S.Fp8Linear(w, torch.ones(-(-N // 128), 33, device="cuda"))
    at = torch.tensor([0, 127, 2 ** 18, 2 ** 19 + 70, 2 ** 20 - 2, N - 1], device="cuda")
    picked = w.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
    for M in (1, 8, 50, 70, 130):
        x = integers((M, K)).half()
        got = S.fp8_linear_forward(layer, x)
        assert torch.equal(got[:, at], (x.double() @ picked.t()).half())
