"""The 8-bit operators on the GPU against their 64-bit definitions (needs an
MI355X).

Tolerances.  A product of a code and an activation is exact in fp32 (4 and 8
significant bits).  Sums of K products in any order, the block scales applied
to block sums: 2 K 2^-24 sum |x w| covers the additions, the scale products
and a bf16 or fp32 rounding is counted on top (half a step: 2^-8 and 2^-24
relative).  The block's bars are those of the bf16 block (tests/gpu_util.py).
"""
import numpy as np
import pytest
import torch

from moe_block_skinny_amd import binding as mb
from moe_block_skinny_amd import synth
from tests import fp8_ref as ref
from tests.gpu_util import check_block_output, dev, host, rms, say, widen

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def rng(*key):
    return np.random.default_rng([int(k) for k in key])


def dev8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(F8)


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def bf16(a):
    return synth.to_bf16_bits(np.asarray(a, np.float32))


class Guarded:
    """A tensor inside a larger buffer of a fixed pattern: nothing beside it may be written."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.n, self.buf = n, torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.buf[256:256 + n].view(dtype).view(shape)

    def check(self):
        b = self.buf.cpu().numpy()
        assert (b[:256] == 0xA5).all() and (b[256 + self.n:] == 0xA5).all(), "bytes beside the output were written"


# ---- quantiser ---------------------------------------------------------------


def hard_values(r, n, rows, cols):
    """Rows of different sizes, a block of zeros, exact ties, the largest of a group at and next to 448 times a
    power of two, subnormals, the largest finite values."""
    x = r.standard_normal((n, rows, cols)) * np.exp2(6 * r.standard_normal((n, rows, 1)))
    x[:, ::3, :16] = np.exp2(r.integers(-3, 9, (n, len(range(0, rows, 3)), 16))) * 1.0625
    x[:, ::5, -1] = 448.0 * np.exp2(r.integers(-20, 20, (n, len(range(0, rows, 5)))))
    x[:, 1::7, -2] = 450.0
    if cols > 128:
        x[:, :, 128:256] = 0.0
    if rows > 2:
        x[:, 2, :] = 2.0 ** -133 * r.integers(0, 9, cols)
    if rows > 4:
        x[:, 4, :] = 3.3e38 * r.choice([-1.0, 1.0, 0.5], cols)
    return x


@pytest.mark.parametrize("layout", ["rows", "blocks"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 16), (1, 3, 128), (2, 5, 144), (1, 130, 272), (3, 129, 1040), (1, 61, 4112)])
def test_quantize_bit_exact(layout, dtype, n, rows, cols):
    x = hard_values(rng(1, n, rows, cols), n, rows, cols)
    xh = bf16(x) if dtype == "bf16" else x.astype(np.float32)
    q, s = ref.quantize(widen(xh), layout)
    Q, S = Guarded((n, rows, cols), F8), Guarded(s.shape, torch.float32)
    mb.moe_quantize_fp8(dev(xh), Q.t, S.t, layout)
    torch.cuda.synchronize()
    assert np.array_equal(host(S.t), s)
    assert np.array_equal(codes_of(Q.t), q)
    Q.check()
    S.check()


@pytest.mark.parametrize("layout", ["rows", "blocks"])
def test_quantize_two_dimensions_and_not_finite(layout):
    x = rng(2).standard_normal((1, 40, 272))
    x[0, 3, 5], x[0, 3, 200], x[0, 7, 270] = np.inf, np.nan, -np.inf
    x[0, 9, :128] = np.nan
    xh = x.astype(np.float32)
    q, s = ref.quantize(widen(xh), layout)
    Q = torch.empty((40, 272), dtype=F8, device="cuda")
    S = torch.empty(s.shape[1:], dtype=torch.float32, device="cuda")
    mb.moe_quantize_fp8(dev(xh[0]), Q, S, layout)
    assert np.array_equal(host(S), s[0])
    got, want = ref.VALUES[codes_of(Q)], ref.VALUES[q[0]]
    assert np.array_equal(got, want, equal_nan=True)


# ---- dense product -------------------------------------------------------------


class Dense:
    def __init__(self, B, N, K, xt, seed=0):
        r = rng(3, B, N, K, seed)
        self.B, self.N, self.K, self.xt = B, N, K, xt
        self.w = ref.encode(np.clip(r.standard_normal((N, K)) * 107, -448, 448))
        self.ws = ((1 + 0.5 * r.random((ref.blocks(N), ref.blocks(K)))) * K ** -0.5 / 107).astype(np.float32)
        self.R = bf16(r.standard_normal((B, N)))
        if xt == "e4m3":
            self.x = ref.encode(np.clip(r.standard_normal((B, K)) * 128, -448, 448))
            self.xs = (np.exp2(r.integers(-9, -5, (B, ref.blocks(K)))) * (1 + r.random((B, 1)))).astype(np.float32)
            self.X64 = ref.VALUES[self.x] * np.repeat(self.xs.astype(np.float64), 128, axis=1)[:, :K]
            self.args = (dev8(self.x), dev(self.xs))
        else:
            self.x = bf16(r.standard_normal((B, K)))
            self.X64 = widen(self.x)
            self.args = (dev(self.x), None)
        self.W64 = ref.dequantize(self.w, self.ws)
        self.weight = mb.Fp8Weight(dev8(self.w), dev(self.ws))
        need = mb.workspace_bytes(mb.OP_SKINNY_GEMM_FP8, mb.DT_E4M3 if xt == "e4m3" else mb.DT_BF16, B=B, N=N, K=K)
        self.ws_buf = mb.workspace(need) if need else None

    def call(self, Y, R=None, stream=None):
        mb.skinny_gemm_fp8(self.args[0], self.weight, Y, x_scale=self.args[1], R=R, ws=self.ws_buf, stream=stream)

    def check(self, got, residual, out):
        Y = self.X64 @ self.W64.T
        sums = np.abs(self.X64) @ np.abs(self.W64).T
        if residual:
            Y = Y + widen(self.R)
            sums = sums + np.abs(widen(self.R))
        tol = 2.0 * (self.K + 2) * 2.0 ** -24 * sums
        tol += (np.abs(Y) + tol) * (2.0 ** -8 if out == "bf16" else 2.0 ** -24)
        err = np.abs(got - Y)
        bad = ~(err <= tol)
        assert not bad.any(), "%d of %d off, worst %.3g of the bound" % (bad.sum(), bad.size, float((err / tol).max()))


SHAPES = [(1, 1, 16), (1, 7168, 2048), (2, 17, 48), (3, 130, 128), (4, 1001, 144), (5, 16, 7168), (7, 33, 1040), (8, 2304, 1040),
          (9, 130, 2048), (15, 20, 272), (16, 100, 7168), (17, 1001, 1040), (31, 48, 144), (32, 7, 2048), (33, 1001, 1040),
          (48, 64, 272), (49, 130, 144), (63, 40, 8208), (64, 257, 2048), (64, 1, 16), (20, 6408, 4112),
          (40, 300, 4096)]


@pytest.mark.parametrize("xt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N,K", SHAPES)
def test_gemm_against_64_bits(B, N, K, xt):
    c = Dense(B, N, K, xt)
    for out, residual in (("f32", False), ("bf16", True), ("bf16", False), ("f32", True)):
        Y = Guarded((B, N), torch.float32 if out == "f32" else torch.bfloat16)
        c.call(Y.t, dev(c.R) if residual else None)
        torch.cuda.synchronize()
        c.check(host(Y.t), residual, out)
        Y.check()


@pytest.mark.parametrize("B,N,K", [(5, 33, 2048), (6, 100, 2064), (8, 1001, 2176), (8, 40, 4112), (7, 257, 8208), (33, 300, 7168)])
def test_gemm_rows_of_several_steps(B, N, K):
    # 5 to 8 tokens on both sides of the row length that changes their layout; K slices of an odd number of blocks
    c = Dense(B, N, K, "bf16")
    for out, residual in (("f32", False), ("bf16", True)):
        Y = Guarded((B, N), torch.float32 if out == "f32" else torch.bfloat16)
        c.call(Y.t, dev(c.R) if residual else None)
        torch.cuda.synchronize()
        c.check(host(Y.t), residual, out)
        Y.check()


@pytest.mark.parametrize("B,N,K,xt", [(17, 100, 4112, "bf16"), (33, 200, 4096, "e4m3"), (64, 100, 4112, "e4m3"), (33, 6400, 4112, "bf16"),
                                      (64, 6401, 4096, "bf16"), (17, 8193, 4096, "bf16"), (34, 8196, 4112, "e4m3"), (49, 8193, 4096, "e4m3"),
                                      (20, 16400, 4096, "e4m3"), (32, 8192, 4096, "bf16"), (64, 8192, 4096, "e4m3"), (32, 4095, 4096, "e4m3")])
def test_gemm_many_tokens_beside_the_limits_of_each_kernel(B, N, K, xt):
    c = Dense(B, N, K, xt)
    Y = Guarded((B, N), torch.bfloat16)
    c.call(Y.t, dev(c.R))
    torch.cuda.synchronize()
    c.check(host(Y.t), True, "bf16")
    Y.check()


@pytest.mark.parametrize("xt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N,K", [(4, 4097, 2032), (4, 40, 2048), (2, 33, 8208), (8, 4096, 2048), (5, 4095, 2048), (7, 4100, 2064), (13, 4096, 144),
                                   (16, 4095, 272)])
def test_gemm_beside_the_limits_of_each_shape(B, N, K, xt):
    # row groups and columns on both sides of where the blocks in flight and the waves change
    c = Dense(B, N, K, xt)
    Y = Guarded((B, N), torch.bfloat16)
    c.call(Y.t, dev(c.R))
    torch.cuda.synchronize()
    c.check(host(Y.t), True, "bf16")
    Y.check()


@pytest.mark.parametrize("B,N,K,xt", [(3, 130, 400, "bf16"), (20, 130, 400, "bf16"), (20, 130, 400, "e4m3")])
def test_gemm_small_integers_are_exact(B, N, K, xt):
    """Codes of small integers, scales of powers of two: every sum is exact in fp32, whatever its order."""
    r = rng(4, B)
    w, x = r.integers(-3, 4, (N, K)).astype(np.float64), r.integers(-3, 4, (B, K)).astype(np.float64)
    ws = np.exp2(r.integers(-2, 3, (ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    xs = np.exp2(r.integers(-2, 3, (B, ref.blocks(K)))).astype(np.float32) if xt == "e4m3" else None
    want = (x * (np.repeat(xs, 128, axis=1)[:, :K] if xs is not None else 1.0)) @ (w * ref.spread(ws, N, K)).T
    Y = torch.empty((B, N), dtype=torch.float32, device="cuda")
    X = dev8(ref.encode(x)) if xt == "e4m3" else dev(bf16(x))
    mb.skinny_gemm_fp8(X, mb.Fp8Weight(dev8(ref.encode(w)), dev(ws)), Y, x_scale=None if xs is None else dev(xs))
    assert np.array_equal(host(Y), want)


@pytest.mark.parametrize("xt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [2, 6, 12, 40])
def test_gemm_every_code_and_what_is_not_finite_stays_in_its_row(B, xt):
    """All 256 codes in the weights; a NaN code marks its own output row only, a NaN activation its own token."""
    N, K = 48, 272
    c = Dense(B, N, K, xt, seed=1)
    c.w[: 16, :256] = np.arange(256, dtype=np.uint8)
    c.w[: 16, [127, 255]] = 0
    c.w[20, 100] = 0x7f
    c.W64 = ref.dequantize(c.w, c.ws)
    c.weight = mb.Fp8Weight(dev8(c.w), dev(c.ws))
    Y = torch.empty((B, N), dtype=torch.float32, device="cuda")
    c.call(Y)
    y = host(Y)
    assert np.isnan(y[:, 20]).all() and np.isfinite(np.delete(y, 20, axis=1)).all()
    keep = [n for n in range(N) if n != 20]
    tol = 2.0 * (K + 2) * 2.0 ** -24 * (np.abs(c.X64) @ np.abs(c.W64[keep]).T) + 1e-30
    want = c.X64 @ c.W64[keep].T
    assert (np.abs(y[:, keep] - want) <= tol + np.abs(want) * 2.0 ** -24).all()
    if xt == "bf16":
        x = c.x.copy()
        x[1, 270] = 0x7f80   # +inf
        mb.skinny_gemm_fp8(dev(x), c.weight, Y)
    else:
        x = c.x.copy()
        x[1, 270] = 0x7f
        mb.skinny_gemm_fp8(dev8(x), c.weight, Y, x_scale=c.args[1])
    z = host(Y)
    assert not np.isfinite(z[1]).any()
    rows = [t for t in range(B) if t != 1]
    assert np.array_equal(z[rows][:, keep], y[rows][:, keep])


@pytest.mark.parametrize("B", [1, 8, 16, 40])
def test_gemm_in_place_residual_and_other_streams(B):
    c = Dense(B, 500, 1040, "bf16", seed=2)
    Y = torch.empty((B, 500), dtype=torch.bfloat16, device="cuda")
    c.call(Y, dev(c.R))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    Z = dev(c.R)
    side.wait_stream(torch.cuda.current_stream())
    c.call(Z, Z, stream=side)
    side.synchronize()
    assert torch.equal(Y.view(torch.int16), Z.view(torch.int16))
    with torch.cuda.stream(side):
        Z2 = dev(c.R)
        c.call(Z2, Z2)
    side.synchronize()
    assert torch.equal(Y.view(torch.int16), Z2.view(torch.int16))


# ---- the block -------------------------------------------------------------------


class Moe:
    def __init__(self, B, d, E, k, I, Is, routing="plain", seed=0):
        r = rng(5, B, d, E, k, I, Is, seed)
        self.B, self.d, self.E, self.k, self.I, self.Is = B, d, E, k, I, Is
        self.Wr = bf16(r.standard_normal((E, d)) * d ** -0.5)
        self.bias, self.bias_ld, full = None, 0, np.zeros((1, E))
        if routing == "zipf":
            self.bias = (-1.1 * np.log(r.permutation(E) + 1)).astype(np.float32)
            full = self.bias[None].astype(np.float64)
        # tokens whose choice does not hang on the order of a sum
        rows, noise = [], []
        while len(rows) < B:
            x = bf16(r.standard_normal(d))
            g = -np.log(-np.log(r.random(E))).astype(np.float32) if routing == "gumbel" else None
            l = np.sort(widen(self.Wr) @ widen(x) + (g.astype(np.float64) if g is not None else full[0]))[::-1]
            if k == E or l[k - 1] - l[k] >= 1e-3:
                rows.append(x)
                noise.append(g)
        self.x = np.stack(rows)
        if routing == "gumbel":
            self.bias, self.bias_ld = np.stack(noise), E
            full = self.bias.astype(np.float64)
        self.full = full

        def w(shape, fan, blk):
            return (ref.encode(np.clip(r.standard_normal(shape) * 107, -448, 448)),
                    ((1 + 0.5 * r.random(blk)) * fan ** -0.5 / 107).astype(np.float32))

        b = ref.blocks
        self.W13, self.s13 = w((E, 2 * I, d), d, (E, 2 * b(I), b(d)))
        self.W2, self.s2 = w((E, d, I), I, (E, b(d), b(I)))
        self.shared = None
        extra = []
        if Is:
            self.Ws13, self.ss13 = w((2 * Is, d), d, (2 * b(Is), b(d)))
            self.Ws2, self.ss2 = w((d, Is), Is, (b(d), b(Is)))
            self.shared = (ref.dequantize13(self.Ws13, self.ss13), ref.dequantize(self.Ws2, self.ss2))
            extra = [dev8(self.Ws13), dev(self.ss13), dev8(self.Ws2), dev(self.ss2)]
        self.experts = mb.Fp8Experts(dev8(self.W13), dev(self.s13), dev8(self.W2), dev(self.s2), *extra)
        self.X, self.gWr = dev(self.x), dev(self.Wr)
        self.gbias = None if self.bias is None else dev(self.bias)
        self.ws = mb.workspace(mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, B=B, d=d, E=E, k=k, I=I, Is=Is))

    def call(self, out, ids=None, w=None, X=None, stream=None, ws=None):
        mb.moe_block_fp8(self.X if X is None else X, self.gWr, self.k, self.experts, out, self.ws if ws is None else ws,
                         bias=self.gbias, bias_ld=self.bias_ld, topk_ids=ids, topk_w=w, stream=stream)

    def outputs(self):
        return (Guarded((self.B, self.d), torch.bfloat16), Guarded((self.B, self.k), torch.int32),
                Guarded((self.B, self.k), torch.float32))

    def reference(self):
        return ref.moe(widen(self.x), widen(self.Wr), self.k, lambda e: ref.dequantize13(self.W13[e], self.s13[e]),
                       lambda e: ref.dequantize(self.W2[e], self.s2[e]), self.full, self.shared)


BLOCKS = [
    (1, 32, 4, 1, 32, 0, "plain"), (1, 1024, 32, 8, 128, 128, "plain"), (1, 7168, 24, 8, 128, 128, "plain"),
    (2, 1024, 32, 4, 64, 64, "plain"), (2, 160, 40, 16, 96, 32, "gumbel"), (3, 544, 33, 6, 160, 0, "gumbel"),
    (4, 256, 512, 16, 32, 256, "plain"), (5, 1056, 8, 8, 224, 96, "plain"), (8, 2048, 64, 8, 128, 128, "gumbel"),
    (8, 256, 48, 16, 64, 64, "gumbel"), (9, 256, 32, 2, 256, 256, "zipf"), (16, 1024, 16, 4, 96, 192, "zipf"),
    (17, 96, 5, 5, 32, 32, "plain"), (33, 544, 20, 7, 128, 64, "zipf"), (48, 256, 64, 1, 64, 128, "gumbel"),
    (64, 7168, 20, 8, 256, 256, "zipf"), (64, 8192, 80, 16, 32, 64, "gumbel"), (64, 256, 512, 16, 32, 32, "gumbel"),
    (64, 9248, 3, 2, 64, 0, "plain"),
]


@pytest.mark.parametrize("B,d,E,k,I,Is,routing", BLOCKS)
def test_block_against_64_bits(B, d, E, k, I, Is, routing):
    c = Moe(B, d, E, k, I, Is, routing)
    out, ids, w = c.outputs()
    c.call(out.t, ids.t, w.t)
    torch.cuda.synchronize()
    want, want_ids, want_w = c.reference()
    assert np.array_equal(host(ids.t), want_ids)
    assert np.abs(host(w.t) - want_w).max() <= 1e-5
    say(mb.last_variant(), check_block_output(host(out.t), want))
    for g in (out, ids, w):
        g.check()
    assert mb.workspace_status(c.ws) == 0
    # ids and weights are optional, and the workspace serves the next call as the first left it
    again = torch.empty((B, d), dtype=torch.bfloat16, device="cuda")
    c.call(again)
    assert torch.equal(again.view(torch.int16), out.t.view(torch.int16))


@pytest.mark.parametrize("B,routing", [(1, "plain"), (2, "plain"), (8, "gumbel"), (24, "zipf")])
def test_block_routes_as_the_bf16_block(B, routing):
    """ids and weights bit for bit those of moe_block on the same activations, router and bias, and the output
    that of moe_block over the dequantised weights (powers of two as scales: bf16 holds them exactly) up to the
    order of its sums."""
    c = Moe(B, 512, 48, 4, 64, 64, routing, seed=3)
    c.s13[:] = np.exp2(np.round(np.log2(c.s13)))
    c.s2[:] = np.exp2(np.round(np.log2(c.s2)))
    c.ss13[:] = np.exp2(np.round(np.log2(c.ss13)))
    c.ss2[:] = np.exp2(np.round(np.log2(c.ss2)))
    c.experts = mb.Fp8Experts(dev8(c.W13), dev(c.s13), dev8(c.W2), dev(c.s2), dev8(c.Ws13), dev(c.ss13), dev8(c.Ws2), dev(c.ss2))
    c.shared = (ref.dequantize13(c.Ws13, c.ss13), ref.dequantize(c.Ws2, c.ss2))
    ids, w, out = (torch.empty((B, 4), dtype=torch.int32, device="cuda"), torch.empty((B, 4), device="cuda"),
                   torch.empty((B, 512), dtype=torch.bfloat16, device="cuda"))
    c.call(out, ids, w)
    W13 = np.stack([bf16(ref.dequantize13(c.W13[e], c.s13[e])) for e in range(48)])
    W2 = np.stack([bf16(ref.dequantize(c.W2[e], c.s2[e])) for e in range(48)])
    ids2, w2, out2 = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(out)
    ws = mb.workspace(mb.workspace_bytes(mb.OP_BLOCK, mb.DT_BF16, B=B, d=512, E=48, k=4, I=64, Is=64))
    mb.moe_block(c.X, c.gWr, 4, dev(W13), dev(W2), out2, ws, dev(bf16(c.shared[0])), dev(bf16(c.shared[1])),
                 bias=c.gbias, bias_ld=c.bias_ld, topk_ids=ids2, topk_w=w2)
    assert torch.equal(ids, ids2) and torch.equal(w.view(torch.int32), w2.view(torch.int32))
    want = c.reference()[0]
    check_block_output(host(out), want)
    check_block_output(host(out2), want)


@pytest.mark.parametrize("B", [1, 2, 8, 20])
def test_block_schedules_and_shared_workspace(B):
    """The router in a launch of its own gives the same bits; a workspace of a larger call serves a smaller one
    and calls of moe_block in turn; the fused schedule is refused."""
    c = Moe(B, 256, 32, 4, 64, 64, "plain", seed=4)
    big = mb.workspace(mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, B=64, d=1024, E=64, k=8, I=256, Is=256))
    out = torch.empty((B, 256), dtype=torch.bfloat16, device="cuda")
    a, b = torch.empty_like(out), torch.empty_like(out)
    c.call(out)
    c.call(a, ws=big)
    prev = mb.set_block_schedule("launches")
    try:
        c.call(b, ws=big)
        mb.set_block_schedule("fused")
        with pytest.raises(mb.MoeError) as e:
            c.call(b)
        assert e.value.status == mb.EUNSUPPORTED
    finally:
        mb.set_block_schedule(prev)
    assert torch.equal(out.view(torch.int16), a.view(torch.int16))
    assert torch.equal(out.view(torch.int16), b.view(torch.int16))


def test_block_same_token_in_every_row():
    """64 copies of one token: one expert set, every row the same bits."""
    c = Moe(64, 512, 32, 4, 128, 128, "plain", seed=5)
    X = c.X[:1].expand(64, -1).contiguous()
    out = torch.empty((64, 512), dtype=torch.bfloat16, device="cuda")
    c.call(out, X=X)
    o = out.view(torch.int16)
    assert (o == o[:1]).all()


@pytest.mark.parametrize("B", [1, 2, 8, 40])
def test_graph_replays_of_the_whole_run(B):
    """Quantise the activations, 8-bit projection with residual, block: captured together; replays with eager calls
    on the same buffers in between give the eager bits."""
    c = Moe(B, 512, 32, 4, 64, 64, "plain", seed=6)
    g = Dense(B, 512, 512, "bf16", seed=6)
    X0 = dev(g.x)
    Q = torch.empty((B, 512), dtype=F8, device="cuda")
    S = torch.empty((B, 4), device="cuda")
    H = torch.empty((B, 512), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(H)

    def step(x):
        mb.moe_quantize_fp8(x, Q, S, "rows")
        mb.skinny_gemm_fp8(Q, g.weight, H, x_scale=S, R=x, ws=g.ws_buf)
        c.call(out, X=H)

    step(X0)
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step(X0)
    other = torch.flip(X0, dims=[1]).contiguous()
    for rep in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), rep
        step(other)
    torch.cuda.synchronize()
    # and the run's values: the projection against its definition, the block on what it produced
    step(X0)
    q, s = ref.quantize(g.X64[None], "rows")
    X8 = ref.VALUES[q[0]] * np.repeat(s[0], 128, axis=1)
    Y = X8 @ g.W64.T + g.X64
    assert np.abs(host(H) - Y).max() <= 2.0 ** -8 * np.abs(Y).max() + 1e-4 * rms(Y)


# ---- ends of the ranges, and calls beside each other --------------------------------


@pytest.mark.parametrize("xt,B", [("bf16", 2), ("e4m3", 6), ("bf16", 12), ("e4m3", 64), ("bf16", 64)])
def test_gemm_longest_rows(xt, B):
    c = Dense(B, 70, 65536, xt, seed=7)
    Y = Guarded((B, 70), torch.float32)
    c.call(Y.t)
    c.check(host(Y.t), False, "f32")
    Y.check()


@pytest.mark.parametrize("B", [1, 20])
def test_gemm_weight_past_4_gib(B):
    """Rows beyond 2^32 bytes of the weight: zeros but for the first and the last block row."""
    N, K = 66049, 65536
    W = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
    r = rng(8, B)
    rows = np.r_[0:3, N - 65:N]
    codes = ref.encode(np.clip(r.standard_normal((len(rows), K)) * 107, -448, 448))
    W[torch.from_numpy(rows).cuda()] = torch.from_numpy(codes).cuda()
    S = torch.full((ref.blocks(N), ref.blocks(K)), 2.0 ** -14, device="cuda")
    S[-1] = 2.0 ** -13
    X = bf16(r.standard_normal((B, K)))
    need = mb.workspace_bytes(mb.OP_SKINNY_GEMM_FP8, mb.DT_BF16, B=B, N=N, K=K)
    Y = torch.empty((B, N), dtype=torch.float32, device="cuda")
    mb.skinny_gemm_fp8(dev(X), mb.Fp8Weight(W.view(F8), S), Y, ws=mb.workspace(need) if need else None)
    y = host(Y)
    last = (N - 1) // 128 * 128
    scale = np.where(rows < last, 2.0 ** -14, 2.0 ** -13)
    W64 = ref.VALUES[codes] * scale[:, None]
    want, sums = widen(X) @ W64.T, np.abs(widen(X)) @ np.abs(W64).T
    assert (np.abs(y[:, rows] - want) <= (2.0 * (K + 2) + 1) * 2.0 ** -24 * sums).all()
    y[:, rows] = 0
    assert not y.any()


@pytest.mark.parametrize("layout", ["rows", "blocks"])
def test_quantize_past_4_gib(layout):
    rows, cols = 66049, 65536
    X = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = hard_values(rng(9), 1, 129, cols)
    th = bf16(tail)[0]
    X[rows - 129:] = dev(th)
    Q = torch.empty((rows, cols), dtype=F8, device="cuda")
    S = torch.empty((rows if layout == "rows" else ref.blocks(rows), ref.blocks(cols)), device="cuda")
    mb.moe_quantize_fp8(X, Q, S, layout)
    # the last 128-row block starts at row 66048, one row before the end; the 128 rows ahead of it are one block
    q, s = ref.quantize(widen(th)[None], layout)
    if layout == "blocks":
        q1, s1 = ref.quantize(widen(th[:128])[None], layout)
        q2, s2 = ref.quantize(widen(th[128:])[None], layout)
        q, s = np.concatenate([q1, q2], axis=1), np.concatenate([s1, s2], axis=1)
    assert np.array_equal(codes_of(Q[rows - 129:]), q[0])
    assert np.array_equal(host(S[-s.shape[1]:]), s[0])
    assert not Q[: rows - 129].view(torch.uint8).any() and bool((S[: S.shape[0] - s.shape[1]] == 1).all())


def test_quantize_longest_row():
    # the last group, 112 columns, ends at column 2^31 - 16
    cols, t = 2 ** 31 - 16, 240
    X = torch.zeros((1, cols), dtype=torch.bfloat16, device="cuda")
    th = bf16(hard_values(rng(10), 1, 1, t))[0]
    X[:, cols - t:] = dev(th)
    Q = torch.empty((1, cols), dtype=F8, device="cuda")
    S = torch.empty((1, ref.blocks(cols)), device="cuda")
    mb.moe_quantize_fp8(X, Q, S, "rows")
    q, s = ref.quantize(widen(th)[None], "rows")
    assert np.array_equal(codes_of(Q[:, cols - t:]), q[0])
    assert np.array_equal(host(S[:, -2:]), s[0])
    assert not Q[:, : cols - t].view(torch.uint8).any() and bool((S[:, :-2] == 1).all())


@pytest.mark.parametrize("B", [3, 20])
def test_block_experts_past_4_gib_and_widest_hidden_size(B):
    """d = 65536, and W13 of more than 2^32 bytes with the last expert chosen by every token."""
    d, E, k, I = 65536, 130, 2, 256
    r = rng(10, B)
    g = torch.Generator(device="cuda").manual_seed(B)
    code = lambda *s: torch.randint(0, 0x70, s, generator=g, device="cuda", dtype=torch.uint8)   # noqa: E731
    W13, W2 = code(E, 2 * I, d), code(E, d, I)
    s13 = torch.full((E, 2 * ref.blocks(I), ref.blocks(d)), 2.0 ** -14, device="cuda")
    s2 = torch.full((E, ref.blocks(d), ref.blocks(I)), 2.0 ** -10, device="cuda")
    X = bf16(r.standard_normal((B, d)))
    Wr = bf16(r.standard_normal((E, d)) * d ** -0.5)
    bias = np.zeros(E, np.float32)
    bias[[5, E - 1]] = 50.0
    out = torch.empty((B, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((B, k), dtype=torch.int32, device="cuda")
    ws = mb.workspace(mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, B=B, d=d, E=E, k=k, I=I, Is=0))
    mb.moe_block_fp8(dev(X), dev(Wr), k, mb.Fp8Experts(W13.view(F8), s13, W2.view(F8), s2), out, ws, bias=dev(bias), topk_ids=ids)
    assert np.array_equal(host(ids), np.tile([5, E - 1], (B, 1)))
    full = np.tile(bias.astype(np.float64), (B, 1))
    want, _, _ = ref.moe(widen(X), widen(Wr), k, lambda e: ref.VALUES[W13[e].cpu().numpy()] * 2.0 ** -14,
                         lambda e: ref.VALUES[W2[e].cpu().numpy()] * 2.0 ** -10, full)
    check_block_output(host(out), want)


@pytest.mark.parametrize("variant", ["gemv", "splitk", "mfma"])
def test_block_with_a_forced_router(variant):
    """A forced shape is the router's: same choices, an output within the bars; refused where it does not reach."""
    c = Moe(2, 256, 32, 4, 64, 64, "plain", seed=11)
    out, ids, w = c.outputs()
    prev = mb.set_variant(variant)
    try:
        c.call(out.t, ids.t, w.t)
        big = Moe(20, 256, 32, 4, 64, 64, "plain", seed=11)
        o = torch.empty((20, 256), dtype=torch.bfloat16, device="cuda")
        if variant == "mfma":
            big.call(o)
        else:
            with pytest.raises(mb.MoeError) as e:
                big.call(o)
            assert e.value.status == mb.EUNSUPPORTED
    finally:
        mb.set_variant(prev)
    want, want_ids, _ = c.reference()
    assert np.array_equal(host(ids.t), want_ids)
    check_block_output(host(out.t), want)


@pytest.mark.parametrize("B", [2, 7, 12, 40])
def test_block_a_token_that_is_not_finite_stays_alone(B):
    c = Moe(B, 256, 32, 4, 64, 64, "plain", seed=12)
    a, b = torch.empty((B, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((B, 256), dtype=torch.bfloat16, device="cuda")
    c.call(a)
    X = c.X.clone()
    X[1, 7] = float("nan")
    c.call(b, X=X)
    rows = [t for t in range(B) if t != 1]
    assert torch.equal(a[rows].view(torch.int16), b[rows].view(torch.int16))
    assert mb.workspace_status(c.ws) == 0


def test_one_workspace_serves_every_op_in_turn():
    """Dense with K slices, blocks of 8-bit and of bf16 weights, large and small, over one workspace: each call leaves
    its counters as it found them."""
    g = Dense(40, 300, 4096, "bf16", seed=13)
    assert g.ws_buf is not None
    blocks = [Moe(B, 512, 32, 4, 64, 64, "plain", seed=13) for B in (1, 2, 8, 40)]
    W13 = (torch.randn((32, 128, 512), device="cuda") * 0.04).to(torch.bfloat16)
    W2 = (torch.randn((32, 512, 64), device="cuda") * 0.1).to(torch.bfloat16)
    ws = mb.workspace(max([g.ws_buf.numel()] + [c.ws.numel() for c in blocks] + [
        mb.workspace_bytes(mb.OP_BLOCK, mb.DT_BF16, B=B, d=512, E=32, k=4, I=64, Is=0) for B in (1, 40)]))
    want = []
    for rep in range(3):
        got = []
        for c in blocks:
            o = torch.empty((c.B, 512), dtype=torch.bfloat16, device="cuda")
            c.call(o, ws=ws)
            got.append(o)
            y = torch.empty((40, 300), dtype=torch.float32, device="cuda")
            mb.skinny_gemm_fp8(g.args[0], g.weight, y, ws=ws)
            got.append(y)
            z = torch.empty((c.B, 512), dtype=torch.bfloat16, device="cuda")
            mb.moe_block(c.X, c.gWr, 4, W13, W2, z, ws)
            got.append(z)
        torch.cuda.synchronize()
        want = want or got
        for p, q in zip(want, got):
            assert torch.equal(p, q)


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own: the bits of the calls one after the other."""
    g = Dense(64, 6400, 4096, "e4m3", seed=14)
    c = Moe(8, 1024, 64, 8, 128, 128, "gumbel", seed=14)
    y0, o0 = torch.empty((64, 6400), device="cuda"), torch.empty((8, 1024), dtype=torch.bfloat16, device="cuda")
    g.call(y0)
    c.call(o0)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    y, o = [torch.empty_like(y0) for _ in range(20)], [torch.empty_like(o0) for _ in range(20)]
    for i in range(20):
        g.call(y[i], stream=s)
        c.call(o[i], stream=t)
    torch.cuda.synchronize()
    assert all(torch.equal(y0, v) for v in y) and all(torch.equal(o0, v) for v in o)


def test_shared_kernel_replays():
    """The dense product with K slices in a graph, replayed between eager calls on the same workspace."""
    g = Dense(40, 300, 4096, "e4m3", seed=15)
    h = Dense(64, 300, 4096, "bf16", seed=15)
    ws = mb.workspace(max(g.ws_buf.numel(), h.ws_buf.numel()))
    g.ws_buf = h.ws_buf = ws
    R = dev(g.R)
    Y, Z = torch.empty((40, 300), dtype=torch.bfloat16, device="cuda"), torch.empty((64, 300), device="cuda")
    g.call(Y, R)
    h.call(Z)
    torch.cuda.synchronize()
    y, z = Y.clone(), Z.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        g.call(Y, R)
    for rep in range(4):
        Y.zero_()
        graph.replay()
        h.call(Z)
        torch.cuda.synchronize()
        assert torch.equal(Y, y) and torch.equal(Z, z), rep
