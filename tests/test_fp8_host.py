"""The 8-bit operators on the host, no GPU: every bad argument is refused with
the documented status before any HIP call (fake device pointers, only in calls
that must fail), and by the binding before any pointer reaches the library."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from moe_block_skinny_amd import binding as mb
from tests import fp8_ref as ref

A, MIS, BIG = 0x10000, 0x10004, 1 << 34
lib, bf, f8, f32 = mb.lib, torch.bfloat16, torch.float8_e4m3fn, torch.float32


def test_reference_codes_are_the_formats():
    """The tests' own e4m3 against torch's: every code, ties and the ends of the range."""
    t = torch.arange(256, dtype=torch.uint8).view(f8).double().numpy()
    assert np.array_equal(t, ref.VALUES, equal_nan=True)
    v = np.concatenate([ref.VALUES[:127], (ref.VALUES[:126] + ref.VALUES[1:127]) / 2, np.linspace(0, 448, 4001)])
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).float().to(f8).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(v.astype(np.float32).astype(np.float64)), want)
    for a, s in ((0, 1), (448, 1), (449, 2), (1, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (2.0 ** -140, 2.0 ** -126),
                 (3.4028234e38, 2.0 ** 120)):
        assert ref.group_scale(a) == s


QUANT = dict(layout=0, dtype=mb.DT_BF16, n=1, rows=4, cols=128, X=A, Q=A, scale=A)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=mb.DT_E4M3), mb.EINVAL), (dict(dtype=7), mb.EINVAL), (dict(layout=2), mb.EINVAL), (dict(layout=-1), mb.EINVAL),
    (dict(n=0), mb.EINVAL), (dict(rows=-1), mb.EINVAL), (dict(cols=0), mb.EINVAL), (dict(X=0), mb.EINVAL), (dict(Q=MIS), mb.EINVAL),
    (dict(scale=0), mb.EINVAL), (dict(cols=24), mb.EUNSUPPORTED), (dict(n=1 << 20, rows=1 << 20), mb.EUNSUPPORTED),
    (dict(layout=1, n=1 << 24), mb.EUNSUPPORTED), (dict(layout=1, n=1 << 13, rows=1 << 18), mb.EUNSUPPORTED),
])
def test_quantize_validation(kw, status):
    a = {**QUANT, **kw}
    assert lib.moe_quantize_fp8(*[a[n] for n in QUANT], None) == status
    assert lib.moe_last_error()


GEMM = dict(x_dtype=mb.DT_BF16, B=4, N=64, K=256, X=A, x_scale=None, W=A, w_scale=A, R=None, Y=A, y_dtype=mb.DT_BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(x_dtype=mb.DT_F32), mb.EINVAL), (dict(x_dtype=9), mb.EINVAL), (dict(y_dtype=mb.DT_E4M3), mb.EINVAL), (dict(B=0), mb.EINVAL),
    (dict(N=0), mb.EINVAL), (dict(K=-16), mb.EINVAL), (dict(X=0), mb.EINVAL), (dict(W=MIS), mb.EINVAL), (dict(w_scale=0), mb.EINVAL),
    (dict(Y=MIS), mb.EINVAL), (dict(x_scale=A), mb.EINVAL), (dict(x_dtype=mb.DT_E4M3), mb.EINVAL),
    (dict(x_dtype=mb.DT_E4M3, x_scale=MIS), mb.EINVAL), (dict(R=MIS), mb.EINVAL), (dict(B=65), mb.EUNSUPPORTED),
    (dict(K=40), mb.EUNSUPPORTED), (dict(K=65552), mb.EUNSUPPORTED), (dict(N=(1 << 24) + 1), mb.EUNSUPPORTED),
])
def test_gemm_validation(kw, status):
    a = {**GEMM, **kw}
    assert lib.skinny_gemm_fp8(*[a[n] for n in GEMM], A, BIG, None) == status
    assert lib.moe_last_error()


BLOCK = dict(dtype=mb.DT_BF16, B=2, d=256, E=16, k=4, I=64, Is=32, X=A, Wr=A, bias=None, bias_ld=0)
NAMES = ("W13", "s13", "W2", "s2", "Ws13", "ss13", "Ws2", "ss2")


def block(experts=None, out=A, ids=None, w=None, ws=A, ws_bytes=BIG, **kw):
    a = {**BLOCK, **kw}
    e = {n: A for n in NAMES}
    e.update(experts or {})
    s = mb._ExpertsStruct(*[e[n] for n in NAMES])
    return lib.moe_block_fp8(*[a[n] for n in BLOCK], ctypes.addressof(s), out, ids, w, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=mb.DT_F32), mb.EUNSUPPORTED), (dict(dtype=mb.DT_E4M3), mb.EINVAL), (dict(B=0), mb.EINVAL), (dict(B=65), mb.EUNSUPPORTED),
    (dict(k=17, E=32), mb.EUNSUPPORTED), (dict(k=17), mb.EINVAL), (dict(E=513), mb.EUNSUPPORTED), (dict(d=272), mb.EUNSUPPORTED),
    (dict(d=65568), mb.EUNSUPPORTED), (dict(I=48), mb.EUNSUPPORTED), (dict(I=288), mb.EUNSUPPORTED), (dict(I=0), mb.EINVAL),
    (dict(Is=40), mb.EUNSUPPORTED), (dict(X=0), mb.EINVAL), (dict(Wr=MIS), mb.EINVAL), (dict(out=0), mb.EINVAL),
    (dict(bias=MIS), mb.EINVAL), (dict(bias=A, bias_ld=3), mb.EINVAL), (dict(ids=MIS), mb.EINVAL), (dict(w=MIS), mb.EINVAL),
    (dict(ws=0), mb.EINVAL), (dict(ws_bytes=1024), mb.EWORKSPACE),
] + [(dict(experts={n: 0}), mb.EINVAL) for n in NAMES if n != "Ws13"] + [(dict(experts={n: MIS}), mb.EINVAL) for n in NAMES])
def test_block_validation(kw, status):
    assert block(**kw) == status
    assert lib.moe_last_error()


def test_block_null_experts_and_workspace():
    a = list(BLOCK.values())
    assert lib.moe_block_fp8(*a, None, A, None, None, A, BIG, None) == mb.EINVAL
    need = mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, B=2, d=256, E=16, k=4, I=64, Is=32)
    assert need > 0 and need % 256 == 0
    assert block(ws_bytes=need - 1) == mb.EWORKSPACE
    prev = mb.set_block_schedule("fused")
    try:
        assert block() == mb.EUNSUPPORTED
    finally:
        mb.set_block_schedule(prev)


def test_e4m3_is_no_dtype_of_the_other_calls():
    assert lib.skinny_gemm(mb.DT_E4M3, 4, 64, 256, A, A, A, mb.DT_F32, A, BIG, None) == mb.EINVAL


# ---- binding -------------------------------------------------------------------


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def weight(N=64, K=256):
    w = mb.Fp8Weight.__new__(mb.Fp8Weight)   # the constructor wants GPU memory
    w.N, w.K, w.index = N, K, -1
    w.codes, w.scale = z(N, K, dtype=f8), z(-(-N // 128), -(-K // 128), dtype=f32)
    w._ptrs = (w.codes.data_ptr(), w.scale.data_ptr())
    return w


def test_weight_and_experts_reject():
    for codes, scale, exc in ((z(64, 256), z(1, 2, dtype=f32), TypeError), (z(64, 256, dtype=f8), z(1, 1, dtype=f32), ValueError),
                              (z(64, 256, dtype=f8), z(1, 2), TypeError), (z(256, 64, dtype=f8).t(), z(1, 2, dtype=f32), ValueError),
                              (z(64, dtype=f8), z(1, 2, dtype=f32), ValueError), (z(64, 256, dtype=f8), None, ValueError)):
        with pytest.raises(exc):
            mb.Fp8Weight(codes, scale)
    with pytest.raises(ValueError, match="GPU memory"):
        mb.Fp8Weight(z(64, 256, dtype=f8), z(1, 2, dtype=f32))
    ok = dict(W13=z(4, 64, 256, dtype=f8), s13=z(4, 2, 2, dtype=f32), W2=z(4, 256, 32, dtype=f8), s2=z(4, 2, 1, dtype=f32),
              Ws13=z(64, 256, dtype=f8), ss13=z(2, 2, dtype=f32), Ws2=z(256, 32, dtype=f8), ss2=z(2, 1, dtype=f32))
    with pytest.raises(ValueError, match="GPU memory"):
        mb.Fp8Experts(**ok)
    for over, exc in ((dict(s13=z(4, 1, 2, dtype=f32)), ValueError), (dict(W2=z(4, 32, 256, dtype=f8)), ValueError),
                      (dict(W13=z(4, 63, 256, dtype=f8)), ValueError), (dict(ss2=None), ValueError), (dict(Ws13=None), ValueError),
                      (dict(ss13=z(2, 2)), TypeError), (dict(W13=z(4, 64, 256)), TypeError)):
        with pytest.raises(exc):
            mb.Fp8Experts(**{**ok, **over})


def test_gemm_rejects():
    w = weight()
    for args, kw, exc in (((z(4, 128), w, z(4, 64)), {}, ValueError), ((z(4, 256, dtype=f32), w, z(4, 64)), {}, TypeError),
                          ((z(4, 256), w, z(4, 63)), {}, ValueError), ((z(4, 256), w, z(4, 64, dtype=torch.float16)), {}, TypeError),
                          ((z(4, 256), w, z(4, 64)), dict(x_scale=z(4, 2, dtype=f32)), ValueError),
                          ((z(4, 256, dtype=f8), w, z(4, 64)), {}, ValueError),
                          ((z(4, 256, dtype=f8), w, z(4, 64)), dict(x_scale=z(4, 1, dtype=f32)), ValueError),
                          ((z(4, 256), w, z(4, 64)), dict(R=z(4, 64, dtype=f32)), TypeError),
                          ((z(4, 256), z(64, 256, dtype=f8), z(4, 64)), {}, TypeError), ((z(256, 4).t(), w, z(4, 64)), {}, ValueError),
                          ((z(4, 256), w, z(4, 64)), dict(ws=z(64)), TypeError), ((None, w, z(4, 64)), {}, TypeError)):
        with pytest.raises(exc):
            mb.skinny_gemm_fp8(*args, **kw)
    with pytest.raises(ValueError, match="GPU memory"):
        mb.skinny_gemm_fp8(z(4, 256), w, z(4, 64))


def test_quantize_rejects():
    X, Q, S = z(4, 256), z(4, 256, dtype=f8), z(4, 2, dtype=f32)
    for args, exc in (((X, Q, S, "columns"), ValueError), ((X, Q, S, "blocks"), ValueError), ((X, z(4, 256), S, "rows"), TypeError),
                      ((X, z(4, 128, dtype=f8), S, "rows"), ValueError), ((X, Q, z(4, 2), "rows"), TypeError),
                      ((z(4, 256, dtype=torch.float16), Q, S, "rows"), TypeError), ((z(256), Q, S, "rows"), ValueError),
                      ((z(256, 4).t(), Q, S, "rows"), ValueError), ((None, Q, S, "rows"), TypeError), ((X, None, S, "rows"), ValueError)):
        with pytest.raises(exc):
            mb.moe_quantize_fp8(*args)
    with pytest.raises(ValueError, match="GPU memory"):
        mb.moe_quantize_fp8(X, Q, S, "rows")


def test_block_rejects():
    e = mb.Fp8Experts.__new__(mb.Fp8Experts)
    e.E, e.d, e.I, e.Is, e.index, e._ref = 8, 64, 32, 0, -1, None
    ok = dict(X=z(2, 64), Wr=z(8, 64), k=2, experts=e, out=z(2, 64), ws=z(1024, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU memory"):
        mb.moe_block_fp8(**ok)
    for over, exc in ((dict(X=z(2, 32)), ValueError), (dict(Wr=z(7, 64)), ValueError), (dict(out=z(2, 64, dtype=f32)), TypeError),
                      (dict(ws=None), ValueError), (dict(ws=z(4)), TypeError), (dict(experts=None), TypeError),
                      (dict(bias=z(8, dtype=f32), bias_ld=3), ValueError), (dict(bias=z(8, dtype=f32), bias_ld=8), ValueError),
                      (dict(topk_ids=z(2, 2, dtype=torch.int64)), TypeError), (dict(topk_w=z(2, 3, dtype=f32)), ValueError)):
        with pytest.raises(exc):
            mb.moe_block_fp8(**{**ok, **over})


# ---- sizes past the scope --------------------------------------------------------


QUERIES = r"""
from moe_block_skinny_amd import binding as mb
top = 2 ** 31 - 1
for B in (1, 17, 64, 65, 1 << 20, 1 << 24, top):
    for N in (1, 6400, 1 << 24, top):
        for K in (16, 4096, 65536, top):
            got = mb.workspace_bytes(mb.OP_SKINNY_GEMM_FP8, mb.DT_BF16, B=B, N=N, K=K)
            if B > 64 or N > 1 << 24 or K > 65536:
                assert got == 0, (B, N, K, got)
ok = dict(B=64, d=256, E=16, k=4, I=64, Is=32)
assert mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, **ok) > 0
for name, bad in (("B", (65, 1 << 24, top)), ("d", (65568, top)), ("E", (513, top)), ("k", (17, top)),
                  ("I", (-32, 257, top)), ("Is", (-32, 257, top))):
    for v in bad:
        assert mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, **{**ok, name: v}) == 0, (name, v)
"""


def test_workspace_queries_past_the_scope():
    # in a process of its own: a query that divided by a size that had wrapped to zero ended the process
    r = subprocess.run([sys.executable, "-c", QUERIES], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def test_binding_refuses_sizes_past_31_bits():
    # a C int keeps their low bits: [2^32 + 8][16] would be taken for 8 rows
    def big(*shape, dtype=bf):
        return torch.empty(shape, dtype=dtype, device="meta")

    n = 2 ** 32 + 8
    with pytest.raises(ValueError, match="2147483647"):
        mb.moe_quantize_fp8(big(n, 16), big(n, 16, dtype=f8), big(n, 1, dtype=f32), "rows")
    with pytest.raises(ValueError, match="2147483647"):
        mb.moe_quantize_fp8(big(n, 2, 16), big(n, 2, 16, dtype=f8), big(n, 2, 1, dtype=f32), "rows")
    with pytest.raises(ValueError, match="2147483647"):
        mb.skinny_gemm_fp8(big(n, 256), weight(), big(n, 64))
    with pytest.raises(ValueError, match="2147483647"):
        mb.Fp8Weight(big(n, 16, dtype=f8), big((n + 127) // 128, 1, dtype=f32))
    with pytest.raises(ValueError, match="2147483647"):
        mb.Fp8Experts(big(n, 64, 32, dtype=f8), big(n, 2, 1, dtype=f32), big(n, 32, 32, dtype=f8), big(n, 1, 1, dtype=f32))
    e = mb.Fp8Experts.__new__(mb.Fp8Experts)
    e.E, e.d, e.I, e.Is, e.index, e._ref = 8, 64, 32, 0, -1, None
    with pytest.raises(ValueError, match="2147483647"):
        mb.moe_block_fp8(z(2, 64), z(8, 64), n, e, z(2, 64), z(1024, dtype=torch.uint8))
