"""Refusals of the norm, INT8 head and distillation entry points, without a GPU: every call
here is rejected by validation, or returns early for an empty problem, before any HIP call.
The addresses are never dereferenced."""
import math

import pytest

A16 = 1 << 20            # 16-byte aligned
B16 = 1 << 21
C16 = 1 << 22
BIG = 2**63 - 1
INVALID, UNSUPPORTED = 1, 2
E4M3, INT8 = 0, 1
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _norm(m, X=A16, ldx=64, R=B16, ldr=64, nsrc=100, d=64, i=BF16, gain=A16, g=BF16, eps=1e-6, idx=A16, count=None,
          rows=10, sum=None, lds=64, out=C16, code=INT8, q=None, sc=None):
    return m.lib.mosaic_add_rmsnorm(X, ldx, R, ldr, nsrc, d, i, gain, g, eps, idx, count, rows, sum, lds, out, code,
                                    q, sc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nsrc=-1), INVALID), (dict(d=-1), INVALID), (dict(rows=-1), INVALID), (dict(d=0), INVALID),
    (dict(nsrc=0), INVALID), (dict(i=2), INVALID), (dict(g=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=2.0 ** -127), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(X=None), INVALID), (dict(gain=None), INVALID), (dict(out=None), INVALID),
    (dict(q=A16), INVALID), (dict(q=A16, sc=A16, code=2), INVALID), (dict(q=A16, sc=A16, code=-1), INVALID),
    (dict(ldx=63), INVALID), (dict(ldr=63), INVALID), (dict(sum=C16 + 4096, lds=63), INVALID),
    (dict(idx=None, rows=101), INVALID),
    (dict(X=A16 + 1), INVALID), (dict(R=A16 + 1), INVALID), (dict(out=A16 + 1), INVALID), (dict(gain=A16 + 1), INVALID),
    (dict(idx=A16 + 2), INVALID), (dict(count=A16 + 2), INVALID), (dict(q=A16, sc=A16 + 2), INVALID),
    (dict(i=F32, X=A16 + 2), INVALID), (dict(sum=C16 + 1), INVALID),
    (dict(sum=A16), INVALID), (dict(sum=B16), INVALID),                         # in place, but gathered
    (dict(idx=None, sum=A16, lds=65), INVALID), (dict(idx=None, sum=B16, lds=72), INVALID),   # another stride
    (dict(out=A16), INVALID), (dict(out=B16), INVALID), (dict(sum=C16), INVALID),
    (dict(nsrc=BIG, ldx=BIG), INVALID), (dict(ldx=2**62, nsrc=2**10), INVALID),
    (dict(nsrc=2**31), UNSUPPORTED), (dict(rows=2**31), UNSUPPORTED),
    (dict(d=2**30 + 1, ldx=2**31, ldr=2**31), UNSUPPORTED),
])
def test_norm_refusals(m, kw, status):
    assert _norm(m, **kw) == status


def test_norm_empty(m):
    assert _norm(m, rows=0, X=None, R=None, gain=None, out=None, idx=None) == 0


def _quant(m, X=A16, nsrc=100, d=64, i=BF16, idx=A16, rows=10, q=A16, sc=A16):
    return m.lib.mosaic_quantize_rows_int8(X, nsrc, d, i, idx, rows, q, sc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nsrc=-1), INVALID), (dict(d=-1), INVALID), (dict(rows=-1), INVALID), (dict(i=7), INVALID),
    (dict(X=None), INVALID), (dict(q=None), INVALID), (dict(sc=None), INVALID), (dict(nsrc=0), INVALID),
    (dict(idx=None, rows=101), INVALID), (dict(X=A16 + 1), INVALID), (dict(sc=A16 + 2), INVALID),
    (dict(idx=A16 + 1), INVALID), (dict(nsrc=BIG, d=8), INVALID),
    (dict(nsrc=2**31), UNSUPPORTED), (dict(rows=2**31), UNSUPPORTED), (dict(d=2**30 + 1), UNSUPPORTED),
])
def test_quantize_int8_refusals(m, kw, status):
    assert _quant(m, **kw) == status
    assert _quant(m, rows=0, X=None, q=None, sc=None) == 0 and _quant(m, d=0, X=None) == 0


def _head(m, code=INT8, hq=A16, hs=A16, M=10, count=None, wq=A16, ws=A16, V=50, d=128, out=A16, o=BF16):
    return m.lib.mosaic_quantized_logits(code, hq, hs, M, count, wq, ws, V, d, out, o, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(d=-1), INVALID), (dict(d=0), INVALID),
    (dict(o=2), INVALID), (dict(code=2), INVALID), (dict(code=-1), INVALID),
    (dict(hq=None), INVALID), (dict(hs=None), INVALID), (dict(wq=None), INVALID), (dict(ws=None), INVALID),
    (dict(out=None), INVALID), (dict(out=A16 + 8), INVALID), (dict(hs=A16 + 2), INVALID), (dict(ws=A16 + 2), INVALID),
    (dict(count=A16 + 2), INVALID), (dict(M=2**40, V=2**30), INVALID),
    (dict(d=131072), UNSUPPORTED), (dict(M=2**31), UNSUPPORTED), (dict(V=2**31, M=1), UNSUPPORTED),
    (dict(M=2**20, V=2**17), UNSUPPORTED),                                       # 2^25 tiles
    (dict(code=E4M3, o=F32), UNSUPPORTED), (dict(code=E4M3, d=64), UNSUPPORTED),
    (dict(code=E4M3, count=A16), UNSUPPORTED), (dict(code=E4M3, hq=A16 + 8), INVALID),
    (dict(code=E4M3, wq=A16 + 8), INVALID), (dict(code=E4M3, ws=A16 + 4), INVALID),
])
def test_quantized_logits_refusals(m, kw, status):
    assert _head(m, **kw) == status
    assert _head(m, M=0, hq=None, hs=None, out=None) == 0 and _head(m, V=0, wq=None, ws=None, out=None) == 0


def _masked(m, H=A16, L=100, d=64, i=BF16, idx=A16, M=10, wq=A16, ws=A16, V=50, out=A16, C=0, o=BF16, w=A16,
            wb=1 << 20):
    return m.lib.mosaic_masked_logits_int8(H, L, d, i, idx, M, wq, ws, V, out, C, o, w, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(L=-1), INVALID), (dict(d=-1), INVALID), (dict(i=3), INVALID),
    (dict(o=3), INVALID), (dict(L=0), INVALID), (dict(d=0), INVALID),
    (dict(H=None), INVALID), (dict(idx=None), INVALID), (dict(wq=None), INVALID), (dict(ws=None), INVALID),
    (dict(out=None), INVALID), (dict(w=None), INVALID), (dict(w=A16 + 8), INVALID), (dict(out=A16 + 8), INVALID),
    (dict(H=A16 + 1), INVALID), (dict(idx=A16 + 1), INVALID), (dict(ws=A16 + 1), INVALID),
    (dict(M=2**40, V=2**30), INVALID), (dict(L=2**31), UNSUPPORTED), (dict(d=131072, wb=1 << 30), UNSUPPORTED),
])
def test_masked_logits_int8_refusals(m, kw, status):
    assert _masked(m, **kw) == status


def test_masked_logits_int8_workspace(m):
    f = m.mosaic_logits_int8_workspace_bytes
    assert f(10, 0, 64) == 10 * 64 + 40 and f(10, 3, 5) == 16 + 12 and f(0, 0, 5) == 0
    for M, C, d in ((10, 0, 64), (10, 3, 5), (1001, 100, 300)):
        assert _masked(m, M=M, C=C, d=d, wb=f(M, C, d) - 1) == INVALID
    with pytest.raises(ValueError):
        f(-1, 0, 64)
    with pytest.raises(ValueError):
        f(2**60, 0, 64)
    assert _masked(m, M=0, H=None, idx=None, out=None, w=None) == 0 and _masked(m, V=0, wq=None, out=None) == 0


def _distill(m, z=A16, ldz=50, M=10, V=50, dt=BF16, t=A16, tt=F32, ids=A16, K=4, T=1.0, count=None, loss=A16,
             stats=A16, gl=None, grad=None, ldg=50, w=A16, wb=1 << 30):
    return m.lib.mosaic_distill_topk(z, ldz, M, V, dt, t, tt, ids, K, T, count, loss, stats, gl, grad, ldg, w, wb,
                                     None)


def _grad(m, z=A16, ldz=50, M=10, V=50, dt=BF16, t=A16, tt=F32, ids=A16, K=4, T=1.0, count=None, stats=A16, gl=None,
          grad=B16, ldg=50):
    return m.lib.mosaic_distill_topk_grad(z, ldz, M, V, dt, t, tt, ids, K, T, count, stats, gl, grad, ldg, None)


SHARED = [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(K=-1), INVALID), (dict(V=0, ldz=0), INVALID),
    (dict(dt=2), INVALID), (dict(tt=2), INVALID), (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID),
    (dict(T=math.nan), INVALID), (dict(T=math.inf), INVALID), (dict(T=2.0**-21), INVALID), (dict(T=2.0**21), INVALID),
    (dict(z=None), INVALID), (dict(t=None), INVALID), (dict(ids=None), INVALID), (dict(stats=None), INVALID),
    (dict(ldz=49), INVALID), (dict(grad=B16, ldg=49), INVALID), (dict(grad=A16, ldg=51), INVALID),
    (dict(z=A16 + 1), INVALID), (dict(grad=B16 + 1), INVALID), (dict(t=A16 + 2), INVALID), (dict(ids=A16 + 2), INVALID),
    (dict(count=A16 + 2), INVALID), (dict(gl=A16 + 2), INVALID), (dict(stats=A16 + 4), INVALID),
    (dict(ldz=2**61, M=2**10), INVALID),
    (dict(K=1025), UNSUPPORTED), (dict(M=2**31), UNSUPPORTED), (dict(V=2**30 + 1, ldz=2**31, ldg=2**31), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", SHARED)
def test_distill_refusals(m, kw, status):
    assert _distill(m, **kw) == status
    assert _grad(m, **kw) == status


def test_distill_refusals_of_one(m):
    assert _distill(m, loss=None) == INVALID and _distill(m, loss=A16 + 2) == INVALID
    assert _distill(m, w=A16 + 8) == INVALID
    assert _grad(m, grad=None) == INVALID
    assert _distill(m, M=0, z=None, t=None, ids=None, loss=None, stats=None) == 0
    assert _grad(m, M=0, z=None, t=None, ids=None, stats=None, grad=None) == 0


def test_distill_workspace(m):
    f = m.mosaic_distill_topk_workspace_bytes
    with pytest.raises(ValueError):
        f(-1, 5, 5)
    with pytest.raises(ValueError):
        f(5, 5, 1025)
    # the loss alone and the gradient may split rows at different lengths: one size serves both
    assert all(f(M, V, 4) >= 4 * M * (2 + 4) for M in (1, 2, 128) for V in (16384, 102400, 102401, 204801, 1 << 30))
    for M, V in ((1, 152064), (20, 152064), (20, 126464), (700, 126464), (4096, 126464), (3, 100)):
        need = f(M, V, 4)
        assert need >= 0
        if need:
            assert _distill(m, M=M, V=V, ldz=V, wb=need - 1) == INVALID
            assert _distill(m, M=M, V=V, ldz=V, w=None, wb=need) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes(m):
    import torch
    x, g = torch.zeros(4, 8), torch.ones(8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: m.mosaic_add_rmsnorm(x, g), lambda: m.mosaic_quantize_rows_int8(x),
                 lambda: m.mosaic_quantized_logits(x.to(torch.int8), g, x.to(torch.int8), g),
                 lambda: m.mosaic_masked_logits_int8(x, i[:, 0].contiguous(), x.to(torch.int8), g),
                 lambda: m.mosaic_distill_topk(x, i.float(), i),
                 lambda: m.mosaic_distill_topk_grad(x, i.float(), i, i.float()),
                 lambda: m.mosaic_add_rmsnorm(x[0], g), lambda: m.mosaic_add_rmsnorm(x, g[:4]),
                 lambda: m.mosaic_add_rmsnorm(x, g, code=5), lambda: m.mosaic_distill_topk(x[0], i, i)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        m.mosaic_quantized_logits(x, g, x, g)
