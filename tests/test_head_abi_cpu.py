"""Refusals of the layer norm, MXFP4 head and token log-probability entry points, without a
GPU: every call here is rejected by validation, or returns early for an empty problem, before
any HIP call.  The addresses are never dereferenced."""
import math

import pytest
import torch

A16 = 1 << 20            # 16-byte aligned
B16 = 1 << 21
C16 = 1 << 22
D16 = 1 << 23
BIG = 2**63 - 1
INVALID, UNSUPPORTED = 1, 2
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _norm(m, X=A16, ldx=64, R=B16, ldr=64, nsrc=100, d=64, i=BF16, gain=A16, bias=A16, g=BF16, eps=1e-5, idx=A16,
          count=None, rows=10, sum=None, lds=64, out=C16, stats=None):
    return m.lib.mosaic_add_layernorm(X, ldx, R, ldr, nsrc, d, i, gain, bias, g, eps, idx, count, rows, sum, lds, out,
                                      stats, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nsrc=-1), INVALID), (dict(d=-1), INVALID), (dict(rows=-1), INVALID), (dict(d=0), INVALID),
    (dict(nsrc=0), INVALID), (dict(i=2), INVALID), (dict(g=2), INVALID), (dict(g=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=2.0 ** -127), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(X=None), INVALID), (dict(out=None), INVALID),
    (dict(ldx=63), INVALID), (dict(ldr=63), INVALID), (dict(sum=D16, lds=63), INVALID), (dict(idx=None, rows=101), INVALID),
    (dict(X=A16 + 1), INVALID), (dict(R=A16 + 1), INVALID), (dict(out=A16 + 1), INVALID), (dict(gain=A16 + 1), INVALID),
    (dict(bias=A16 + 1), INVALID), (dict(idx=A16 + 2), INVALID), (dict(count=A16 + 2), INVALID),
    (dict(stats=A16 + 4), INVALID), (dict(i=F32, X=A16 + 2), INVALID), (dict(sum=D16 + 1), INVALID),
    (dict(sum=A16), INVALID), (dict(sum=B16), INVALID),                         # in place, but gathered
    (dict(idx=None, sum=A16, lds=65), INVALID), (dict(idx=None, sum=B16, lds=72), INVALID),   # another stride
    (dict(out=A16), INVALID), (dict(out=B16), INVALID), (dict(sum=C16), INVALID),
    (dict(nsrc=BIG, ldx=BIG), INVALID), (dict(ldx=2**62, nsrc=2**10), INVALID),
    (dict(nsrc=2**31), UNSUPPORTED), (dict(rows=2**31), UNSUPPORTED),
    (dict(d=2**30 + 1, ldx=2**31, ldr=2**31), UNSUPPORTED),
])
def test_layernorm_refusals(m, kw, status):
    assert _norm(m, **kw) == status


def test_layernorm_empty(m):
    assert _norm(m, rows=0, X=None, R=None, gain=None, out=None, idx=None) == 0


def _grad(m, dY=A16, lddy=64, S=B16, lds=64, nsrc=100, d=64, i=BF16, stats=A16, gain=A16, g=BF16, idx=None, count=None,
          rows=10, dsum=None, ldds=64, dX=C16, lddx=64, dg=A16, db=B16, w=A16, wb=1 << 40):
    return m.lib.mosaic_layernorm_grad(dY, lddy, S, lds, nsrc, d, i, stats, gain, g, idx, count, rows, dsum, ldds, dX,
                                       lddx, dg, db, w, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nsrc=-1), INVALID), (dict(d=-1), INVALID), (dict(rows=-1), INVALID), (dict(d=0), INVALID),
    (dict(nsrc=0), INVALID), (dict(i=2), INVALID), (dict(g=5), INVALID), (dict(dY=None), INVALID), (dict(S=None), INVALID),
    (dict(stats=None), INVALID), (dict(dX=None, dg=None, db=None), INVALID), (dict(rows=101), INVALID),
    (dict(lddy=63), INVALID), (dict(lds=63), INVALID), (dict(lddx=63), INVALID), (dict(dsum=D16, ldds=63), INVALID),
    (dict(dY=A16 + 1), INVALID), (dict(S=A16 + 1), INVALID), (dict(stats=A16 + 4), INVALID), (dict(gain=A16 + 1), INVALID),
    (dict(idx=A16 + 1), INVALID), (dict(count=A16 + 1), INVALID), (dict(dsum=D16 + 1), INVALID), (dict(dX=C16 + 1), INVALID),
    (dict(dg=A16 + 2), INVALID), (dict(db=A16 + 2), INVALID), (dict(dg=A16, db=A16), INVALID),
    (dict(w=A16 + 8), INVALID), (dict(w=None), INVALID), (dict(wb=16), INVALID),
    (dict(dX=A16, lddx=65), INVALID), (dict(dX=D16, dsum=D16, lddx=65), INVALID), (dict(dX=B16, lddx=72), INVALID),
    (dict(dX=B16, idx=A16), INVALID), (dict(nsrc=BIG, lds=BIG), INVALID),
    (dict(nsrc=2**31), UNSUPPORTED), (dict(rows=2**31, nsrc=2**31), UNSUPPORTED),
    (dict(d=2**30 + 1, lddy=2**31, lds=2**31, lddx=2**31), UNSUPPORTED),
])
def test_layernorm_grad_refusals(m, kw, status):
    assert _grad(m, **kw) == status


def test_layernorm_grad_workspace(m):
    f = m.mosaic_layernorm_grad_workspace_bytes
    assert f(0, 64) == 0 and f(1, 0) == 0 and f(1, 1) > 0
    for rows, d in ((1, 1), (10, 64), (5000, 1021), (100000, 4096), (3, 20000), (2**31 - 1, 2**20)):
        assert _grad(m, rows=rows, nsrc=rows, d=d, lddy=d, lds=d, lddx=d, wb=f(rows, d) - 1) == INVALID
    for rows, d in ((-1, 4), (4, -1), (2**31, 4), (4, 2**30 + 1)):
        with pytest.raises(ValueError):
            f(rows, d)
    assert _grad(m, rows=0, dY=None, S=None, stats=None, dg=None, db=None, w=None, wb=0) == 0


def _quant(m, X=A16, nsrc=100, d=64, i=BF16, idx=A16, rows=10, q=A16, sc=A16, v=None):
    return m.lib.mosaic_quantize_rows_mxfp4(X, nsrc, d, i, idx, rows, q, sc, v, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nsrc=-1), INVALID), (dict(d=-1), INVALID), (dict(rows=-1), INVALID), (dict(i=7), INVALID),
    (dict(X=None), INVALID), (dict(q=None), INVALID), (dict(sc=None), INVALID), (dict(q=None, sc=None), INVALID),
    (dict(nsrc=0), INVALID), (dict(idx=None, rows=101), INVALID), (dict(X=A16 + 1), INVALID), (dict(q=A16 + 8), INVALID),
    (dict(v=B16 + 1), INVALID), (dict(v=A16), INVALID), (dict(idx=A16 + 1), INVALID), (dict(nsrc=BIG, d=8), INVALID),
    (dict(nsrc=2**31), UNSUPPORTED), (dict(rows=2**31), UNSUPPORTED), (dict(d=2**30 + 1), UNSUPPORTED),
])
def test_quantize_mxfp4_refusals(m, kw, status):
    assert _quant(m, **kw) == status
    assert _quant(m, rows=0, X=None, q=None, sc=None) == 0 and _quant(m, d=0, X=None) == 0


def _head(m, hq=A16, hs=A16, M=10, count=None, wq=A16, ws=A16, V=50, d=128, out=A16, o=BF16):
    return m.lib.mosaic_quantized_logits_mxfp4(hq, hs, M, count, wq, ws, V, d, out, o, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(d=-1), INVALID), (dict(d=0), INVALID), (dict(o=2), INVALID),
    (dict(hq=None), INVALID), (dict(hs=None), INVALID), (dict(wq=None), INVALID), (dict(ws=None), INVALID),
    (dict(out=None), INVALID), (dict(out=A16 + 8), INVALID), (dict(hq=A16 + 8), INVALID), (dict(wq=A16 + 4), INVALID),
    (dict(count=A16 + 2), INVALID), (dict(M=2**40, V=2**30), INVALID), (dict(M=2**50, d=2**25, V=1), INVALID),
    (dict(d=2**25 + 1), UNSUPPORTED), (dict(M=2**31), UNSUPPORTED), (dict(V=2**31, M=1), UNSUPPORTED),
    (dict(M=2**20, V=2**17), UNSUPPORTED),                                       # 2^25 tiles
])
def test_quantized_logits_mxfp4_refusals(m, kw, status):
    assert _head(m, **kw) == status
    assert _head(m, M=0, hq=None, hs=None, out=None) == 0 and _head(m, V=0, wq=None, ws=None, out=None) == 0


def _masked(m, H=A16, L=100, d=64, i=BF16, idx=A16, M=10, wq=A16, ws=A16, V=50, out=A16, C=0, o=BF16, w=A16,
            wb=1 << 30):
    return m.lib.mosaic_masked_logits_mxfp4(H, L, d, i, idx, M, wq, ws, V, out, C, o, w, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(L=-1), INVALID), (dict(d=-1), INVALID), (dict(i=3), INVALID),
    (dict(o=3), INVALID), (dict(L=0), INVALID), (dict(d=0), INVALID),
    (dict(H=None), INVALID), (dict(idx=None), INVALID), (dict(wq=None), INVALID), (dict(ws=None), INVALID),
    (dict(out=None), INVALID), (dict(w=None), INVALID), (dict(w=A16 + 8), INVALID), (dict(out=A16 + 8), INVALID),
    (dict(H=A16 + 1), INVALID), (dict(idx=A16 + 1), INVALID), (dict(wq=A16 + 1), INVALID),
    (dict(M=2**40, V=2**30), INVALID), (dict(L=2**31), UNSUPPORTED), (dict(d=2**25 + 1), UNSUPPORTED),
])
def test_masked_logits_mxfp4_refusals(m, kw, status):
    assert _masked(m, **kw) == status


def test_masked_logits_mxfp4_workspace(m):
    f = m.mosaic_logits_mxfp4_workspace_bytes
    assert f(10, 0, 64) == 10 * 34 and f(10, 3, 33) == 3 * 34 and f(0, 0, 5) == 0
    for M, C, d in ((10, 0, 64), (10, 3, 5), (1001, 100, 300)):
        assert _masked(m, M=M, C=C, d=d, wb=f(M, C, d) - 1) == INVALID
    with pytest.raises(ValueError):
        f(-1, 0, 64)
    with pytest.raises(ValueError):
        f(2**62, 0, 64)
    assert _masked(m, M=0, H=None, idx=None, out=None, w=None) == 0 and _masked(m, V=0, wq=None, out=None) == 0


def _score(m, z=A16, ldz=500, M=10, V=500, t=BF16, tok=A16, T=1.0, count=None, lp=A16, H=None, n=3, ids=A16, top=A16,
           st=A16, w=A16, wb=1 << 30):
    return m.lib.mosaic_token_logprobs(z, ldz, M, V, t, tok, T, count, lp, H, n, ids, top, st, w, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(V=0), INVALID), (dict(n=-1), INVALID), (dict(t=2), INVALID),
    (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID), (dict(T=math.nan), INVALID), (dict(T=2.0 ** 21), INVALID),
    (dict(T=2.0 ** -21), INVALID), (dict(z=None), INVALID), (dict(tok=None), INVALID), (dict(lp=None), INVALID),
    (dict(ids=None), INVALID), (dict(top=None), INVALID), (dict(st=None), INVALID), (dict(ldz=499), INVALID),
    (dict(z=A16 + 1), INVALID), (dict(t=F32, z=A16 + 2), INVALID), (dict(tok=A16 + 1), INVALID),
    (dict(count=A16 + 1), INVALID), (dict(lp=A16 + 1), INVALID), (dict(H=A16 + 1), INVALID), (dict(ids=A16 + 2), INVALID),
    (dict(top=A16 + 2), INVALID), (dict(st=A16 + 4), INVALID), (dict(w=A16 + 8), INVALID),
    (dict(ldz=2**62, M=2**10), INVALID), (dict(n=65), UNSUPPORTED), (dict(M=2**31), UNSUPPORTED),
    (dict(V=2**30 + 1, ldz=2**31), UNSUPPORTED),
])
def test_token_logprobs_refusals(m, kw, status):
    assert _score(m, **kw) == status


def test_token_logprobs_workspace(m):
    f = m.mosaic_token_logprobs_workspace_bytes
    for M, V, n in ((20, 1 << 20, 20), (1, 1 << 30, 64), (100, 300000, 0)):
        need = f(M, V, n)
        if need:
            assert _score(m, M=M, V=V, ldz=V, n=n, wb=need - 1) == INVALID and _score(m, M=M, V=V, ldz=V, n=n, w=None) == INVALID
    for bad in ((-1, 5, 5), (5, -1, 5), (5, 5, -1), (5, 5, 65), (2**31, 5, 5), (5, 2**30 + 1, 5)):
        with pytest.raises(ValueError):
            f(*bad)
    assert _score(m, M=0, z=None, tok=None, lp=None, st=None, ids=None) == 0


def _score_grad(m, z=A16, ldz=500, M=10, V=500, t=BF16, tok=A16, T=1.0, count=None, st=A16, H=None, g=A16, h=None,
                grad=B16, ldg=500):
    return m.lib.mosaic_token_logprobs_grad(z, ldz, M, V, t, tok, T, count, st, H, g, h, grad, ldg, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(V=0), INVALID), (dict(t=2), INVALID), (dict(T=0.0), INVALID),
    (dict(z=None), INVALID), (dict(tok=None), INVALID), (dict(g=None), INVALID), (dict(g=None, tok=None), INVALID),
    (dict(h=A16), INVALID), (dict(st=None), INVALID), (dict(grad=None), INVALID), (dict(ldz=499), INVALID),
    (dict(ldg=499), INVALID), (dict(grad=A16, ldg=501), INVALID), (dict(grad=B16 + 1), INVALID), (dict(st=A16 + 4), INVALID),
    (dict(g=A16 + 1), INVALID), (dict(h=A16 + 1, H=A16), INVALID), (dict(h=A16, H=A16 + 1), INVALID),
    (dict(M=2**31), UNSUPPORTED), (dict(V=2**30 + 1, ldz=2**31, ldg=2**31), UNSUPPORTED),
])
def test_token_logprobs_grad_refusals(m, kw, status):
    assert _score_grad(m, **kw) == status
    assert _score_grad(m, M=0, z=None, tok=None, g=None, st=None, grad=None) == 0


def test_binding_refuses_host_tensors_and_shapes(m):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        m.mosaic_add_layernorm(x)
    with pytest.raises(ValueError):
        m.mosaic_layernorm_grad(x, x, torch.zeros(4, 2, dtype=torch.float64))
    with pytest.raises(ValueError):
        m.mosaic_quantize_rows_mxfp4(x)
    with pytest.raises(ValueError):
        m.mosaic_token_logprobs(x)
    with pytest.raises(ValueError):
        m.mosaic_token_logprobs_grad(x, None, x, None)
    with pytest.raises(ValueError):
        m.mosaic_add_layernorm(torch.zeros(4))
    with pytest.raises(ValueError):
        m.mosaic_add_layernorm(x, torch.ones(63))
    with pytest.raises(TypeError):
        m.mosaic_add_layernorm(x, torch.ones(64), torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.mosaic_layernorm_grad(x, torch.zeros(4, 63), x)
    with pytest.raises(TypeError):
        m.mosaic_layernorm_grad(x, x.bfloat16(), x)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.mosaic_quantized_logits_mxfp4(q, s, q, s[:, :1])
    with pytest.raises(ValueError):
        m.mosaic_quantized_logits_mxfp4(q, s, q[:, :16], s[:, :1])
    with pytest.raises(ValueError):
        m.mosaic_quantized_logits_mxfp4(q, s, q, s, M=5)
    with pytest.raises(ValueError):
        m.mosaic_masked_logits_mxfp4(torch.zeros(4, 65), torch.zeros(4, dtype=torch.int32), q, s)
    with pytest.raises(ValueError):
        m.mosaic_token_logprobs(x, logprob=torch.zeros(4))
