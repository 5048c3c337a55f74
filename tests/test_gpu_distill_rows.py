"""Every row of the distillation loss and its gradient, in the forms for many long rows too:
special rows in a workgroup's first and later turns, the gradient in place, device counts,
replays."""
import math

import pytest
import torch

import device64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _data(seed, M, V, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = (2 * torch.randn(M, V, generator=g, device=DEV)).to(dtype)
    t = 2 * torch.randn(M, K, generator=g, device=DEV)
    ids = torch.randint(0, V, (M, K), generator=g, dtype=torch.int32, device=DEV)
    w = torch.rand(M, generator=g, device=DEV) - 0.3
    return z, t, ids, w


def _special(z, t, ids):
    """Every kind of special row, near each other and in a workgroup's first and later turns
    (workgroups walk their rows 256 apart)."""
    M, V = z.shape
    low = torch.finfo(z.dtype).min
    for base in (0, 256, 257 + 16, 512):
        if base + 14 > M:
            continue
        ids[base] = -1                               # no entry
        t[base + 1] = -INF                           # no entry either
        ids[base + 2] = ids[base + 2, 0]             # one entry, named by all
        ids[base + 3, 1] = ids[base + 3, 0]
        ids[base + 4, ::2] = V                       # some outside
        z[base + 5] = -INF
        z[base + 6, V // 3] = float("nan")
        z[base + 7, V - 1] = INF
        z[base + 8, int(ids[base + 8, 0])] = -INF    # an infinite loss
        z[base + 9] = low
        z[base + 10, :-1] = -INF                     # one logit left, the last
        z[base + 11, : V // 2] = low
        ids[base + 12, 0] = V - 1                    # the row's ends
        ids[base + 12, 1] = 0
        ids[base + 13] = -1                          # no entry, and a NaN
        z[base + 13, 5] = float("nan")


# forms: a wave to 16 waves per row, the stream's three lengths with one and with more rows per
# workgroup, rows read twice, and rows in parts
SHAPES = [(BF, 40, 1001), (BF, 2100, 2047), (BF, 2100, 8001), (BF, 300, 16001), (BF, 700, 30011), (BF, 600, 65001),
          (BF, 600, 70001), (BF, 530, 100003), (BF, 600, 126464), (BF, 560, 140003), (BF, 540, 160001), (BF, 60, 50021),
          (F32, 40, 1001), (F32, 600, 8001), (F32, 530, 30011), (F32, 600, 40001), (F32, 530, 50003), (F32, 540, 70001),
          (F32, 530, 80001), (F32, 60, 50021)]


@pytest.mark.parametrize("dtype,M,V", SHAPES)
def test_distill_every_row(m, dtype, M, V):
    z, t, ids, w = _data(M + V, M, V, 9, dtype)
    _special(z, t, ids)
    loss, stats, grad = m.mosaic_distill_topk(z, t, ids, temperature=1.3, with_grad=True, grad_loss=w)
    device64.check_distill(z, t, ids, 1.3, w, loss, stats, grad, "both")
    loss, stats, _ = m.mosaic_distill_topk(z, t, ids, temperature=1.3)
    device64.check_distill(z, t, ids, 1.3, w, loss, stats, None, "loss")
    grad = m.mosaic_distill_topk_grad(z, t, ids, stats, grad_loss=w, temperature=1.3)
    device64.check_distill(z, t, ids, 1.3, w, None, None, grad, "gradient")


@pytest.mark.parametrize("dtype,M,V", [s for s in SHAPES if s[1] >= 300])
def test_distill_every_row_in_place_and_strided(m, dtype, M, V):
    pad = 13
    z, t, ids, w = _data(M + V, M, V + pad, 5, dtype)
    ids = ids % V
    for off in (8, 3):
        _special(z[:, off:off + V], t, ids)
        want = m.mosaic_distill_topk(z[:, off:off + V], t, ids, with_grad=True, grad_loss=w)
        for later in (False, True):
            zc = z.clone()
            view = zc[:, off:off + V]
            if later:
                got = [m.mosaic_distill_topk_grad(view, t, ids, want[1], grad_loss=w, grad=view)]
                device64.check_distill(z[:, off:off + V], t, ids, 1.0, w, None, None, view, "gradient in place")
            else:
                got = m.mosaic_distill_topk(view, t, ids, grad_loss=w, grad=view)
                for a, b in zip(got, want):          # the bits of the call with buffers of its own
                    assert torch.equal(torch.nan_to_num(a, 77.0), torch.nan_to_num(b, 77.0))
            assert got[-1].data_ptr() == view.data_ptr()
            assert torch.equal(torch.nan_to_num(zc[:, :off], 77.0), torch.nan_to_num(z[:, :off], 77.0))
            assert torch.equal(torch.nan_to_num(zc[:, off + V:], 77.0), torch.nan_to_num(z[:, off + V:], 77.0))
        z = z.nan_to_num(0.0, 0.0, 0.0)


@pytest.mark.parametrize("dtype,M,V", [s for s in SHAPES if s[1] >= 500])
def test_distill_long_rows_device_count(m, dtype, M, V):
    z, t, ids, w = _data(M, M, V, 6, dtype)
    want = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
    for cnt in (-1, 0, 1, 255, 256, 257, M - 1, M + 3):
        n = max(0, min(cnt, M))
        count = torch.tensor([cnt], dtype=torch.int32, device=DEV)
        outs = [torch.full_like(x, 3) for x in want]
        m.mosaic_distill_topk(z, t, ids, count=count, loss=outs[0], stats=outs[1], grad=outs[2], grad_loss=w)
        for got, ref in zip(outs, want):
            assert torch.equal(got[:n], ref[:n]) and bool((got[n:] == 3).all()), cnt


@pytest.mark.parametrize("dtype,M,V", [(BF, 600, 70001), (BF, 540, 160001), (F32, 600, 40001), (BF, 60, 50021)])
def test_distill_long_rows_replayed(m, dtype, M, V):
    z, t, ids, w = _data(M, M, V, 6, dtype)
    count = torch.tensor([M], dtype=torch.int32, device=DEV)
    outs = [torch.zeros(M, device=DEV), torch.zeros(M, 2, device=DEV), torch.zeros_like(z)]
    ws = torch.zeros(max(16, m.mosaic_distill_topk_workspace_bytes(M, V, 6)), dtype=torch.uint8, device=DEV)

    def call():
        m.mosaic_distill_topk(z, t, ids, count=count, loss=outs[0], stats=outs[1], grad=outs[2], grad_loss=w, workspace=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for i, n in enumerate((M, 0, 300, M)):
        z.copy_(torch.roll(z, 1 + i, 1))
        count.fill_(n)
        call()                                       # eager, on the new data
        want = [x.clone() for x in outs]
        for x in outs:
            x.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a[:n], b[:n]) and bool((a[n:] == 5).all())


def test_distill_more_rows_than_a_grid(m):
    M = (1 << 20) + 37                               # workgroups walk over rows beyond 2^20
    z, t, ids, w = _data(3, M, 5, 2, F32)
    loss, stats, grad = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
    device64.check_distill(z, t, ids, 1.0, w, loss, stats, grad, "both")
    device64.check_distill(z, t, ids, 1.0, w, None, None, m.mosaic_distill_topk_grad(z, t, ids, stats, grad_loss=w), "grad")


@pytest.mark.parametrize("dtype,M,V", SHAPES + [(BF, 20, 152064), (BF, 1000, 50001), (F32, 300, 126464), (BF, 300, 200003)])
def test_distill_exact_sums(m, dtype, M, V):
    # T = log2(e) as fp32 holds it makes the exponentials powers of two, and whole logits down to -6
    # below the maximum make their sums exact in any order: a chunk left out or taken twice, or a
    # sum in fewer bits, shows beside a few half steps
    U = device64.U32
    T = float(torch.tensor(math.log2(math.e), dtype=F32))
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.randint(-6, 1, (M, V), generator=g, device=DEV).to(dtype)
    z[:, V // 2] = 0
    z += torch.randint(-9, 9, (M, 1), generator=g, device=DEV).to(dtype)
    t = torch.randint(-4, 5, (M, 8), generator=g, device=DEV).float()
    ids = torch.randint(0, V, (M, 8), generator=g, dtype=torch.int32, device=DEV)
    w = torch.rand(M, generator=g, device=DEV) + 0.1
    loss, stats, grad = m.mosaic_distill_topk(z, t, ids, temperature=T, with_grad=True, grad_loss=w)
    alone, stats2, _ = m.mosaic_distill_topk(z, t, ids, temperature=T)
    later = m.mosaic_distill_topk_grad(z, t, ids, stats, grad_loss=w, temperature=T)
    assert torch.equal(stats, stats2)                # the same exact sum, whatever the form
    step = max(1, (1 << 25) // V)
    for i in range(0, M, step):
        r = slice(i, min(M, i + step))
        zd = z[r].double()
        top = zd.amax(1, keepdim=True)
        logq = (zd - top) / T
        l = torch.logsumexp(logq, 1, keepdim=True)
        logq -= l
        p = torch.softmax(t[r].double() / T, 1)
        # the powers stand for exp(x) with an x of T's half step: 5 U at 6 below the maximum, once
        # for the term and once for the sum; the logarithm: 4 U of l
        assert bool(((stats[r, 1:].double() - l).abs() <= (4 * l + 6) * U).all()), i
        lq = torch.gather(logq, 1, ids[r].long())
        want = (T * T * (p * (p.log() - lq)).sum(1))
        # p: 6 U of T's half step twice, a division; the terms and their sums: 20 U of each
        size = (p * (p.log().abs() + lq.abs() + l)).sum(1) + (p * 14 * (p.log().abs() + lq.abs() + 1)).sum(1)
        tol = T * T * U * (20 * size + 4 * l[:, 0] + 6)
        for got in (loss, alone):
            assert bool(((got[r].double() - want).abs() <= tol).all()), i
        q = torch.exp(logq)
        P = torch.zeros_like(zd).scatter_add_(1, ids[r].long(), p)
        tg = T * w[r].double()[:, None]
        grad_want = tg * (q - P)
        # q: 10 U of T's half step, five roundings (and exp(l) where l is given: l's error and 4 U);
        # P: 14 U, a division, two products, eight additions; the difference and the stored type
        for got, extra in ((grad, 0.0), (later, 4 * l + 10)):
            tol = tg * U * (q * (16 + extra) + P * 26) + grad_want.abs() * (device64.HALF[dtype] + 2 * U)
            bad = (got[r].double() - grad_want).abs() > tol
            assert not bool(bad.any()), (i, bad.nonzero()[:3].tolist())
