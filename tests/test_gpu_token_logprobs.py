"""Token log-probabilities, entropy, top alternatives and their gradient against 64-bit
arithmetic."""
import math

import pytest
import torch

import head64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _draw(seed, M, V, dtype, std=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = (torch.randn(M, V, generator=g, device=DEV) * std).to(dtype)
    t = torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)
    return z, t, torch.randn(M, generator=g, device=DEV), torch.randn(M, generator=g, device=DEV)


def _all(m, z, t, T=1.0, n=5, what="", **kw):
    lp, H, ids, top, st = m.mosaic_token_logprobs(z, t, temperature=T, top_n=n, with_entropy=True, **kw)
    head64.check_logprobs(z, t, T, lp, H, ids, top, st, what)
    return lp, H, ids, top, st


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [0, 1, 2, 5, 20, 63, 64])
@pytest.mark.parametrize("M,V", [(3, 1), (5, 7), (4, 64), (9, 500), (33, 2048), (5, 2049), (20, 5003), (7, 16411),
                                 (5, 32000), (3, 65537), (3, 126464), (2, 300001)])
def test_rows(m, M, V, n, dtype):
    z, t, g, h = _draw(V + n, M, V, dtype)
    lp, H, ids, top, st = m.mosaic_token_logprobs(z, t, top_n=n, with_entropy=True)
    head64.check_logprobs(z, t, 1.0, lp, H, ids, top, st, f"{M} x {V}")
    # without the entropy: the same numbers
    lp2, H2, ids2, top2, st2 = m.mosaic_token_logprobs(z, t, top_n=n)
    assert H2 is None and torch.equal(lp, lp2) and torch.equal(st, st2)
    assert n == 0 or (torch.equal(ids, ids2) and torch.equal(top, top2))
    if n == 5:
        grad = m.mosaic_token_logprobs_grad(z, t, st, g, entropy=H, grad_entropy=h)
        head64.check_logprobs_grad(z, t, 1.0, g, h, grad, f"{M} x {V}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V", [(1, 152064), (20, 152064), (129, 20000), (300, 126464), (900, 50000), (2500, 8192),
                                 (3000, 1000), (2100, 20000), (5000, 300), (1, 1 << 20), (130, 400000)])
def test_row_counts(m, M, V, dtype):
    z, t, g, h = _draw(M + V, M, V, dtype)
    lp, H, ids, top, st = _all(m, z, t, n=8, what=f"{M} x {V}")
    again = m.mosaic_token_logprobs(z, t, top_n=8, with_entropy=True)
    assert all(torch.equal(a, b) for a, b in zip(again, (lp, H, ids, top, st)))
    grad = m.mosaic_token_logprobs_grad(z, t, st, g, entropy=H, grad_entropy=h)
    head64.check_logprobs_grad(z, t, 1.0, g, h, grad, f"{M} x {V}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [2.0 ** -20, 0.1, 0.7, 2.0, 100.0, 2.0 ** 20])
@pytest.mark.parametrize("V", [100, 5003, 40000])
def test_temperatures(m, V, T, dtype):
    z, t, g, h = _draw(V, 6, V, dtype)
    lp, H, _, _, st = _all(m, z, t, T=T)
    grad = m.mosaic_token_logprobs_grad(z, t, st, g, entropy=H, grad_entropy=h, temperature=T)
    head64.check_logprobs_grad(z, t, T, g, h, grad)


def _special(V, dtype):
    """Rows whose order or range is out of the ordinary."""
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dtype).min
    z = torch.randn(26, V, generator=g)
    z[0] = 0.0                                           # all equal
    z[1] = torch.arange(V) * 2.0 ** -6                   # ascending (in bf16: with ties)
    z[2] = -torch.arange(V) * 2.0 ** -6                  # descending
    z[3] = -math.inf
    z[3, V // 2] = 1.0                                   # one entry allowed
    z[4] = low
    z[4, V // 3:V // 3 + 5] = torch.randn(5, generator=g)[:max(0, min(5, V - V // 3))]   # five, by the lowest value
    z[5] = low                                           # nothing but masks of the lowest value
    z[6] = -math.inf                                     # nothing at all
    z[7, V - 1] = math.inf
    z[8, V // 2] = math.nan
    z[9] = math.nan
    z[10] = torch.where(torch.rand(V, generator=g) < 0.9, torch.tensor(-math.inf), z[10])
    z[11] *= 1e4
    z[12] = z[12] * 3 + 1e4
    z[13] *= 1e37
    z[14] = 60.0 * (torch.arange(V) == 3 % V)            # confident
    z[15] = torch.where(torch.arange(V) % 2 == 0, torch.tensor(0.0), torch.tensor(-0.0))
    z[16] = torch.floor(z[16])                           # many ties
    z[17] = torch.arange(V).flip(0) // 7 * 0.5           # descending in steps
    z[18] = -3e38 + 0 * z[18]
    z[18, V // 2] = 3e38
    z[19] *= 1e-40
    z[20] = torch.arange(V) // 1000 * 1.0                # ascending in steps
    z[21] = torch.where(torch.arange(V) < V - 70, torch.tensor(0.0), z[21].abs() + 1)   # the largest at the end
    z[22] = torch.where(torch.arange(V) > 70, torch.tensor(0.0), z[22].abs() + 1)
    z[23] = -1e4
    z[24, 0] = -math.inf
    z[25, V - 1] = 50.0
    return z.to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 20, 64])
@pytest.mark.parametrize("V,copies", [(1, 1), (6, 100), (511, 12), (1000, 1), (1000, 100), (9001, 12), (9001, 100),
                                      (20000, 1), (20000, 100), (126464, 1), (126464, 12)])
def test_special_rows(m, V, n, copies, dtype):
    z = _special(V, dtype).repeat(copies, 1)
    M = z.shape[0]
    g = torch.Generator(device=DEV).manual_seed(n)
    t = torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)
    t[3 % M], t[7 % M] = V // 2, V - 1
    lp, H, _, _, st = _all(m, z, t, n=n, what=f"{V}")
    up, uh = torch.randn(M, generator=g, device=DEV), torch.randn(M, generator=g, device=DEV)
    for T in (1.0, 0.7):
        if T != 1.0:
            lp, H, _, _, st = _all(m, z, t, T=T, n=n)
        grad = m.mosaic_token_logprobs_grad(z, t, st, up, entropy=H, grad_entropy=uh, temperature=T)
        head64.check_logprobs_grad(z, t, T, up, uh, grad, f"{V}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [300, 9000, 40000])
def test_absent_tokens_and_parts(m, V, dtype):
    z, t, g, h = _draw(V, 8, V, dtype)
    t[1], t[2], t[3], t[4] = -1, V, 2 ** 31 - 1, -100
    lp, H, _, _, st = _all(m, z, t)
    assert bool((lp[1:5] == 0).all())
    grad = m.mosaic_token_logprobs_grad(z, t, st, g)
    head64.check_logprobs_grad(z, t, 1.0, g, None, grad)
    assert bool((grad[1:5] == 0).all())
    only = m.mosaic_token_logprobs_grad(z, None, st, None, entropy=H, grad_entropy=h)
    head64.check_logprobs_grad(z, None, 1.0, None, h, only)
    lp, H2, ids, top, st2 = m.mosaic_token_logprobs(z, with_entropy=True)
    assert lp is None and ids is None and top is None and torch.equal(H, H2) and torch.equal(st, st2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V,extra,shift", [(9, 500, 3, 1), (9, 5003, 1, 3), (40, 33000, 5, 2), (300, 20000, 8, 1)])
def test_strides_in_place_and_counts(m, M, V, extra, shift, dtype):
    z, t, g, h = _draw(V, M, V, dtype)
    room = torch.full((M * (V + extra) + shift,), 7.0, dtype=dtype, device=DEV)
    zs = room[shift:].view(M, V + extra)[:, :V]
    zs.copy_(z)
    want = m.mosaic_token_logprobs(z, t, top_n=6, with_entropy=True)
    got = m.mosaic_token_logprobs(zs, t, top_n=6, with_entropy=True)
    head64.check_logprobs(z, t, 1.0, *got)
    assert torch.equal(got[2], want[2])
    lp, H, ids, top, st = want
    grad = m.mosaic_token_logprobs_grad(z, t, st, g, entropy=H, grad_entropy=h)
    for c in (-2, 0, 1, M // 2, M + 5):
        k = max(0, min(c, M))
        count = torch.tensor([c], dtype=torch.int32, device=DEV)
        bufs = [torch.full_like(x, 3) for x in want]
        m.mosaic_token_logprobs(z, t, top_n=6, count=count, logprob=bufs[0], entropy=bufs[1], top_ids=bufs[2],
                                top_logprobs=bufs[3], stats=bufs[4])
        for a, b in zip(bufs, want):
            assert torch.equal(a[:k], b[:k]) and bool((a[k:] == 3).all())
        to = torch.full_like(grad, 3)
        m.mosaic_token_logprobs_grad(z, t, st, g, entropy=H, grad_entropy=h, count=count, grad=to)
        assert torch.equal(to[:k], grad[:k]) and bool((to[k:] == 3).all())
    m.mosaic_token_logprobs_grad(zs, t, st, g, entropy=H, grad_entropy=h, grad=zs)
    head64.check_logprobs_grad(z, t, 1.0, g, h, zs)
    assert bool((room[:shift] == 7).all()) and bool((room[shift:].view(M, -1)[:, V:] == 7).all())


def test_gradient_against_differences(m):
    z, t, g, h = _draw(1, 4, 700, F32)
    for T in (1.0, 0.7):
        _, H, _, _, st = m.mosaic_token_logprobs(z, t, temperature=T, with_entropy=True)
        grad = m.mosaic_token_logprobs_grad(z, t, st, g, entropy=H, grad_entropy=h, temperature=T).double()

        def value(x):
            lp = torch.log_softmax(x / T, dim=1)
            return (g.double() * lp.gather(1, t.long()[:, None])[:, 0] - h.double() * (lp * lp.exp()).sum(1)).sum()
        gen = torch.Generator(device=DEV).manual_seed(2)
        for _ in range(4):
            v = torch.randn(z.shape, generator=gen, device=DEV, dtype=torch.float64)
            e = 1e-4
            diff = (value(z.double() + e * v) - value(z.double() - e * v)) / (2 * e)
            # e^2 / 6 of a third derivative of the gradient's order, and 2^10 half steps of fp32
            assert abs(float(diff) - float((grad * v).sum())) <= 1e-4 * float((grad * v).abs().sum())


def test_long_rows_of_memory(m):
    # offsets past 2^31 elements: the last rows of a large array
    V = 126464
    M = (1 << 31) // V + 2
    z = torch.zeros(M, V, dtype=BF, device=DEV)
    z[-2:] = torch.randn(2, V, generator=torch.Generator().manual_seed(0)).to(BF).to(DEV)
    t = torch.full((M,), 77, dtype=torch.int32, device=DEV)
    lp, H, ids, top, st = m.mosaic_token_logprobs(z, t, top_n=3, with_entropy=True)
    head64.check_logprobs(z[-2:], t[-2:], 1.0, lp[-2:], H[-2:], ids[-2:], top[-2:], st[-2:])
    assert ids[:-2].eq(torch.arange(3, device=DEV)).all()
    g = torch.ones(M, device=DEV)
    grad = m.mosaic_token_logprobs_grad(z, t, st, g)
    head64.check_logprobs_grad(z[-2:], t[-2:], 1.0, g[-2:], None, grad[-2:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V,n", [(600, 40000, 20), (600, 130000, 3), (3, 130000, 20), (3, 130001, 64), (700, 5003, 5)])
def test_largest_logits_close_together_in_memory(m, M, V, n, dtype):
    """The largest logits in a few of every 256 chunks of 16 bytes, so that few threads see them all."""
    z, t, _, _ = _draw(V, M, V, dtype)
    v = torch.arange(V, device=z.device)
    for lanes in (1, 2, 12):
        x = torch.where(v // (8 if dtype == BF else 4) % 256 < lanes, z + 50, z)
        head64.check_logprobs(x, t, 1.0, *m.mosaic_token_logprobs(x, t, top_n=n, with_entropy=True), f"{M} x {V}, {lanes}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V,n", [(2, 2**20, 64), (1, 2**20 + 5, 63), (16, 2**20, 2)])
def test_largest_logits_in_a_stretch_of_a_long_row(m, M, V, n, dtype):
    """All of the largest logits at one end of the row, or in its middle, sorted either way."""
    z, t, _, _ = _draw(V + n, M, V, dtype)
    v = torch.arange(V, device=z.device)
    for lo, hi in ((0, 9 * 16384), (V - 150000, V), (400000, 400064)):
        x = torch.where((v >= lo) & (v < hi), z + 50, z)
        head64.check_logprobs(x, t, 1.0, *m.mosaic_token_logprobs(x, t, top_n=n, with_entropy=True), f"{lo}:{hi}")
    x = z.sort(dim=1).values
    for y in (x, x.flip(1)):
        head64.check_logprobs(y, t, 1.0, *m.mosaic_token_logprobs(y, t, top_n=n, with_entropy=True), "sorted")


def test_more_rows_than_a_launch_holds(m):
    """17 million rows of one logit, or of two with one absent."""
    M = 2**24 + 5
    z = torch.randn(M, 1, device=DEV)
    t = torch.zeros(M, dtype=torch.int32, device=DEV)
    lp, H, ids, top, st = m.mosaic_token_logprobs(z, t, top_n=1, with_entropy=True)
    # The entropy's sum is held against a rounded maximum k in powers of two: |k| < 16, so what k lost, off, is
    # 2^-21 at most, and off - off, where both passed two roundings of 2^-24, is 4 * 2^-45 at most.
    assert bool((H.abs() <= 2.0 ** -43).all())
    assert bool((lp == 0).all()) and bool((ids == 0).all()) and bool((top == 0).all())
    assert torch.equal(st[:, :1], z) and bool((st[:, 1] == 0).all())
    g = m.mosaic_token_logprobs_grad(z, t, st, torch.ones(M, device=DEV))
    # 1 - p, where p's two exponentials are off by 2^-23 and its quotient and product by 2^-24 each
    assert bool((g.abs() <= 3 * 2.0 ** -23 + 2.0 ** -40).all())
    two = torch.stack([z[:, 0], torch.full((M,), -float("inf"), device=DEV)], 1)
    n = torch.tensor([M - 3], dtype=torch.int32, device=DEV)
    lp = torch.full((M,), 5.0, device=DEV)
    m.mosaic_token_logprobs(two, t, logprob=lp, count=n)
    assert bool((lp[:M - 3] == 0).all()) and bool((lp[M - 3:] == 5).all())
