"""Distillation loss and gradient against the plain 64-bit form, and against differences."""
import math

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _data(seed, M, V, K, dtype, t_dtype=F32):
    g = torch.Generator().manual_seed(seed)
    z = (2 * torch.randn(M, V, generator=g)).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(M)]).to(torch.int32) if K <= V else \
        torch.randint(0, V, (M, K), generator=g, dtype=torch.int32)
    t = (2 * torch.randn(M, K, generator=g)).to(t_dtype)
    w = torch.rand(M, generator=g) - 0.3
    return z.to(DEV), t.to(DEV), ids.to(DEV), w.to(DEV)


def _check(m, z, t, ids, T, w, what):
    ref = plain64.distill(z, t, ids, T, w)
    loss, stats, none = m.mosaic_distill_topk(z, t, ids, temperature=T)
    assert none is None
    plain64.check_distill(ref, loss, stats, None, what + " loss")
    loss2, stats2, grad = m.mosaic_distill_topk(z, t, ids, temperature=T, with_grad=True, grad_loss=w)
    plain64.check_distill(ref, loss2, stats2, grad, what + " both")
    plain64.check_distill(ref, None, None,
                          m.mosaic_distill_topk_grad(z, t, ids, stats, grad_loss=w, temperature=T), what + " grad")
    return ref


SIZES = [(1, 1, 1), (1, 2, 1), (3, 5, 4), (2, 1000, 1), (7, 1021, 17), (64, 504, 32), (65, 2048, 64), (5, 8192, 256),
         (4, 8200, 100), (3, 33333, 33), (2, 126464, 64), (20, 152064, 32), (300, 4096, 8), (700, 1024, 16),
         (1, 200000, 1024), (2, 300007, 5), (520, 20000, 3)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V,K", SIZES)
def test_distill_sizes(m, M, V, K, dtype):
    z, t, ids, w = _data(M + V + K, M, V, K, dtype)
    _check(m, z, t, ids, 1.0, w, "T=1")


# row counts and lengths on both sides of each form's limits
FORMS = [(200, 2047), (200, 2049), (2100, 2048), (2050, 8192), (150, 8191), (140, 8193), (130, 16384), (130, 16385),
         (130, 32768), (130, 32769), (129, 38401), (129, 57601), (129, 65536), (129, 65537), (129, 76801),
         (129, 99841), (129, 130561), (129, 153600), (129, 153601), (2049, 4097), (1025, 16400), (300, 126464),
         (128, 102400), (128, 102401), (40, 204800), (40, 204801), (257, 32800), (768, 32769), (769, 32769), (200, 210000)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V", FORMS)
def test_distill_forms(m, M, V, dtype):
    g = torch.Generator(device=DEV).manual_seed(M + V)
    z = (2 * torch.randn(M, V, generator=g, device=DEV)).to(dtype)
    t = 2 * torch.randn(M, 7, generator=g, device=DEV)
    ids = torch.randint(-1, V, (M, 7), generator=g, dtype=torch.int32, device=DEV)
    w = torch.rand(M, generator=g, device=DEV)
    # the plain form on rows at both ends and in between; the others against the two calls' agreement
    rows = torch.tensor(sorted({0, 1, M // 3, M // 2, M - 2, M - 1}), device=DEV)
    ref = plain64.distill(z[rows], t[rows], ids[rows], 1.0, w[rows])
    loss, stats, grad = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
    plain64.check_distill(ref, loss[rows], stats[rows], grad[rows], "both")
    alone, stats2, _ = m.mosaic_distill_topk(z, t, ids)
    plain64.check_distill(ref, alone[rows], stats2[rows], None, "loss")
    later = m.mosaic_distill_topk_grad(z, t, ids, stats2, grad_loss=w)
    plain64.check_distill(ref, None, None, later[rows], "gradient")
    assert torch.equal(stats[:, 0], stats2[:, 0]) and torch.equal(stats[:, 0], z.float().amax(1))
    # both carry L_ABS of l's error on each row's q, and a rounding of the result
    size = float(w.max()) * 2 * (8 * plain64.L_ABS + 2 * plain64.HALF[dtype])
    assert float((later.float() - grad.float()).abs().max()) <= size
    assert float((loss - alone).abs().max()) <= 64 * plain64.L_ABS


@pytest.mark.parametrize("T", [2.0 ** -20, 0.05, 0.7, 3.0, 100.0, 2.0 ** 20])
@pytest.mark.parametrize("t_dtype", [BF, F32])
def test_distill_temperatures(m, T, t_dtype):
    z, t, ids, w = _data(3, 33, 1500, 20, BF, t_dtype)
    if T < 0.01:   # arguments of 64 at most, which the tolerance counts
        z, t = (z.float() * T).to(BF), (t.float() * T).to(t_dtype)
    _check(m, z, t, ids, T, w, f"T={T}")


def _sparse(V, K, M):
    """Rows with absent, repeated and missing entries."""
    z, t, ids, w = _data(V, M, V, K, F32)
    ids[0] = -1                                  # nothing present
    ids[1, ::2] = V                              # half outside
    ids[2] = ids[2, 0]                           # one entry named K times
    ids[3, 1:] = ids[3, 0]
    t[3, K // 2:] = -INF
    t[4] = -INF                                  # present ids, no mass
    t[5, 1:] = -INF                              # one entry left
    ids[6] = 2**31 - 1
    ids[7] = -2**31
    ids[8, : K // 2] = ids[8, K - K // 2:]       # every id twice
    t[9] = torch.finfo(F32).min                  # the lowest value everywhere: equal shares
    t[10, 0] = 1e30                              # all mass on one entry
    return z, t, ids, w


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,K", [(1000, 16), (1003, 40), (40000, 9), (150000, 64)])
def test_distill_absent_and_repeated_entries(m, V, K, dtype):
    z, t, ids, w = _sparse(V, K, 12)
    z = z.to(dtype)
    ref = _check(m, z, t, ids, 1.5, w, "sparse")
    for row in (0, 4, 6, 7):
        assert float(ref["loss"][row]) == 0
    loss, _, grad = m.mosaic_distill_topk(z, t, ids, temperature=1.5, with_grad=True)
    assert bool((loss[[0, 4, 6, 7]] == 0).all()) and bool((grad[[0, 4, 6, 7]] == 0).all())


def test_distill_without_entries(m):
    z, _, _, _ = _data(1, 5, 300, 4, BF)
    none = torch.empty((5, 0), device=DEV)
    loss, stats, grad = m.mosaic_distill_topk(z, none, none.to(torch.int32), with_grad=True)
    assert bool((loss == 0).all()) and bool((grad == 0).all()) and bool((stats[:, 0] == z.float().amax(1)).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [100, 1024, 5003, 70000, 152064])
def test_distill_masked_logits(m, V, dtype):
    z, t, ids, w = _data(V, 10, V, 6, dtype)
    low = torch.finfo(dtype).min
    z[0, 50:] = -INF                             # a masked vocabulary
    ids[0] = torch.arange(6, dtype=torch.int32)
    z[1, 50:] = low
    ids[1] = torch.arange(6, dtype=torch.int32)
    z[2] = -INF                                  # nothing left
    z[3, 7] = float("nan")
    z[4, 9] = INF
    z[5, int(ids[5, 0])] = -INF                  # mass where the student has none: infinite loss
    z[6] = low                                   # all equal
    z[7] = -INF
    z[7, 11] = 3.0                               # one entry left, the teacher elsewhere
    ids[7] = torch.arange(20, 26, dtype=torch.int32)
    z[8] = 0.0
    z[8, : V // 2] = -INF
    ids[8] = V // 2 + torch.arange(6, dtype=torch.int32)
    ref = _check(m, z, t, ids, 1.0, w, "masked")
    loss, _, grad = m.mosaic_distill_topk(z, t, ids, with_grad=True)
    assert math.isinf(float(loss[5])) and math.isinf(float(loss[7]))
    assert torch.isnan(loss[2:5]).all() and torch.isnan(grad[2:5]).all()
    assert torch.isfinite(grad[[0, 1, 5, 6, 7, 8, 9]]).all() and math.isinf(float(ref["loss"][5]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [300, 9000, 40000, 120000])
def test_distill_large_magnitudes(m, V, dtype):
    # logits around +-1e3 .. 1e38: only those next to the maximum count, whatever its size
    z, t, ids, w = _data(V, 10, V, 6, F32)
    for row, base in enumerate((1e3, -1e5, 3e7, -1e9, 7e9, -1e12, 1e18, -1e25, 3e38, -3e38)):
        z[row] = torch.nextafter(torch.full((V,), base, device=DEV), torch.tensor(-3.4e38, device=DEV)) \
            if dtype == F32 else base * 1.01
        z[row, ::3] = base
        z[row, 1::3] = base - 1 - abs(base) * 2.0 ** -6   # well below
    _check(m, z.to(dtype), t, ids, 0.5, w, "large")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V", [(3, 70000), (40, 1000), (600, 1001), (300, 9000)])
def test_distill_strides_and_in_place(m, M, V, dtype):
    z, t, ids, w = _data(M, M, V + 29, 5, dtype)
    ids = torch.randint(0, V, ids.shape, dtype=torch.int32, device=DEV)
    for off in (0, 8, 3):
        zs = z[:, off:off + V]
        ref = plain64.distill(zs, t, ids, 2.0, w)
        buf = torch.full((M, V + 16), 7.0, dtype=dtype, device=DEV)
        loss, stats, grad = m.mosaic_distill_topk(zs, t, ids, temperature=2.0, grad_loss=w, grad=buf[:, 8:8 + V])
        plain64.check_distill(ref, loss, stats, grad, "strided")
        assert bool((buf[:, :8] == 7).all()) and bool((buf[:, 8 + V:] == 7).all())
        zc = z.clone()
        loss2, stats2, g2 = m.mosaic_distill_topk(zc[:, off:off + V], t, ids, temperature=2.0, grad_loss=w,
                                                  grad=zc[:, off:off + V])
        plain64.check_distill(ref, loss2, stats2, g2, "in place")
        assert torch.equal(zc[:, :off], z[:, :off]) and torch.equal(zc[:, off + V:], z[:, off + V:])
        zc = z.clone()
        g3 = m.mosaic_distill_topk_grad(zc[:, off:off + V], t, ids, stats, grad_loss=w, temperature=2.0,
                                        grad=zc[:, off:off + V])
        plain64.check_distill(ref, None, None, g3, "gradient in place")


@pytest.mark.parametrize("M,V", [(20, 152064), (40, 1000), (600, 2000)])
def test_distill_device_count(m, M, V):
    z, t, ids, w = _data(M, M, V, 9, BF)
    want = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
    for cnt in (-2, 0, 1, M // 2, M, M + 9):
        n = max(0, min(M, cnt))
        count = torch.tensor([cnt], dtype=torch.int32, device=DEV)
        outs = [torch.full_like(x, 3) for x in want]
        m.mosaic_distill_topk(z, t, ids, count=count, loss=outs[0], stats=outs[1], grad=outs[2], grad_loss=w)
        outs.append(torch.full_like(z, 3))
        m.mosaic_distill_topk_grad(z, t, ids, want[1], grad_loss=w, count=count, grad=outs[3])
        for got, ref in zip(outs, (*want, want[2])):
            assert bool((got[n:] == 3).all()), cnt
        assert torch.equal(outs[0][:n], want[0][:n]) and torch.equal(outs[1][:n], want[1][:n])
        assert torch.equal(outs[2][:n], want[2][:n])
        ref = plain64.distill(z[:n], t[:n], ids[:n], 1.0, w[:n]) if n else None
        if n:
            plain64.check_distill(ref, None, None, outs[3][:n], "gradient")


def test_distill_gradient_against_differences(m):
    # (loss(z + h e) - loss(z - h e)) / 2h in fp64, from the plain form, at some entries
    z, t, ids, _ = _data(9, 3, 40, 6, F32)
    ids[0, 1] = ids[0, 0]
    T, h = 1.7, 1e-5
    grad = m.mosaic_distill_topk(z, t, ids, temperature=T, with_grad=True)[2].cpu().double()
    for v in (int(ids[0, 0]), int(ids[1, 2]), 0, 17, 39):
        up, dn = z.cpu().double().clone(), z.cpu().double().clone()
        up[:, v] += h
        dn[:, v] -= h
        diff = (plain64.distill(up, t, ids, T)["loss"] - plain64.distill(dn, t, ids, T)["loss"]) / (2 * h)
        # h^2 of the third derivative (at most T^-1 here) and fp64's rounding over 2h, well under 1e-8
        assert ((grad[:, v] - diff).abs() <= 1e-8 + 2.0 ** -12 * (diff.abs() + T)).all()


def test_distill_same_bits_every_call(m):
    for M, V in ((20, 152064), (600, 5000)):
        z, t, ids, w = _data(M, M, V, 33, BF)
        a = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
        b = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_distill_past_32_bit_offsets(m):
    V = 126464
    M = (1 << 31) // V + 40                      # more than 2^31 logits
    z = torch.zeros((M, V), dtype=BF, device=DEV)
    rows = [0, 1, M // 2, M - 2, M - 1]
    z[rows] = torch.randn(len(rows), V, device=DEV).to(BF)
    t, ids = torch.randn(M, 7, device=DEV), torch.randint(0, V, (M, 7), dtype=torch.int32, device=DEV)
    loss, stats, grad = m.mosaic_distill_topk(z, t, ids, with_grad=True)
    ref = plain64.distill(z[rows], t[rows], ids[rows], 1.0)
    plain64.check_distill(ref, loss[rows], stats[rows], grad[rows], "far rows")
    grad = m.mosaic_distill_topk_grad(z, t, ids, stats, grad=z)
    plain64.check_distill(ref, None, None, grad[rows], "far rows in place")


def test_distill_other_streams_at_once(m):
    data = [_data(s, 24, 100000, 11, BF) for s in (1, 2)]
    want = [m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w) for z, t, ids, w in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = []
    for _ in range(4):
        for s, (z, t, ids, w) in zip(streams, data):
            got.append(m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w, stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2]))
